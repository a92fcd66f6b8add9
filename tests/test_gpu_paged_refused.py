"""Requests that the page step refused, in the calls behind it: their rows get zeros, and the others their time."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    from self_speculative_block_gb300 import build, gocr
    build.build()
    gocr.load()
    return gocr


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _beside_tokens(rows, kv, Hq, Hkv, d, tokens=16, keys=500, ps=16):
    """Single tokens of some requests; between two of them, others of `rows` rows and `kv` keys each."""
    r = torch.Generator(device="cuda").manual_seed(1)
    width = -(-keys // ps)
    n_pages = tokens * width
    kc, vc = (torch.randn((n_pages, Hkv, ps, d), generator=r, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(n_pages, generator=r, device="cuda").to(torch.int32).view(tokens, width)
    half = tokens // 2
    n = [1] * half + list(rows) + [1] * half
    kv_len = [keys] * half + list(kv) + [keys] * half
    order = list(range(half)) + [0] * len(rows) + list(range(half, tokens))
    T = sum(n)
    q = torch.randn((T, Hq, d), generator=r, device="cuda").bfloat16()
    return dict(q=q, kc=kc, vc=vc, table=table[order].contiguous(), cu=i32([0] + n).cumsum(0).to(torch.int32), kv_len=i32(kv_len)), n, half


@pytest.mark.parametrize("kind", ["verify", "draft"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,kv", [([16384], [0]), ([700, 0, 3, 5000], [0, 0, 2, 0]), ([1] * 3000, [0] * 3000),
                                     ([1, 2, 33] * 300, [0, 1, 5] * 300)])
def test_rows_of_refused_requests(g, rows, kv, d, kind):
    """Zeros and -infinity in the rows that have no key, the other rows as without these requests."""
    Hq, Hkv = 6, 2
    k = g.FWD_DRAFT if kind == "draft" else g.FWD_VERIFY
    c, n, half = _beside_tokens(rows, kv, Hq, Hkv, d)
    T = c["q"].shape[0]
    o, lse = torch.full((T, Hq, d), 7.0, device="cuda").bfloat16(), torch.full((Hq, T), 7.0, device="cuda")
    g.op_attention_paged(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["kv_len"], kind=k, o=o, lse=lse)
    g.op_status()
    none = []
    for m, l in zip(n, c["kv_len"].tolist()):
        none += [l == 0 or (l - m + i < 0 and (k != g.FWD_DRAFT or i == 0)) for i in range(m)]
    none = torch.tensor(none, device="cuda")
    assert (o[none] == 0).all() and (lse[:, none] == -math.inf).all()
    assert torch.isfinite(lse[:, ~none]).all() and not (lse[:, ~none] == 7.0).any()
    # every other request by itself: the same within twice the sums' and roundings' errors (2^-8 a rounding to bf16 of o, and of p)
    keep = torch.cat([torch.arange(half, device="cuda"), torch.arange(T - half, T, device="cuda")])
    R = len(n)
    alone = torch.cat([torch.arange(half, device="cuda"), torch.arange(R - half, R, device="cuda")])
    o1, lse1 = g.op_attention_paged(c["q"][keep], c["kc"], c["vc"], c["table"][alone], i32(list(range(2 * half + 1))),
                                    c["kv_len"][alone], kind=k)
    bound = c["vc"].abs().max().float()
    assert ((o[keep].float() - o1.float()).abs() <= 4 * 2.0 ** -8 * bound).all()
    assert ((lse[:, keep] - lse1).abs() <= 1e-4).all()


def test_a_refused_prompt_does_not_hold_up_the_others(g):
    """16,384 rows of 12 heads of 128 are 50 MB of zeros, 10 us for the whole device; one SM would take 2,700."""
    c, _, _ = _beside_tokens([16384], [0], 12, 4, 128, tokens=64)
    T = c["q"].shape[0]
    out = dict(o=torch.empty_like(c["q"]), lse=torch.empty((12, T), device="cuda"))
    out["workspace"] = torch.empty((g.load().gocr_op_attention_paged_workspace(T, 12, 4, 128),), dtype=torch.uint8, device="cuda")
    best = math.inf
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.op_attention_paged(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["kv_len"], **out)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    assert best < 0.5  # milliseconds
