"""Sizes past 32-bit offsets and odd alignments of the embedding gradient and
the cross entropy: tables of more than 2^31 elements, vocabularies that need
more CTAs than usual for their zeros, token arrays that begin anywhere."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32 = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    from self_speculative_block_gb300 import build, gocr
    build.build()
    gocr.load()
    yield gocr
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _grad_into(g, dy, ids, d_embed, d_mask):
    """gocr_op_embed_backward into given arrays."""
    lib = g.load()
    (T, H), V = dy.shape, d_embed.shape[0]
    ws = torch.full((lib.gocr_op_embed_backward_workspace(T, H),), 255, dtype=torch.uint8, device="cuda")
    rc = lib.gocr_op_embed_backward(g.DTYPE_BF16 if dy.dtype == torch.bfloat16 else g.DTYPE_F32, dy.data_ptr(),
                                    ids.data_ptr(), d_embed.data_ptr(), d_mask.data_ptr() if d_mask is not None else None,
                                    T, H, V, 1.0, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == g.GOCR_OK, g.last_error()


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("T", [1, 3, 6, 18, 1000, 5003])
def test_embed_gradient_of_token_arrays_that_begin_anywhere(g, T, offset):
    """Integer gradients, so that every sum is exact; the output holds NaN before the call."""
    V, H = 700, 24
    r = _gen(T + offset)
    ids = torch.randint(-1, V + 2, (T + offset,), generator=r, device="cuda", dtype=torch.int32)[offset:]
    dy = torch.randint(-3, 4, (T, H), generator=r, device="cuda").float()
    dE = torch.full((V, H), math.nan, device="cuda")
    dm = torch.full((H,), math.nan, device="cuda")
    _grad_into(g, dy, ids, dE, dm)
    at = torch.where(ids < 0, V, torch.where(ids < V, ids, V + 1)).long()
    ref = torch.zeros((V + 2, H), device="cuda").index_add(0, at, dy)
    assert torch.equal(dE, ref[:V]) and torch.equal(dm, ref[V])


@pytest.mark.parametrize("T", [32768, 32769, 32768 + 128, 100_003])
@pytest.mark.parametrize("V,kind", [(1, "even"), (300, "even"), (2500, "even"), (50_000, "even"), (4000, "often"),
                                    (97, "runs")])
def test_embed_gradient_of_many_tokens(g, T, V, kind):
    """Runs of every length against pieces of every length; integer gradients, so that every sum is exact."""
    H = 24
    r = _gen(T + V)
    u = torch.rand(T, generator=r, device="cuda")
    if kind == "runs":  # token v occurs 8 v + 1 times or so, which puts runs' ends everywhere in the pieces
        ids = torch.repeat_interleave(torch.arange(V, device="cuda"), torch.arange(V, device="cuda") * 8 + 1)
        ids = ids[torch.randint(0, len(ids), (T,), generator=r, device="cuda")].to(torch.int32)
    else:
        ids = (torch.exp(u * math.log(V)) - 1 if kind == "often" else u * V).long().clamp(0, V - 1).to(torch.int32)
    ids[torch.rand(T, generator=r, device="cuda") < 0.2] = -1
    ids[torch.rand(T, generator=r, device="cuda") < 0.05] = V + 3
    dy = torch.randint(-3, 4, (T, H), generator=r, device="cuda").float()
    dE = torch.full((V, H), math.nan, device="cuda")
    dm = torch.full((H,), math.nan, device="cuda")
    _grad_into(g, dy, ids, dE, dm)
    at = torch.where(ids < 0, V, torch.where(ids < V, ids, V + 1)).long()
    ref = torch.zeros((V + 2, H), device="cuda").index_add(0, at, dy)
    assert torch.equal(dE, ref[:V]) and torch.equal(dm, ref[V])


@pytest.mark.parametrize("V,H", [(10_000_123, 8), (32768 * 304 + 1, 8), (31, 8), (33, 4096)])
def test_embed_gradient_writes_every_row(g, V, H):
    """Tables with more rows than the usual CTAs' shares hold, and with fewer rows than bits in a word."""
    T = 999
    r = _gen(V)
    ids = (torch.rand(T, generator=r, device="cuda", dtype=torch.float64) * V).long().clamp(0, V - 1).to(torch.int32)
    ids[0], ids[1] = 0, V - 1
    dy = torch.randint(-3, 4, (T, H), generator=r, device="cuda").bfloat16()
    dE = torch.full((V, H), math.nan, dtype=torch.bfloat16, device="cuda")
    dm = torch.full((H,), math.nan, dtype=torch.bfloat16, device="cuda")
    _grad_into(g, dy, ids, dE, dm)
    assert not dm.any()
    ref = torch.zeros((V, H), device="cuda").index_add(0, ids.long(), dy.float()).bfloat16()
    assert torch.equal(dE, ref)


def test_embed_past_32_bit_offsets(g):
    V, H, T = 2_200_000, 1024, 777  # 2.25e9 elements
    r = _gen(1)
    ids = V - 1 - torch.randint(0, 5000, (T,), generator=r, device="cuda", dtype=torch.int32)
    ids[:5] = torch.tensor([0, -1, V - 1, V, 2097152], device="cuda", dtype=torch.int32)
    E = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    E[-5000:] = torch.randn((5000, H), generator=r, device="cuda").bfloat16()
    y = g.op_embed(ids, E)
    keep = (ids >= 0) & (ids < V)
    assert torch.equal(y[keep], E[ids[keep].long()]) and not y[~keep].any()
    del E
    dy = torch.randint(-3, 4, (T, H), generator=r, device="cuda").bfloat16()
    dE = torch.full((V, H), math.nan, dtype=torch.bfloat16, device="cuda")
    _grad_into(g, dy, ids, dE, None)
    named = ids[keep].unique().long()
    ref = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    ref[named] = torch.stack([dy[ids == v].float().sum(0) for v in named]).bfloat16()
    assert torch.equal(dE, ref)


def test_linear_ce_past_32_bit_offsets(g):
    """A head of 2.25e9 elements: loss, lse, dx, and the rows of dw at both ends."""
    T, V, H = 40, 2_200_000, 1024
    r = _gen(2)
    x = torch.randn((T, H), generator=r, device="cuda").bfloat16()
    w = torch.empty((V, H), dtype=torch.bfloat16, device="cuda")
    for c in range(0, V, 200_000):
        w[c:c + 200_000] = (H ** -0.5 * torch.randn((min(200_000, V - c), H), generator=r, device="cuda")).bfloat16()
    labels = V - 1 - torch.randint(0, 1000, (T,), generator=r, device="cuda", dtype=torch.int32)
    labels[0], labels[1], labels[2] = -1, 0, V - 1
    dloss = torch.rand(T, generator=r, device="cuda") + 0.5
    loss, lse = g.op_linear_ce(x, w, labels)
    dx, dw = g.op_linear_ce_backward(dloss, x, w, labels, lse)
    g.op_status()

    xd = x.double()
    parts = range(0, V, 100_000)
    z = torch.cat([xd @ w[c:c + 100_000].double().T for c in parts], 1)
    # |x||w|, of which a product's rounding takes (H / 16 + 16) truncations of 2^-23
    zmag = torch.cat([xd.abs() @ w[c:c + 100_000].double().abs().T for c in parts], 1)
    dz = ((H / 16 + 16) * 2.0 ** -23) * zmag
    del zmag
    ref = torch.logsumexp(z, 1)
    has = labels >= 0
    at = torch.where(has, labels, 0).long()[:, None]
    zl = z.gather(1, at)[:, 0]
    want = torch.where(has, ref - zl, 0.0)
    # a sum over the vocabulary in fp32: columns of a tile, then tiles of 128 to 256 columns, 128 at a time
    tol_lse = dz.amax(1) + (80 + V / 128 / 128 + 8 * z.abs().amax(1)) * F32 + 4 * F32 * ref.abs()
    tol_loss = torch.where(has, tol_lse + dz.gather(1, at)[:, 0] + F32 * want.abs(), 0.0)
    assert ((lse.double() - ref).abs() <= tol_lse).all()
    assert ((loss.double() - want).abs() <= tol_loss).all()
    f = torch.where(has, dloss.double(), 0.0)[:, None]
    p = torch.exp(z - ref[:, None])
    del z
    gr = p * f
    gr.scatter_add_(1, at, -f)
    dg = p * f.abs() * (dz + tol_lse[:, None] + 16 * F32) + gr.abs() * 2.0 ** -8
    dg.scatter_add_(1, at, f * F32)
    del p, dz
    sums = torch.zeros((3, T, H), dtype=torch.float64, device="cuda")
    for c in parts:
        wd = w[c:c + 100_000].double()
        sums[0] += gr[:, c:c + 100_000] @ wd
        sums[1] += dg[:, c:c + 100_000] @ wd.abs()
        sums[2] += gr[:, c:c + 100_000].abs() @ wd.abs()
    u = 2.0 ** -8
    tol = (sums[1] + (V / 16 + 64) * 2.0 ** -23 * sums[2]) * (1 + u) + u * sums[0].abs() + 1e-38
    assert ((dx.double() - sums[0]).abs() <= tol).all()
    for c in (slice(0, 1000), slice(2_097_000, 2_098_000), slice(V - 1000, V)):
        d = gr[:, c].T @ xd
        tol = (dg[:, c].T @ xd.abs() + (T / 16 + 64) * 2.0 ** -23 * (gr[:, c].abs().T @ xd.abs())) * (1 + u) + u * d.abs() + 1e-38
        assert ((dw[c].double() - d).abs() <= tol).all()


def test_attention_packed_past_32_bit_offsets(g):
    """1,870 sequences, 2.15e9 elements of q: each has the bits that it has alone."""
    Hq, Hkv, d = 12, 4, 128
    lens = [1000, 1, 1003, 996] * 467 + [1000, 130]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    T = int(cu[-1])
    assert T * Hq * d > 2 ** 31
    r = _gen(3)

    def rows(h):
        t = torch.empty((T, h, d), dtype=torch.bfloat16, device="cuda")
        for c in range(0, T, 100_000):
            t[c:c + 100_000] = torch.randn((min(100_000, T - c), h, d), generator=r, device="cuda").bfloat16()
        return t

    q, k, v, do = rows(Hq), rows(Hkv), rows(Hkv), rows(Hq)
    o, lse = g.op_attention_packed(q, k, v, cu)
    dq, dk, dv = g.op_attention_packed_backward(do, q, k, v, o, lse, cu)
    g.op_status()
    for s in (0, 700, len(lens) - 3, len(lens) - 2, len(lens) - 1):
        a, b = int(cu[s]), int(cu[s + 1])
        one = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        part = [t[a:b].clone() for t in (q, k, v, do)]
        o1, l1 = g.op_attention_packed(*part[:3], one)
        grads = g.op_attention_packed_backward(part[3], *part[:3], o1, l1, one)
        assert torch.equal(o1, o[a:b]) and torch.equal(l1, lse[:, a:b]), s
        for x, y in zip(grads, (dq, dk, dv)):
            assert torch.equal(x, y[a:b]), s


def test_attention_packed_rows_far_apart(g):
    """Row pitches of 2^20 elements and more: the offset of the last rows of q, k and v passes 2^32 bytes."""
    Hq, Hkv, d, T = 4, 2, 64, 2100
    ld = 2 ** 20 + 8
    r = _gen(4)
    wide = torch.zeros((T, ld), dtype=torch.bfloat16, device="cuda")
    n = (Hq + 2 * Hkv) * d
    wide[:, :n] = torch.randn((T, n), generator=r, device="cuda").bfloat16()
    x = wide[:, :n].unflatten(1, (Hq + 2 * Hkv, d))
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu = torch.tensor([0, 900, 2100], dtype=torch.int32, device="cuda")
    do = torch.randn((T, Hq, d), generator=r, device="cuda").bfloat16()
    o, lse = g.op_attention_packed(q, k, v, cu)
    near = [t.contiguous() for t in (q, k, v)]
    o1, l1 = g.op_attention_packed(*near, cu)
    assert torch.equal(o, o1) and torch.equal(lse, l1)
    for a, b in zip(g.op_attention_packed_backward(do, q, k, v, o, lse, cu),
                    g.op_attention_packed_backward(do, *near, o, lse, cu)):
        assert torch.equal(a, b)
