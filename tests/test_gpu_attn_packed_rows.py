"""Rows of the packed attention beside others: the same bits whatever the scores of a
neighbouring sequence do, and where a non-finite row of the own sequence reaches."""
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


def _run(g, q, k, v, do, cu, scale):
    o, lse = g.op_attention_packed(q, k, v, cu, scale=scale)
    dq, dk, dv = g.op_attention_packed_backward(do, q, k, v, o, lse, cu, scale=scale)
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


@pytest.mark.parametrize("d,scale,size", [(128, None, 20.0), (128, None, 60.0), (64, None, 40.0), (64, 0.3, 10.0)])
def test_attention_packed_row_does_not_depend_on_growing_neighbours(g, d, scale, size):
    """The last query tile of a sequence holds the next one's rows, too.  Their scores grow from key
    block to key block, so that their running maxima, and the sums that follow them, are rescaled."""
    H, n, m = 4, 1055, 200
    r = torch.Generator(device="cuda").manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=r, device="cuda")
    q, k, v, do = (size * rnd(n, H, d)).bfloat16(), rnd(n, H, d).bfloat16(), rnd(n, H, d).bfloat16(), rnd(n, H, d).bfloat16()
    cu = torch.tensor([0, n, n + m], dtype=torch.int32, device="cuda")
    alone = _run(g, q, k, v, do, cu[:2], scale)
    late = sum((b + 1) * k[64 * b + 32].float() for b in range(n // 64))  # [H, d]
    score = (4 * late).bfloat16()[0].float() @ k[:, 0].float().T * (scale or d ** -0.5) * 1.4427
    ref, grown = score[:64].max(), 0
    for b in range(1, n // 64):
        if score[64 * b:64 * b + 64].max() - ref > 8:
            ref, grown = score[64 * b:64 * b + 64].max(), grown + 1
    assert grown >= 3
    more = [rnd(m, H, d).bfloat16() for _ in range(3)]
    both = _run(g, torch.cat([q, (4 * late).bfloat16().expand(m, H, d)]),
                *(torch.cat([a, b]) for a, b in zip((k, v, do), more)), cu, scale)
    for name, a in alone.items():
        assert torch.equal(both[name][:, :n] if name == "lse" else both[name][:n], a), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["q", "k", "v", "do"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_packed_non_finite_row(g, d, what, bad):
    """Rows before row 300 of one sequence do not see it: o and lse keep their bits (with a
    non-finite v, those of the blocks of 128 before its own), dq of the blocks before, too."""
    n, H, at = 500, 2, 300
    r = torch.Generator(device="cuda").manual_seed(d)
    t = {x: torch.randn((n, H, d), generator=r, device="cuda").bfloat16() for x in ("q", "k", "v", "do")}
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    clean = _run(g, t["q"], t["k"], t["v"], t["do"], cu, None)
    t[what] = t[what].clone()
    t[what][at, 1, 5] = bad
    got = _run(g, t["q"], t["k"], t["v"], t["do"], cu, None)
    block = at // 128 * 128
    keep = block if what == "v" else at
    assert torch.equal(got["o"][:keep], clean["o"][:keep]) and torch.equal(got["lse"][:, :keep], clean["lse"][:, :keep])
    assert torch.equal(got["dq"][:block], clean["dq"][:block])
    assert all(torch.equal(got[x][:, 0], clean[x][:, 0]) for x in ("o", "dq", "dk", "dv"))  # the other head
    if what in ("q", "do"):  # row 300 is the only one that reads them: later blocks of keys are not its
        assert all(torch.equal(got[x][block + 128:], clean[x][block + 128:]) for x in ("o", "dq", "dk", "dv"))
