"""Rows of the packed attention beside rows of other sequences: the same bits,
whatever the neighbours' scores do."""
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
