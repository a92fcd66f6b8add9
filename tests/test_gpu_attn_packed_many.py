"""The packed attention over thousands of short sequences: right, and in a time
that grows with their number."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, TC = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    from self_speculative_block_gb300 import build, gocr
    build.build()
    gocr.load()
    return gocr


def _case(n, L, Hq, Hkv, d, seed):
    r = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda h: torch.randn((n * L, h, d), generator=r, device="cuda").bfloat16()
    return rnd(Hq), rnd(Hkv), rnd(Hkv), rnd(Hq)


@pytest.mark.parametrize("n,L,d", [(255, 3, 64), (256, 7, 128), (257, 7, 128), (2049, 2, 64), (30_000, 5, 64), (1000, 130, 128)])
def test_attention_packed_of_many_equal_sequences(g, n, L, d):
    """Every sequence against the batched formulas in 64 bits; every seventh slot of cu_seqlens is an empty one."""
    Hq, Hkv = 4, 2
    q, k, v, do = _case(n, L, Hq, Hkv, d, seed=n)
    cu = (torch.arange(n + 1, device="cuda") * L).to(torch.int32)
    cu = torch.repeat_interleave(cu, 1 + (torch.arange(n + 1, device="cuda") % 7 == 0))
    o, lse = g.op_attention_packed(q, k, v, cu)
    dq, dk, dv = g.op_attention_packed_backward(do, q, k, v, o, lse, cu)
    g.op_status()
    Q, dO = (t.view(n, L, Hq, d).double().transpose(1, 2) for t in (q, do))
    K, V = (t.view(n, L, Hkv, d).double().transpose(1, 2).repeat_interleave(Hq // Hkv, 1) for t in (k, v))
    c = d ** -0.5
    S = (Q @ K.transpose(2, 3) * c).masked_fill(torch.ones((L, L), dtype=torch.bool, device="cuda").triu(1), -math.inf)
    P = torch.softmax(S, 3)
    O = P @ V
    dP = dO @ V.transpose(2, 3)
    x = dP - (dO * O).sum(3, keepdim=True)
    dS = P * x
    group = lambda t: t.view(n, Hkv, Hq // Hkv, L, d).sum(2)
    ref = dict(o=O, dq=c * dS @ K, dk=group(c * dS.transpose(2, 3) @ Q), dv=group(P.transpose(2, 3) @ dO))
    # an exponential is off by its argument's error: of d / 16 truncated steps, and lse's
    e = 4 * (d / 16 + 16) * TC * c * (Q.abs() @ K.abs().transpose(2, 3)).amax(3, keepdim=True) + 64 * TC
    tol_o = (U + 2 * e) * (P @ V.abs()) + U * O.abs()
    e_x = (d / 16 + 16) * TC * (dO.abs() @ V.abs().transpose(2, 3)) + (dO.abs() * tol_o).sum(3, keepdim=True)
    e_s = 2 * e * dS.abs() + P * e_x + U * (dS.abs() + P * e_x)
    tol = dict(o=tol_o, dq=c * (e_s @ K.abs()), dk=group(c * e_s.transpose(2, 3) @ Q.abs()),
               dv=group((P * (2 * e + U)).transpose(2, 3) @ dO.abs()))
    for name, got in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        got = got.view(n, L, -1, d).double().transpose(1, 2)
        # fp32 sums of up to L terms, in steps of 16, and the result's rounding
        deep = (L / 16 + 64) * TC * ref[name].abs().amax()
        bad = ~((got - ref[name]).abs() <= tol[name] * (1 + U) + deep + U * ref[name].abs() + 1e-30)
        assert not bad.any(), (name, int(bad.sum()))
    err = (lse.double() - torch.logsumexp(S, 3).transpose(0, 1).reshape(Hq, -1)).abs()
    assert (err <= (e[..., 0].transpose(0, 1).reshape(Hq, -1) + 2.0 ** -20)).all()


def test_attention_packed_time_grows_with_the_sequences(g):
    """Four times the sequences take about four times as long, not sixteen."""
    L, Hq, Hkv, d = 5, 4, 2, 64

    def time(n):
        q, k, v, do = _case(n, L, Hq, Hkv, d, seed=1)
        cu = (torch.arange(n + 1, device="cuda") * L).to(torch.int32)
        o, lse = g.op_attention_packed(q, k, v, cu)
        best = []
        for f in (lambda: g.op_attention_packed(q, k, v, cu, o=o, lse=lse),
                  lambda: g.op_attention_packed_backward(do, q, k, v, o, lse, cu)):
            t = []
            for _ in range(5):
                a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                a.record()
                f()
                b.record()
                b.synchronize()
                t.append(a.elapsed_time(b))
            best.append(min(t))
        return best

    few, many = time(10_000), time(40_000)
    for name, a, b in zip(("forward", "backward"), few, many):
        assert b < 7 * a, (name, a, b)


def test_attention_packed_of_the_most_sequences(g):
    """2^20 sequences of one row: o is v, lse the row's only score, dv the sum of the group's do, and
    what is left of dS = P (dP - delta) is the difference of two fp32 sums of the same products."""
    n, Hq, Hkv, d = 1 << 20, 2, 1, 64
    q, k, v, do = _case(n, 1, Hq, Hkv, d, seed=2)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    o, lse = g.op_attention_packed(q, k, v, cu)
    dq, dk, dv = g.op_attention_packed_backward(do, q, k, v, o, lse, cu)
    g.op_status()
    assert torch.equal(o, v.expand(n, Hq, d))
    score = d ** -0.5 * (q.double() * k.double()).sum(2).T
    # a sum of 64 products in steps of 16, times a scale that is a power of two, through a base 2 logarithm
    err = (d / 16 + 16) * TC * d ** -0.5 * (q.double() * k.double()).abs().sum(2).T + 8 * TC * score.abs()
    assert ((lse.double() - score).abs() <= err).all()
    assert torch.equal(dv, do.float().sum(1, keepdim=True).bfloat16())
    # P is 1 within the error of its exponent
    mag = (do.double() * v.double()).abs().sum(2)
    left = ((d / 16 + 16 + d) * TC * mag + 4 * (err.T + TC) * mag)[..., None] * d ** -0.5
    assert (dq.double().abs() <= left * k.double().abs() * (1 + U) + 1e-38).all()
    assert (dk.double().abs() <= (left * q.double().abs()).sum(1, keepdim=True) * (1 + U) + 1e-38).all()
