"""Causal attention over packed sequences, forward and backward, against a plain
64-bit implementation.  Tolerances are error bounds of the arithmetic, element
by element: a rounding to bf16 counts 2^-8 of the value, a tensor-core sum one
truncation of 2^-23 per 16-deep step, an exponential 2^-22.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, F32, TC = 2.0 ** -8, 2.0 ** -24, 2.0 ** -23


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    from self_speculative_block_gb300 import build, gocr
    build.build()
    gocr.load()
    return gocr


def _case(lens, Hq, Hkv, d, seed, pad=0, qscale=1.0):
    r = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens) + pad
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=r, device="cuda")
    qkv[:, :Hq] *= qscale
    qkv = qkv.bfloat16()
    do = torch.randn((T, Hq, d), generator=r, device="cuda").bfloat16()
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], do, cu


def _ref(q, k, v, do, lens, scale):
    """Values in 64 bits, and the bounds of the kernels' errors, of the rows in sequences."""
    Hq, d = q.shape[1:]
    Hkv = k.shape[1]
    G = Hq // Hkv
    n_rows = sum(lens)
    z = lambda h: torch.zeros((n_rows, h, d), dtype=torch.float64, device=q.device)
    val = dict(o=z(Hq), dq=z(Hq), dk=z(Hkv), dv=z(Hkv), lse=torch.zeros((Hq, n_rows), dtype=torch.float64, device=q.device))
    tol = {n: torch.zeros_like(t) for n, t in val.items()}
    t0 = 0
    for n in lens:
        r = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        seen = torch.tril(torch.ones((n, n), dtype=torch.bool, device=q.device))
        deep = (n / 16 + 64) * TC  # sums over rows
        for h in range(Hq):
            Q, K, V, dO = q[r, h].double(), k[r, h // G].double(), v[r, h // G].double(), do[r, h].double()
            S = (Q @ K.T * scale).masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(S, 1)
            P = torch.exp(S - lse[:, None])
            big = torch.where(seen, S, 0.0).abs().amax(1)
            # relative error of an exponential: its argument's and its own
            e = (torch.where(seen, (Q.abs() @ K.abs().T) * scale, 0.0).amax(1) * (d / 16 + 16) * TC + 4 * big * F32 + 4 * F32)
            e_lse = e + n * F32 + 4 * F32 * lse.abs()
            O = P @ V
            tol_o = (U + 2 * e + deep)[:, None] * (P @ V.abs()) + U * O.abs() + 1e-38
            val["o"][r, h], val["lse"][h, r] = O, lse
            tol["o"][r, h], tol["lse"][h, r] = tol_o, e_lse
            dP = dO @ V.T
            delta = (dO * O).sum(1)
            x = dP - delta[:, None]
            dS = P * x
            e_p = (e + e_lse)[:, None] * P  # P from the forward call's lse
            e_x = (d / 16 + 16) * TC * (dO.abs() @ V.abs().T) + ((dO.abs() * tol_o).sum(1) + d * F32 * (dO * O).abs().sum(1))[:, None]
            e_s = torch.where(seen, e_p * x.abs() + P * e_x + U * (dS.abs() + P * e_x), 0.0)
            dS = torch.where(seen, dS, 0.0)
            val["dq"][r, h] = scale * dS @ K
            tol["dq"][r, h] = scale * (e_s @ K.abs() + deep * (dS.abs() @ K.abs()))
            val["dk"][r, h // G] += scale * dS.T @ Q
            tol["dk"][r, h // G] += scale * (e_s.T @ Q.abs() + G * deep * (dS.abs().T @ Q.abs()))
            val["dv"][r, h // G] += P.T @ dO
            tol["dv"][r, h // G] += (e_p + U * P).T @ dO.abs() + G * deep * (P.T @ dO.abs())
    for n in ("dq", "dk", "dv"):
        tol[n] += U * (val[n].abs() + tol[n]) + 1e-38
    return val, tol


def _close(name, got, val, tol):
    n = val["lse"].shape[1]
    got = got[:, :n] if name == "lse" else got[:n]
    err = (got.double() - val[name]).abs()
    bad = ~(err <= tol[name])
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / tol[name].clamp(min=1e-300)).nan_to_num(float('inf')).max()):.3g} times the bound")


def _run(g, q, k, v, do, cu, scale=None):
    o, lse = g.op_attention_packed(q, k, v, cu, scale=scale)
    dq, dk, dv = g.op_attention_packed_backward(do, q, k, v, o, lse, cu, scale=scale)
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


LENS = [[1], [2, 1], [128], [129], [255], [256, 1], [257, 3], [64, 1, 193, 130, 311], [0, 5, 0, 0, 700, 0], [1] * 300,
        [127, 128, 129, 383, 384, 385], [1500], [40] * 37]


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (12, 4, 128), (1, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("lens", LENS, ids=lambda l: "x".join(map(str, l[:6])) + f"n{len(l)}")
def test_attention_packed_and_gradient(g, lens, Hq, Hkv, d):
    q, k, v, do, cu = _case(lens, Hq, Hkv, d, seed=sum(lens) + Hq)
    val, tol = _ref(q, k, v, do, lens, d ** -0.5)
    for name, got in _run(g, q, k, v, do, cu).items():
        _close(name, got, val, tol)
    g.op_status()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_packed_long(g, d):
    """A long sequence beside short ones: many key blocks, several query heads."""
    lens = [4501, 3, 700]
    q, k, v, do, cu = _case(lens, 2, 1, d, seed=d)
    val, tol = _ref(q, k, v, do, lens, d ** -0.5)
    for name, got in _run(g, q, k, v, do, cu).items():
        _close(name, got, val, tol)


def test_attention_packed_growing_maxima(g):
    """Scores that grow along the keys by hundreds: the running maximum moves in every block, and O with it."""
    lens, d = [900], 128
    q, k, v, do, cu = _case(lens, 2, 1, d, seed=4)
    ramp = torch.linspace(0.0, 12.0, 900, device="cuda")
    q, k = q.clone(), k.clone()
    q[:, :, 0] = 16.0
    k[:, :, 0] = ramp[:, None].bfloat16()
    val, tol = _ref(q, k, v, do, lens, 1.0)
    for name, got in _run(g, q, k, v, do, cu, scale=1.0).items():
        _close(name, got, val, tol)


def test_attention_packed_leaves_other_rows(g):
    """Rows behind the last sequence hold NaN and infinity: they reach nothing and their outputs stay."""
    lens, pad, Hq, Hkv, d = [130, 70], 77, 4, 2, 128
    q, k, v, do, cu = _case(lens, Hq, Hkv, d, seed=5, pad=pad)
    n, T = sum(lens), sum(lens) + pad
    val, tol = _ref(q, k, v, do, lens, d ** -0.5)
    for t in (q, k, v, do):
        t[n:] = math.nan
        t[n + 1] = math.inf
    mark = lambda *s, dt=torch.bfloat16: torch.full(s, 7.0, dtype=dt, device="cuda")
    o, lse = g.op_attention_packed(q, k, v, cu, o=mark(T, Hq, d), lse=mark(Hq, T, dt=torch.float32))
    dq, dk, dv = g.op_attention_packed_backward(do, q, k, v, o, lse, cu, dq=mark(T, Hq, d), dk=mark(T, Hkv, d),
                                                dv=mark(T, Hkv, d))
    for name, got in dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv).items():
        rest = got[:, n:] if name == "lse" else got[n:]
        assert (rest == 7.0).all(), name
        _close(name, got, val, tol)


def test_attention_packed_keeps_nan_in_its_sequence(g):
    lens, Hq, Hkv, d = [100, 90, 200], 2, 1, 64
    q, k, v, do, cu = _case(lens, Hq, Hkv, d, seed=6)
    good = _run(g, q, k, v, do, cu)
    for t in (q, k, v, do):
        t[100:190] = math.nan
    got = _run(g, q, k, v, do, cu)
    keep = torch.ones(390, dtype=torch.bool, device="cuda")
    keep[100:190] = False
    for name in good:
        a, b = (x[:, keep] if name == "lse" else x[keep] for x in (good[name], got[name]))
        assert torch.equal(a, b), name
        assert torch.isnan((got[name][:, ~keep] if name == "lse" else got[name][~keep])).all(), name


def test_attention_packed_row_does_not_depend_on_packing(g):
    """A sequence alone, and the same among others, at another place: the same bits."""
    d, Hq, Hkv = 128, 6, 2
    q, k, v, do, cu = _case([333], Hq, Hkv, d, seed=7)
    alone = _run(g, q, k, v, do, cu)
    q2, k2, v2, do2, cu2 = _case([50, 333, 129], Hq, Hkv, d, seed=8)
    for a, b in ((q2, q), (k2, k), (v2, v), (do2, do)):
        a[50:383] = b
    both = _run(g, q2, k2, v2, do2, cu2)
    for name in alone:
        assert torch.equal(both[name][:, 50:383] if name == "lse" else both[name][50:383], alone[name]), name
    again = _run(g, q2, k2, v2, do2, cu2)
    assert all(torch.equal(again[n], both[n]) for n in both)


def test_attention_packed_dense_and_strided_rows_agree(g):
    q, k, v, do, cu = _case([200, 17], 4, 4, 64, seed=9)
    a = _run(g, q, k, v, do, cu)
    b = _run(g, q.contiguous(), k.contiguous(), v.contiguous(), do, cu)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_attention_packed_nothing_to_do(g):
    q, k, v, do, cu = _case([5], 2, 1, 64, seed=10)
    e = g.op_attention_packed(q[:0], k[:0], v[:0], torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert e[0].shape == (0, 2, 64) and e[1].shape == (2, 0)
    o = torch.full_like(do, 3.0)
    g.op_attention_packed(q, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), o=o)
    g.op_attention_packed(q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda"), o=o)
    assert (o == 3.0).all()


def test_attention_packed_gradient_against_differences(g):
    """Sum of o * do along a direction, by central differences of the forward call."""
    lens, Hq, Hkv, d = [150, 60], 4, 2, 64
    q, k, v, do, cu = (t.contiguous() for t in _case(lens, Hq, Hkv, d, seed=11))
    got = _run(g, q, k, v, do, cu)
    ref, _ = _ref(q, k, v, do, lens, d ** -0.5)
    val = lambda q_, k_, v_: float((_ref(q_, k_, v_, do, lens, d ** -0.5)[0]["o"] * do.double()).sum())
    for i, name in enumerate(("dq", "dk", "dv")):
        step = [torch.zeros_like(t) for t in (q, k, v)]
        step[i] = (1e-4 * torch.sign(got[name].double()))
        base = [t.double() for t in (q, k, v)]
        diff = (val(*[b + s for b, s in zip(base, step)]) - val(*[b - s for b, s in zip(base, step)]))
        want = float((got[name].double() * 2 * step[i]).sum())
        # every term of the sum has one sign, so the gradient's relative error, about two roundings
        # of 2^-8 and P's, bounds the sum's; the steps' third-order term is far below it
        assert abs(diff - want) <= 4 * U * abs(diff), (name, diff, want)


def test_attention_packed_in_a_graph_and_on_a_stream(g):
    """The sequence borders are read on the device: a captured pass replays on other borders."""
    T, Hq, Hkv, d = 600, 4, 2, 64
    q, k, v, do, cu = _case([100, 500], Hq, Hkv, d, seed=12)
    want = _run(g, q, k, v, do, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _run(g, q, k, v, do, cu)
    s.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(g, q, k, v, do, cu)
    for cut in (100, 1, 599, 256):
        cu.copy_(torch.tensor([0, cut, T], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        fresh = _run(g, q, k, v, do, cu)
        assert all(torch.equal(out[n], fresh[n]) for n in out), cut
    g.op_status()


def test_attention_packed_rows_before_the_first_sequence(g):
    """cu_seqlens may start behind row 0: the rows before it belong to no sequence either."""
    lens, lead, Hq, Hkv, d = [70, 200], 33, 2, 1, 64
    q, k, v, do, cu = _case(lens, Hq, Hkv, d, seed=13, pad=lead)
    T = sum(lens) + lead
    roll = lambda t: torch.cat([torch.full_like(t[:lead], math.nan), t[:T - lead]])
    want = _run(g, q[:T - lead], k[:T - lead], v[:T - lead], do[:T - lead].contiguous(), cu)
    q2, k2, v2, do2 = (roll(t) for t in (q, k, v, do))
    o = torch.full_like(do2, 5.0)
    lse = torch.full((Hq, T), 5.0, device="cuda")
    g.op_attention_packed(q2, k2, v2, cu + lead, o=o, lse=lse)
    mark = lambda h: torch.full((T, h, d), 5.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = g.op_attention_packed_backward(do2, q2, k2, v2, o, lse, cu + lead, dq=mark(Hq), dk=mark(Hkv), dv=mark(Hkv))
    for name, got in dict(o=o, dq=dq, dk=dk, dv=dv).items():
        assert (got[:lead] == 5.0).all() and torch.equal(got[lead:], want[name]), name
    assert (lse[:, :lead] == 5.0).all() and torch.equal(lse[:, lead:], want["lse"])


def test_attention_packed_many_mixes_repeat(g):
    """Random mixes of short and long sequences, back to back: equal bits on every call and no wait given up."""
    import random
    rng = random.Random(3)
    for i in range(24):
        lens = [rng.choice([0, 1, 3, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300, 500]) for _ in range(rng.randint(1, 40))]
        if not sum(lens):
            continue
        Hkv = rng.randint(1, 4)
        q, k, v, do, cu = _case(lens, Hkv * rng.randint(1, 3), Hkv, rng.choice([64, 128]), seed=100 + i)
        first = _run(g, q, k, v, do, cu)
        for _ in range(5):
            again = _run(g, q, k, v, do, cu)
            assert all(torch.equal(again[n], first[n]) for n in first), lens
        g.op_status()


def test_attention_packed_on_two_streams_at_once(g):
    q, k, v, do, cu = _case([500, 300, 65], 6, 2, 128, seed=14)
    q2, k2, v2, do2, cu2 = _case([64] * 20, 4, 4, 64, seed=15)
    want, want2 = _run(g, q, k, v, do, cu), _run(g, q2, k2, v2, do2, cu2)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s):
            a = _run(g, q, k, v, do, cu)
        with torch.cuda.stream(t):
            b = _run(g, q2, k2, v2, do2, cu2)
        torch.cuda.synchronize()
        assert all(torch.equal(a[n], want[n]) for n in want) and all(torch.equal(b[n], want2[n]) for n in want2)
    g.op_status()


def test_attention_packed_many_sequences(g):
    """More sequences than one step of the search for a block takes, empty ones among them."""
    lens = [(i * 7) % 23 if i % 5 else 0 for i in range(1300)] + [300, 0, 129, 0]
    q, k, v, do, cu = _case(lens, 2, 1, 64, seed=8)
    val, tol = _ref(q, k, v, do, lens, 0.125)
    for name, got in _run(g, q, k, v, do, cu).items():
        _close(name, got, val, tol)
    g.op_status()
