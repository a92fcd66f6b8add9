"""The embedding and the LM-head cross entropy with their gradients, against
plain 64-bit implementations.  Every tolerance is an error bound of the
arithmetic, element by element: roundings to the output type count half a step
(eps / 2), fp32 sums one step of 2^-24 per addition and tensor-core sums one
truncation of 2^-23 per 16-deep step, each relative to the sum of magnitudes.
"""
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


U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative
F32 = 2.0 ** -24


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _close(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / tol.clamp(min=1e-300)).nan_to_num(float('inf')).max()):.3g} times the bound")


# ---------------------------------------------------------------------- embedding

def _embed_case(T, H, V, dt, seed, mask=0.3, bad=0.1, zipf=True):
    r = _gen(seed)
    u = lambda n: torch.rand(n, generator=r, device="cuda")
    ids = (torch.exp(u(T) * math.log(V)).long() - 1 if zipf else (u(T) * V).long()).clamp(0, V - 1)
    ids = torch.where(u(T) < mask, torch.full_like(ids, -1), ids)
    wrong = torch.tensor([-2, V, V + 7, 2 ** 31 - 1, -2 ** 31], device="cuda")
    ids = torch.where(u(T) < bad, wrong[torch.arange(T, device="cuda") % 5], ids).to(torch.int32)
    rnd = lambda *s: torch.randn(s, generator=r, device="cuda").to(dt)
    return ids, rnd(V, H), rnd(H), rnd(T, H)


EMBED = [(1, 8, 1), (33, 1536, 65536), (257, 264, 1000), (16, 64, 7), (17, 64, 7), (4097, 72, 513), (10240, 1536, 4096)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,V", EMBED)
def test_embed_rows(g, T, H, V, dt):
    ids, E, m, _ = _embed_case(T, H, V, dt, seed=T + H)
    scale = math.sqrt(H)
    y = g.op_embed(ids, E, m, scale=scale)
    i = ids.long()
    table = torch.cat([E.double(), m.double()[None], torch.zeros_like(m.double())[None]])
    at = torch.where((i >= 0) & (i < V), i, torch.where(i == -1, V, V + 1))
    ref = table[at] * scale
    _close(y, ref, ref.abs() * (U[dt] + 3 * F32), "y")  # scale to fp32, one product, one rounding
    # without an [M] row its positions are padding
    y0 = g.op_embed(ids, E, None, scale=scale)
    assert torch.equal(y0[i != -1], y[i != -1]) and not y0[i == -1].any()


def _embed_grad_ref(dy, ids, V, scale, mask):
    i = ids.long()
    at = torch.where((i >= 0) & (i < V), i, torch.where((i == -1) & mask, V, V + 1))
    z = torch.zeros((V + 2, dy.shape[1]), dtype=torch.float64, device=dy.device)
    ref = z.index_add(0, at, dy.double() * scale)
    mag = z.index_add(0, at, (dy.double() * scale).abs())
    n = torch.bincount(at, minlength=V + 2)
    return ref[:V + 1], mag[:V + 1], n[:V + 1]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,V", EMBED)
@pytest.mark.parametrize("mask", [True, False])
def test_embed_gradient(g, T, H, V, dt, mask):
    ids, E, m, dy = _embed_case(T, H, V, dt, seed=T + V)
    scale = 1.0 / 3.0
    dE, dm = g.op_embed_backward(dy, ids, V, scale=scale, mask=mask)
    ref, mag, n = _embed_grad_ref(dy, ids, V, scale, torch.tensor(mask, device="cuda"))
    tol = ref.abs() * U[dt] + mag * ((n[:, None] + 3) * F32)
    _close(dE, ref[:V], tol[:V], "d_embed")
    assert (dm is None) == (not mask)
    if mask:
        _close(dm, ref[V], tol[V], "d_mask")
    again = g.op_embed_backward(dy, ids, V, scale=scale, mask=mask)
    assert torch.equal(dE, again[0])


@pytest.mark.parametrize("ids", ["same", "mask", "bad", "none"])
def test_embed_gradient_of_one_token(g, ids):
    """Every position the same token: one run over every piece; or no position at all."""
    T, H, V = (0 if ids == "none" else 1000), 136, 50
    value = {"same": 49, "mask": -1, "bad": V, "none": 0}[ids]
    i = torch.full((T,), value, dtype=torch.int32, device="cuda")
    dy = torch.randn((T, H), generator=_gen(1), device="cuda")
    dE, dm = g.op_embed_backward(dy, i, V, mask=True)
    ref, mag, n = _embed_grad_ref(dy, i, V, 1.0, torch.tensor(True, device="cuda"))
    tol = mag * ((n[:, None] + 3) * F32)
    _close(dE, ref[:V], tol[:V])
    _close(dm, ref[V], tol[V])
    assert g.op_embed(i, torch.ones((V, H), device="cuda")).shape == (T, H)


# ---------------------------------------------------------------------- cross entropy

def _ce_case(T, V, H, seed, ignored=0.2, lean=8.0):
    r = _gen(seed)
    rnd = lambda *s: torch.randn(s, generator=r, device="cuda")
    u = lambda n: torch.rand(n, generator=r, device="cuda")
    labels = (u(T) * V).long().clamp(0, V - 1)
    w = (H ** -0.5 * rnd(V, H)).bfloat16()
    x = (rnd(T, H) + lean * w.float()[labels] / max(1.0, H ** 0.5 / 16)).bfloat16()
    wrong = torch.tensor([-1, V, -100, 2 ** 31 - 1], device="cuda")
    lab = torch.where(u(T) < ignored, wrong[torch.arange(T, device="cuda") % 4], labels).to(torch.int32)
    return x, w, lab, (u(T) - 0.3)


def _ce_ref(x, w, labels, dloss):
    """(loss, lse, dx, dw) in 64 bits and the bounds of the kernels' errors."""
    xd, wd, V, H = x.double(), w.double(), w.shape[0], x.shape[1]
    z = xd @ wd.T
    dz = ((H / 16 + 16) * 2.0 ** -23) * (xd.abs() @ wd.abs().T)
    lse = torch.logsumexp(z, 1)
    lab = labels.long()
    has = (lab >= 0) & (lab < V)
    at = torch.where(has, lab, 0)
    zl = z.gather(1, at[:, None])[:, 0]
    loss = torch.where(has, lse - zl, 0.0)
    # exp of arguments up to |z| LOG2E rounded in fp32, a sum in fp32 of at most 64 + tiles/32 levels
    soft = dz.amax(1) + (80 + V / 8192 + 8 * z.abs().amax(1)) * F32
    tol_lse = soft + 4 * F32 * lse.abs()
    tol_loss = torch.where(has, tol_lse + dz.gather(1, at[:, None])[:, 0] + F32 * loss.abs(), 0.0)
    f = torch.where(has, dloss.double(), 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    onehot = torch.zeros_like(p).scatter_(1, at[:, None], 1.0)
    gr = (p - onehot) * f
    # exp(z - lse) off by dz and by lse's error, then g rounded to bf16
    dg = p * f.abs() * (dz + tol_lse[:, None] + 16 * F32) + gr.abs() * U[torch.bfloat16] + onehot * f.abs() * F32
    dx, dw = gr @ wd, gr.T @ xd
    T = x.shape[0]
    sum_x = (V / 16 + 64) * 2.0 ** -23 * (gr.abs() @ wd.abs())
    sum_w = (T / 16 + 64) * 2.0 ** -23 * (gr.abs().T @ xd.abs())
    u = U[torch.bfloat16]
    tol_dx = (dg @ wd.abs() + sum_x) * (1 + u) + u * dx.abs() + 1e-38
    tol_dw = (dg.T @ xd.abs() + sum_w) * (1 + u) + u * dw.abs() + 1e-38
    return (loss, lse, dx, dw), (tol_loss, tol_lse, tol_dx, tol_dw)


CE = [(1, 1, 8), (1, 65536, 1536), (33, 1024, 256), (128, 256, 64), (129, 257, 72), (193, 8191, 512), (300, 5000, 264),
      (2047, 4099, 320), (1025, 20000, 1536)]


@pytest.mark.parametrize("T,V,H", CE)
def test_linear_ce_and_gradient(g, T, V, H):
    x, w, labels, dloss = _ce_case(T, V, H, seed=T + V)
    (loss, lse, dx, dw), (t_loss, t_lse, t_dx, t_dw) = _ce_ref(x, w, labels, dloss)
    got_loss, got_lse = g.op_linear_ce(x, w, labels)
    _close(got_lse, lse, t_lse, "lse")
    _close(got_loss, loss, t_loss, "loss")
    has = (labels >= 0) & (labels < V)
    assert not got_loss[~has].any()
    got_dx, got_dw = g.op_linear_ce_backward(dloss, x, w, labels, got_lse)
    _close(got_dx, dx, t_dx, "dx")
    _close(got_dw, dw, t_dw, "dw")
    g.op_status()


@pytest.mark.parametrize("T,V,H", [(33, 19457, 64), (40, 25001, 72), (200, 30001, 136), (600, 7000, 264)])
def test_linear_ce_vocabularies_of_a_round_and_a_bit(g, T, V, H):
    """Vocabularies just past what one round of full tiles covers: narrower tiles, of 160 to 256 columns."""
    test_linear_ce_and_gradient(g, T, V, H)


def test_linear_ce_in_several_pieces(g):
    """More columns than one piece of the vocabulary holds, and a ragged last piece."""
    T, V, H = 5000, 12 * 1024 + 77, 128
    x, w, labels, dloss = _ce_case(T, V, H, seed=3)
    lib = g.load()
    # the workspace holds less than half of the softmax gradient
    assert lib.gocr_op_linear_ce_backward_workspace(T, V, H) < T * V * 2
    (loss, lse, dx, dw), (t_loss, t_lse, t_dx, t_dw) = _ce_ref(x, w, labels, dloss)
    got_loss, got_lse = g.op_linear_ce(x, w, labels)
    _close(got_loss, loss, t_loss, "loss")
    got_dx, got_dw = g.op_linear_ce_backward(dloss, x, w, labels, got_lse)
    _close(got_dx, dx, t_dx, "dx")
    _close(got_dw, dw, t_dw, "dw")
    for a, b in zip((got_dx, got_dw), g.op_linear_ce_backward(dloss, x, w, labels, got_lse)):
        assert torch.equal(a, b)


def test_linear_ce_large_logits(g):
    """Logits of hundreds: the running maximum keeps every exponential finite."""
    x, w, labels, dloss = _ce_case(100, 3001, 128, seed=5)
    x = (x.float() * 100).bfloat16()
    (loss, lse, dx, dw), (t_loss, t_lse, t_dx, t_dw) = _ce_ref(x, w, labels, dloss)
    got_loss, got_lse = g.op_linear_ce(x, w, labels)
    _close(got_loss, loss, t_loss, "loss")
    got_dx, got_dw = g.op_linear_ce_backward(dloss, x, w, labels, got_lse)
    _close(got_dx, dx, t_dx, "dx")
    _close(got_dw, dw, t_dw, "dw")


def test_linear_ce_rows_without_target(g):
    """No row has a target: zero gradients, whatever dloss and lse hold; and no row at all."""
    x, w, _, dloss = _ce_case(70, 500, 64, seed=6)
    labels = torch.full((70,), -1, dtype=torch.int32, device="cuda")
    loss, lse = g.op_linear_ce(x, w, labels)
    assert not loss.any() and torch.isfinite(lse).all()
    dx, dw = g.op_linear_ce_backward(torch.full_like(dloss, math.nan), x, w, labels, torch.full_like(lse, math.nan))
    assert not dx.any() and not dw.any()
    loss, lse = g.op_linear_ce(x[:0], w, labels[:0])
    assert loss.shape == (0,) and lse.shape == (0,)
    dx, dw = g.op_linear_ce_backward(dloss[:0], x[:0], w, labels[:0], lse)
    assert dx.shape == (0, 64) and not dw.any()


def test_linear_ce_nan_stays_in_its_row(g):
    x, w, labels, dloss = _ce_case(140, 700, 64, seed=7, ignored=0.0)
    good = g.op_linear_ce(x, w, labels)
    x2 = x.clone()
    x2[5, 3] = math.nan
    loss, lse = g.op_linear_ce(x2, w, labels)
    keep = torch.arange(140, device="cuda") != 5
    assert torch.isnan(loss[5]) and torch.isnan(lse[5])
    assert torch.equal(loss[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])


def test_linear_ce_gradient_against_differences(g):
    """Sum of dloss * loss along a direction: the central difference over steps that bf16 holds exactly."""
    T, V, H = 64, 1000, 256
    x, w, labels, dloss = _ce_case(T, V, H, seed=8)
    _, lse = g.op_linear_ce(x, w, labels)
    dx, dw = g.op_linear_ce_backward(dloss, x, w, labels, lse)
    f = lambda a, b: float((g.op_linear_ce(a, b, labels)[0].double() * dloss.double()).sum())
    for which, grad in (("x", dx), ("w", dw)):
        t = x if which == "x" else w
        # half a per cent of each value, along the gradient's sign
        step = (t.float().abs() * 2.0 ** -6 * torch.sign(grad.float()))
        hi, lo = (t.float() + step).bfloat16(), (t.float() - step).bfloat16()
        d = f(hi, w) - f(lo, w) if which == "x" else f(x, hi) - f(x, lo)
        want = float((grad.double() * (hi.double() - lo.double())).sum())
        # the gradient is off by at most 2 x 2^-8 of itself here; the third-order term of steps of
        # 2^-6 on logits of a few units is below one per cent
        assert abs(d - want) <= 0.03 * abs(want), (which, d, want)


def test_train_ops_on_another_stream_and_in_a_graph(g):
    """Calls follow the current stream; a captured step replays on new inputs."""
    T, V, H = 200, 3000, 128
    ids, E, m, _ = _embed_case(T, H, V, torch.bfloat16, seed=9, bad=0.0)
    _, w, labels, dloss = _ce_case(T, V, H, seed=9)

    def step():
        x = g.op_embed(ids, E, m, scale=2.0)
        loss, lse = g.op_linear_ce(x, w, labels)
        dx, dw = g.op_linear_ce_backward(dloss, x, w, labels, lse)
        return (loss, dw) + g.op_embed_backward(dx, ids, V, scale=2.0, mask=True)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(2):
        ids2, _, _, _ = _embed_case(T, H, V, torch.bfloat16, seed=20 + k, bad=0.1)
        ids.copy_(ids2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
    g.op_status()


def test_train_ops_workspace_may_hold_anything(g):
    """A workspace is not cleared between calls, and may be the caller's."""
    lib = g.load()
    x, w, labels, dloss = _ce_case(130, 600, 64, seed=11)
    loss, lse = g.op_linear_ce(x, w, labels)
    dx, dw = g.op_linear_ce_backward(dloss, x, w, labels, lse)
    for fill in (0, 255):
        ws = lambda n: torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        l2, s2 = g.op_linear_ce(x, w, labels, workspace=ws(lib.gocr_op_linear_ce_workspace(130, 600)))
        a, b = g.op_linear_ce_backward(dloss, x, w, labels, lse,
                                       workspace=ws(lib.gocr_op_linear_ce_backward_workspace(130, 600, 64)))
        assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(a, dx) and torch.equal(b, dw)
        ids, E, m, dy = _embed_case(100, 64, 30, torch.bfloat16, seed=12)
        want = g.op_embed_backward(dy, ids, 30, mask=True)
        got = g.op_embed_backward(dy, ids, 30, mask=True, workspace=ws(lib.gocr_op_embed_backward_workspace(100, 64)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,first", [(1, 0), (40, 0), (600, 300)])
def test_linear_ce_gradient_of_a_mean(g, T, first):
    """All targets have one weight, which bf16 would round by 2^-8: that error must
    not be in every gradient.  Rows before `first` have no target and a NaN weight."""
    V, H = 5000, 128
    x, w, _, _ = _ce_case(T, V, H, seed=T, ignored=0.0, lean=0.0)
    labels = torch.randint(0, V, (T,), generator=_gen(T), device="cuda", dtype=torch.int32)
    labels[:first] = -1
    _, lse = g.op_linear_ce(x, w, labels)

    def grads(weight):
        dloss = torch.full((T,), weight, device="cuda")
        dloss[:first] = math.nan
        return [t.double() for t in g.op_linear_ce_backward(dloss, x, w, labels, lse)]
    one = grads(1.0)
    for weight in (1.0 + 2.0 ** -8 - 2.0 ** -20, -2.0 ** -9 * (1.0 + 2.0 ** -8 - 2.0 ** -20)):
        for a, b in zip(grads(weight), one):
            # each side rounds its sums once to bf16, by half a step at most
            assert ((a - weight * b).abs() <= (2 * U[torch.bfloat16] + 4 * F32) * (weight * b).abs() + 1e-38).all()
            # these errors are independent, of 2^-7 / sqrt(3) standard deviation at most: their mean over
            # the values that count stays within six deviations
            n = float(b.square().sum() ** 2 / (b ** 4).sum())
            mean = float(((a - weight * b) * b).sum() / (weight * b.square().sum()))
            assert abs(mean) <= 6 * 2.0 ** -7 / 3 ** 0.5 / n ** 0.5, (weight, mean, n)
