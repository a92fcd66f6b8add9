"""Rows of the cross entropy's gradient that a tolerance over the whole softmax
does not see: confident ones, whose gradient is as small as their loss, and the
streams of a joint loss, whose rows share a weight."""
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / tol.clamp(min=1e-300)).nan_to_num(float('inf')).max()):.3g} times the bound")


def _confident(T, V, H, seed):
    """Hidden rows along their targets' weights: losses from about 0.01 down to 1e-8."""
    r = _gen(seed)
    w = (H ** -0.5 * torch.randn((V, H), generator=r, device="cuda")).bfloat16()
    labels = torch.randperm(V, generator=r, device="cuda")[:T].to(torch.int32)
    x = (torch.linspace(12.0, 32.0, T, device="cuda")[:, None] * w.float()[labels.long()]).bfloat16()
    return x, w, labels


def _exact(x, w, labels, dloss):
    """1 - p of the label, the gradient g of the logits, and |x| |w| sums, in 64 bits without cancellation."""
    z = x.double() @ w.double().T
    at = labels.long()[:, None]
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    rest = p.scatter(1, at, 0.0).sum(1)
    gr = p.scatter(1, at, -rest[:, None]) * dloss.double()[:, None]
    return z, rest, gr


@pytest.mark.parametrize("T,V,H", [(500, 1000, 64), (100, 8191, 256), (700, 5000, 136)])
def test_linear_ce_gradient_of_confident_rows(g, T, V, H):
    x, w, labels = _confident(T, V, H, seed=T)
    dloss = torch.rand(T, generator=_gen(T + 1), device="cuda") + 0.5
    z, rest, gr = _exact(x, w, labels, dloss)
    assert rest.min() < 1e-5 and (rest < 1e-3).double().mean() > 0.5
    loss, lse = g.op_linear_ce(x, w, labels)
    dx, dw = g.op_linear_ce_backward(dloss, x, w, labels, lse, loss=loss)
    # a logit is off by one truncation of 2^-23 per 16-deep step of its sum; an exponential's
    # argument by its two logits (the label's and its own, or lse's) and by the rounding of each of
    # three terms as large as the largest logit; then g is rounded once
    dz = ((H / 16 + 16) * TC * (x.double().abs() @ w.double().abs().T)).amax(1)
    big = z.abs().amax(1)
    rel = 2 * dz + (32 + V / 8192 + 8 * big) * F32
    dg = gr.abs() * (U + rel)[:, None]
    for name, got, ref, err, deep in (("dx", dx, gr @ w.double(), dg @ w.double().abs(), (V / 16 + 64) * TC),
                                      ("dw", dw, gr.T @ x.double(), dg.T @ x.double().abs(), (T / 16 + 64) * TC)):
        mag = gr.abs() @ w.double().abs() if name == "dx" else gr.abs().T @ x.double().abs()
        _close(got, ref, (err + deep * mag) * (1 + U) + U * ref.abs() + 1e-38, name)
    g.op_status()


def test_linear_ce_gradient_of_confident_rows_without_their_loss(g):
    """The label's share is never taken for more than one: its own gradient does not change its sign."""
    x, w, labels = _confident(500, 1000, 64, seed=3)
    one = torch.ones(500, device="cuda")
    _, lse = g.op_linear_ce(x, w, labels)
    dx, _ = g.op_linear_ce_backward(one, x, w, labels, lse)
    with_loss, _ = g.op_linear_ce_backward(one, x, w, labels, lse, loss=torch.zeros_like(lse))
    # loss 0 leaves out the label's term; what is left of dx is that term, along -w of the label
    part = ((dx.double() - with_loss.double()) * w.double()[labels.long()]).sum(1)
    size = (with_loss.double().abs() * w.double()[labels.long()].abs()).sum(1)
    # both sides round dx to bf16 once
    assert (part <= 2 * U * (size + part.abs())).all()


def test_linear_ce_gradient_with_and_without_loss_agree_on_unsure_rows(g):
    T, V, H = 193, 3000, 128
    r = _gen(5)
    x, w = torch.randn((T, H), generator=r, device="cuda").bfloat16(), torch.randn((V, H), generator=r, device="cuda").bfloat16()
    labels = torch.randint(-1, V, (T,), generator=r, device="cuda", dtype=torch.int32)
    dloss = torch.rand(T, generator=r, device="cuda")
    loss, lse = g.op_linear_ce(x, w, labels)
    a = g.op_linear_ce_backward(dloss, x, w, labels, lse)
    b = g.op_linear_ce_backward(dloss, x, w, labels, lse, loss=torch.where(labels < 0, float("nan"), loss))
    # the label's terms may round differently, by one step of bf16; so may the results
    for p, q, mag in ((a[0], b[0], w[labels.clamp(min=0).long()].double().abs() * dloss[:, None]),):
        assert ((p.double() - q.double()).abs() <= 2 * U * mag + 2 * U * q.double().abs() + 1e-38).all()
    assert not b[0][labels < 0].any() and torch.isfinite(b[1]).all()


def _off_8_bits(y):
    """Relative distance of y to the nearest number of 8 significant bits."""
    m, e = math.frexp(y)
    return abs(round(m * 256) / 256 / m - 1)


@pytest.mark.parametrize("n1,n2", [(2600, 1100), (3001, 777), (2048, 1999), (1, 1500)])
def test_linear_ce_gradient_of_two_means(g, n1, n2):
    """Two streams, each with a mean's weight: bf16 would round each weight by up to 2^-8, for
    all of its stream's rows alike.  Targets of the two streams are of the two halves of the vocabulary."""
    V, H, T = 5000, 128, n1 + n2
    r = _gen(n1)
    w = (H ** -0.5 * torch.randn((V, H), generator=r, device="cuda")).bfloat16()
    x = torch.randn((T, H), generator=r, device="cuda").bfloat16()
    second = torch.arange(T, device="cuda") >= n1
    labels = torch.where(second, torch.randint(V // 2, V, (T,), generator=r, device="cuda"),
                         torch.randint(0, V // 2, (T,), generator=r, device="cuda")).to(torch.int32)
    _, lse = g.op_linear_ce(x, w, labels)
    grads = lambda dloss: [t.double() for t in g.op_linear_ce_backward(dloss.float(), x, w, labels, lse)]
    weight = [float(torch.tensor(0.5 / n)) for n in (n1, n2)]
    lo, hi = sorted(math.frexp(a)[0] for a in weight)
    # the best that two weights can be in units of a common one, and less than it would be without
    best = min(_off_8_bits(a * hi / lo) for a in range(128, 256))
    assert best < 2.0 ** -11
    apart = [grads(~second), grads(second)]
    both = grads(torch.where(second, weight[1], weight[0]))
    for name, i, parts in (("dx", 0, (slice(0, n1), slice(n1, T))), ("dw", 1, (slice(0, V // 2), slice(V // 2, V)))):
        want = weight[0] * apart[0][i] + weight[1] * apart[1][i]
        for s in parts:
            a, b = both[i][s], want[s]
            # independent roundings, of 2^-7 / sqrt(3) standard deviation at most, over the values that
            # count; and the label's 1 - p, which rounds to one on both sides but for the few rows with
            # a p between 2^-9 and 2^-7, less than one in a hundred
            n = float(b.square().sum() ** 2 / (b ** 4).sum())
            mean = float(((a - b) * b).sum() / b.square().sum())
            assert abs(mean) <= best + 2.0 ** -14 + 6 * 2.0 ** -7 / 3 ** 0.5 / n ** 0.5, (name, s, mean, best, n)


def test_linear_ce_gradient_of_one_target_behind_many_rows(g):
    """Only the last of many rows has a target; the others' weights and lse hold NaN."""
    T, V, H = 5000, 700, 64
    r = _gen(9)
    w, x = torch.randn((V, H), generator=r, device="cuda").bfloat16(), torch.randn((T, H), generator=r, device="cuda").bfloat16()
    labels = torch.full((T,), V, dtype=torch.int32, device="cuda")
    labels[-1] = 5
    dloss = torch.full((T,), math.nan, device="cuda")
    dloss[-1] = 1.0 + 2.0 ** -8 - 2.0 ** -20
    _, lse = g.op_linear_ce(x, w, labels)
    lse[:-1] = math.nan
    dx, dw = g.op_linear_ce_backward(dloss, x, w, labels, lse)
    assert not dx[:-1].any()
    one = g.op_linear_ce_backward(dloss[-1:], x[-1:].contiguous(), w, labels[-1:], lse[-1:])
    # the sums of the two calls are cut into parts differently, in fp32, before the last rounding
    for a, b in ((dx[-1:], one[0]), (dw, one[1])):
        assert ((a.double() - b.double()).abs() <= (2 * U + 2.0 ** -12) * b.double().abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("T,V,H", [(1, 300, 64), (70, 500, 72), (300, 9000, 1000), (5000, 12 * 1024 + 77, 128)])
def test_linear_ce_rows_without_target_may_hold_anything(g, T, V, H):
    """Padding rows, which nothing has written: their x reaches neither dx nor dw, nor do their loss, lse and weight."""
    r = _gen(T + V)
    w, x = (torch.randn(s, generator=r, device="cuda").bfloat16() for s in ((V, H), (T, H)))
    labels = torch.randint(0, V, (T,), generator=r, device="cuda", dtype=torch.int32)
    no = torch.rand(T, generator=r, device="cuda") < 0.4
    no[T // 2] = True
    labels[no] = torch.tensor([-1, V, -100, 2 ** 31 - 1], device="cuda", dtype=torch.int32)[torch.arange(int(no.sum()), device="cuda") % 4]
    dloss = torch.rand(T, generator=r, device="cuda")
    x[no] = 0.0
    loss, lse = g.op_linear_ce(x, w, labels)
    want = g.op_linear_ce_backward(dloss, x, w, labels, lse, loss=loss)
    for junk in (math.nan, math.inf):
        for t in (x, dloss, loss, lse):
            t[no] = junk
        dx, dw = g.op_linear_ce_backward(dloss, x, w, labels, lse, loss=loss)
        assert not dx[no].any()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    loss, lse = g.op_linear_ce(x, w, labels)
    assert not loss[no].any() and torch.isfinite(lse[~no]).all()
