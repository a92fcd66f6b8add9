"""Rows of the cross entropy's gradient that a tolerance over the whole softmax
does not see: confident ones, whose gradient is as small as their loss."""
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
