"""The training operators together, as one training step of a small decoder
uses them: embedding with [M] rows, one attention block over packed sequences
(its projections are plain matrix products here), and the LM-head cross
entropy; then the backward calls in reverse order.  The gradients are compared
with automatic differentiation of the same step in 64 bits.
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


def _reference(ids, labels, dloss, lens, E, m, W, O, H, heads, scale):
    """Gradients of sum(dloss * loss) in 64 bits."""
    Hq, Hkv, d = heads
    leaf = [t.double().requires_grad_() for t in (E, m, W, O, H)]
    E, m, W, O, H = leaf
    i = ids.long()
    x = torch.where((i == -1)[:, None], m[None], E[i.clamp(min=0)]) * scale
    qkv = (x @ W.T).view(len(i), Hq + 2 * Hkv, d)
    outs, t0 = [], 0
    for n in lens:
        q, k, v = (t.transpose(0, 1) for t in (qkv[t0:t0 + n, :Hq], qkv[t0:t0 + n, Hq:Hq + Hkv], qkv[t0:t0 + n, Hq + Hkv:]))
        k, v = (t.repeat_interleave(Hq // Hkv, 0) for t in (k, v))
        s = (q @ k.transpose(1, 2) * d ** -0.5).masked_fill(
            torch.triu(torch.ones((n, n), dtype=torch.bool, device=q.device), 1), -math.inf)
        outs.append((torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, Hq * d))
        t0 += n
    y = x + torch.cat(outs) @ O.T
    lp = torch.log_softmax(y @ H.T, 1)
    has = labels >= 0
    loss = -(lp.gather(1, labels.long().clamp(min=0)[:, None])[:, 0] * has)
    (loss * dloss.double()).sum().backward()
    return loss.detach(), [t.grad for t in leaf]


def _step(g, ids, labels, dloss, cu, E, m, W, O, H, heads, scale):
    Hq, Hkv, d = heads
    T = len(ids)
    x = g.op_embed(ids, E, m, scale=scale)
    qkv = (x @ W.T).view(T, Hq + 2 * Hkv, d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    o, lse = g.op_attention_packed(q, k, v, cu)
    y = x + o.view(T, Hq * d) @ O.T
    loss, z = g.op_linear_ce(y, H, labels)
    dy, dH = g.op_linear_ce_backward(dloss, y, H, labels, z)
    do = dy @ O
    dO = dy.T @ o.view(T, Hq * d)
    dq, dk, dv = g.op_attention_packed_backward(do.view(T, Hq, d), q, k, v, o, lse, cu)
    dqkv = torch.cat([dq, dk, dv], 1).view(T, -1)
    dW = dqkv.T @ x
    dx = dy + dqkv @ W
    dE, dm = g.op_embed_backward(dx, ids, E.shape[0], scale=scale, mask=True)
    return loss, [dE, dm, dW, dO, dH]


@pytest.mark.parametrize("heads", [(4, 2, 64), (6, 2, 128)])
def test_training_step_gradients(g, heads):
    Hq, Hkv, d = heads
    V, H = 1024, 256
    lens = [64, 1, 130, 33]
    T = sum(lens)
    r = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=r, device="cuda")
    E, m = rnd(V, H).bfloat16(), rnd(H).bfloat16()
    W, O = (H ** -0.5 * rnd((Hq + 2 * Hkv) * d, H)).bfloat16(), ((Hq * d) ** -0.5 * rnd(H, Hq * d)).bfloat16()
    head = (H ** -0.5 * rnd(V, H)).bfloat16()
    ids = torch.randint(0, V, (T,), generator=r, device="cuda")
    ids = torch.where(torch.rand(T, generator=r, device="cuda") < 0.3, torch.full_like(ids, -1), ids).to(torch.int32)
    labels = torch.randint(-V // 8, V, (T,), generator=r, device="cuda").clamp(min=-1).to(torch.int32)
    dloss = torch.rand(T, generator=r, device="cuda") / T
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    args = (E, m, W, O, head, heads, 1.5)
    loss, grads = _step(g, ids, labels, dloss, cu, *args)
    want, ref = _reference(ids, labels, dloss, lens, *args)
    # between a leaf and the loss a value is rounded to bf16 about ten times (x, qkv, P, o, the
    # projection, y; dy, do, dS, dqkv, dx, each half a step of 2^-8 at most), independently: the
    # norm of the error stays below ten half steps of the norm
    bound = 10 * 2.0 ** -8
    assert float((loss.double() - want).norm() / want.norm()) < bound
    for name, got, w in zip(("dE", "dm", "dW", "dO", "dH"), grads, ref):
        rel = float((got.double() - w).norm() / w.norm())
        assert rel < bound, (name, rel)
    again = _step(g, ids, labels, dloss, cu, *args)
    assert all(torch.equal(a, b) for a, b in zip(again[1][:1] + again[1][4:], grads[:1] + grads[4:]))
    g.op_status()
