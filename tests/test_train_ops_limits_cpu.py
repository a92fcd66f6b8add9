"""Refusals and limits of the training and scoring operators beyond their first
checks, on the host."""
import ctypes

import pytest

EINVAL, ECAPACITY = -1, -2
P = ctypes.c_void_p(256)      # never dereferenced: each call below is refused first
ODD = ctypes.c_void_p(258)


@pytest.fixture(scope="module")
def lib():
    from self_speculative_block_gb300 import build, gocr
    build.build()
    return gocr.load()


def _message(lib):
    return lib.gocr_last_error(None).decode()


def test_linear_ce_backward_with_loss_refusals(lib):
    need = lib.gocr_op_linear_ce_backward_workspace(4, 100, 64)

    def call(dl=P, x=P, w=P, lab=P, loss=P, lse=P, dx=P, dw=P, T=4, V=100, H=64, ws=P, n=need):
        return lib.gocr_op_linear_ce_backward_with_loss(dl, x, w, lab, loss, lse, dx, dw, T, V, H, ws, n, None)
    for k in ("dl", "x", "w", "lab", "lse", "dx", "dw", "ws"):
        assert call(**{k: None}) == EINVAL and "null" in _message(lib)
    for bad in (dict(T=-1), dict(V=0), dict(H=12)):
        assert call(**bad) == EINVAL and "shape" in _message(lib)
    for k in ("x", "w", "dx", "dw", "ws"):
        assert call(**{k: ODD}) == EINVAL and "aligned" in _message(lib)
    assert call(n=need - 1) == ECAPACITY
    assert call(loss=None, n=need - 1) == ECAPACITY  # no loss is no error


def test_linear_ce_backward_checks_loss():
    torch = pytest.importorskip("torch")
    from self_speculative_block_gb300 import gocr
    b, i, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="loss must be"):
        gocr.op_linear_ce_backward(f, b, b, i, f, loss=f.double())
    with pytest.raises(ValueError, match="loss must be"):
        gocr.op_linear_ce_backward(f, b, b, i, f, loss=f[:3])


def test_wait_probe_refuses_long_waits(lib):
    for us in (0, -1, 1_000_001):
        assert lib.gocr_op_wait_probe(us, None) == EINVAL and "microseconds" in _message(lib)
