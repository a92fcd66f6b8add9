"""Argument checks of the training and scoring operators: every refusal happens
on the host, before any device work, so it can be tested without a GPU."""
import ctypes

import pytest

EINVAL, ECAPACITY = -1, -2
P = ctypes.c_void_p(256)      # never dereferenced: each call below is refused first
ODD = ctypes.c_void_p(258)
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    from self_speculative_block_gb300 import build, gocr
    build.build()
    return gocr.load()


def _message(lib):
    return lib.gocr_last_error(None).decode()


def test_embed_refusals(lib):
    call = lambda dt=1, e=P, m=P, i=P, y=P, T=4, H=64, V=100: lib.gocr_op_embed(dt, e, m, i, y, T, H, V, 1.0, None)
    assert call(dt=2) == EINVAL and "dtype" in _message(lib)
    for bad in (dict(e=None), dict(i=None), dict(y=None)):
        assert call(**bad) == EINVAL and "null" in _message(lib)
    for bad in (dict(T=-1), dict(H=0), dict(H=12), dict(V=0)):
        assert call(**bad) == EINVAL and "shape" in _message(lib)
    for bad in (dict(e=ODD), dict(m=ODD), dict(y=ODD)):
        assert call(**bad) == EINVAL and "aligned" in _message(lib)


def test_embed_backward_refusals(lib):
    need = lib.gocr_op_embed_backward_workspace(4, 64)
    assert need > 0 and lib.gocr_op_embed_backward_workspace(-1, 64) == 0

    def call(dt=1, dy=P, i=P, de=P, dm=P, T=4, H=64, V=100, ws=P, n=need):
        return lib.gocr_op_embed_backward(dt, dy, i, de, dm, T, H, V, 1.0, ws, n, None)
    assert call(dt=-1) == EINVAL
    for bad in (dict(dy=None), dict(i=None), dict(de=None), dict(ws=None)):
        assert call(**bad) == EINVAL and "null" in _message(lib)
    for bad in (dict(T=-1), dict(H=4), dict(H=20), dict(V=0)):
        assert call(**bad) == EINVAL and "shape" in _message(lib)
    for bad in (dict(dy=ODD), dict(de=ODD), dict(dm=ODD), dict(ws=ODD)):
        assert call(**bad) == EINVAL and "aligned" in _message(lib)
    assert call(n=need - 1) == ECAPACITY and "workspace" in _message(lib)


def test_linear_ce_refusals(lib):
    need = lib.gocr_op_linear_ce_workspace(4, 100)
    assert need > 0 and lib.gocr_op_linear_ce_workspace(4, 0) == 0

    def call(x=P, w=P, lab=P, loss=P, lse=P, T=4, V=100, H=64, ws=P, n=need):
        return lib.gocr_op_linear_ce(x, w, lab, loss, lse, T, V, H, ws, n, None)
    for bad in (dict(x=None), dict(w=None), dict(lab=None), dict(loss=None), dict(lse=None), dict(ws=None)):
        assert call(**bad) == EINVAL and "null" in _message(lib)
    for bad in (dict(T=-1), dict(V=0), dict(H=0), dict(H=9)):
        assert call(**bad) == EINVAL and "shape" in _message(lib)
    for bad in (dict(x=ODD), dict(w=ODD), dict(ws=ODD)):
        assert call(**bad) == EINVAL and "aligned" in _message(lib)
    assert call(n=need - 1) == ECAPACITY


def test_linear_ce_backward_refusals(lib):
    need = lib.gocr_op_linear_ce_backward_workspace(4, 100, 64)
    assert need > 0 and lib.gocr_op_linear_ce_backward_workspace(4, 100, 0) == 0

    def call(dl=P, x=P, w=P, lab=P, lse=P, dx=P, dw=P, T=4, V=100, H=64, ws=P, n=need):
        return lib.gocr_op_linear_ce_backward(dl, x, w, lab, lse, dx, dw, T, V, H, ws, n, None)
    for k in ("dl", "x", "w", "lab", "lse", "dx", "dw", "ws"):
        assert call(**{k: None}) == EINVAL and "null" in _message(lib)
    for bad in (dict(T=-1), dict(V=0), dict(H=4), dict(H=17)):
        assert call(**bad) == EINVAL and "shape" in _message(lib)
    for k in ("x", "w", "dx", "dw", "ws"):
        assert call(**{k: ODD}) == EINVAL and "aligned" in _message(lib)
    assert call(n=need - 1) == ECAPACITY


def test_workspaces_stay_bounded(lib):
    """The backward call keeps a piece of the softmax gradient, never all of it."""
    T, V, H = 8192, 65536, 1536
    assert lib.gocr_op_linear_ce_backward_workspace(T, V, H) < T * V // 2
    assert lib.gocr_op_linear_ce_workspace(T, V) < T * V // 16


def test_wrappers_check_tensors():
    torch = pytest.importorskip("torch")
    from self_speculative_block_gb300 import gocr
    f, b, i = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gocr.op_embed(i, f)
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        gocr.op_linear_ce(f, f, i)
    with pytest.raises(ValueError, match="contiguous"):
        gocr.op_linear_ce(torch.zeros(64, 4, dtype=torch.bfloat16).T, b, i)
    with pytest.raises(ValueError, match="dy must be"):
        gocr.op_embed_backward(torch.zeros(4, 64, dtype=torch.float16), i, 10)


def test_attention_packed_refusals(lib):
    def call(q=P, k=P, v=P, o=P, lse=P, cu=P, n=2, T=8, Hq=4, Hkv=2, d=64, ldq=256, ldk=128, ldv=128, scale=0.125):
        return lib.gocr_op_attention_packed(q, k, v, o, lse, cu, n, T, Hq, Hkv, d, ldq, ldk, ldv, scale, None)
    for k in ("q", "k", "v", "o", "lse", "cu"):
        assert call(**{k: None}) == EINVAL and "null" in _message(lib)
    for bad in (dict(n=-1), dict(T=-1), dict(Hq=3), dict(Hkv=0), dict(d=96), dict(Hq=2048, Hkv=1, ldq=1 << 18)):
        assert call(**bad) == EINVAL and "shape" in _message(lib)
    for bad in (dict(ldq=255), dict(ldq=248), dict(ldk=64), dict(ldv=132), dict(ldk=1 << 40)):
        assert call(**bad) == EINVAL and "pitch" in _message(lib)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == EINVAL and "scale" in _message(lib)
    for k in ("q", "k", "v", "o"):
        assert call(**{k: ODD}) == EINVAL and "aligned" in _message(lib)


def test_attention_packed_backward_refusals(lib):
    need = lib.gocr_op_attention_packed_backward_workspace(8, 4)
    assert need > 0 and lib.gocr_op_attention_packed_backward_workspace(8, 0) == 0
    names = ("d_o", "q", "k", "v", "o", "lse", "cu", "dq", "dk", "dv")

    def call(n=2, T=8, Hq=4, Hkv=2, d=64, ld=(256, 128, 128), scale=0.125, ws=P, nb=need, **ptr):
        return lib.gocr_op_attention_packed_backward(*[ptr.get(k, P) for k in names], n, T, Hq, Hkv, d, *ld, scale, ws,
                                                     nb, None)
    for k in names:
        assert call(**{k: None}) == EINVAL and "null" in _message(lib)
    assert call(ws=None) == EINVAL
    for k in names:
        if k not in ("lse", "cu"):
            assert call(**{k: ODD}) == EINVAL and "aligned" in _message(lib)
    assert call(d=32) == EINVAL and call(ld=(256, 128, 100)) == EINVAL and call(scale=-0.5) == EINVAL
    assert call(nb=need - 1) == ECAPACITY and "workspace" in _message(lib)


def test_attention_packed_wrapper_checks_rows():
    torch = pytest.importorskip("torch")
    from self_speculative_block_gb300 import gocr
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="contiguous"):
        gocr.op_attention_packed(torch.zeros(8, 64, 4, dtype=torch.bfloat16).transpose(1, 2), q, q, cu)
    with pytest.raises(ValueError, match="q must be"):
        gocr.op_attention_packed(q[0], q, q, cu)
    with pytest.raises(ValueError, match="bfloat16"):
        gocr.op_attention_packed(q.float(), q, q, cu)
    with pytest.raises(ValueError, match="CUDA"):
        gocr.op_attention_packed(q, q, q, cu)


def test_workspaces_serve_fewer_rows(lib):
    """A workspace for the most rows of a program serves its shorter calls."""
    rows = [1, 2, 33, 128, 129, 256, 257, 300, 4096, 32768, 32769, 40000, 262144, 262145, 1 << 20]
    for H in (8, 256, 1536):
        sizes = [lib.gocr_op_embed_backward_workspace(T, H) for T in rows]
        assert sizes == sorted(sizes)
    for V in (1, 8191, 30000, 65536):
        sizes = [lib.gocr_op_linear_ce_workspace(T, V) for T in rows]
        assert sizes == sorted(sizes)
    for Hq in (1, 12):
        sizes = [lib.gocr_op_attention_packed_backward_workspace(T, Hq) for T in rows]
        assert sizes == sorted(sizes)
