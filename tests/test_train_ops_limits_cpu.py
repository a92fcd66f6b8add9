"""Refusals and limits of the training and scoring operators beyond their first
checks, on the host."""
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


def _packed(lib, n=2, T=8, Hq=4, Hkv=2, d=64, ld=None, scale=0.125, ws=None):
    """Both calls, refused at the latest for a pointer (the forward's o) or the workspace."""
    ld = ld or (Hq * d, Hkv * d, Hkv * d)
    sizes = (n, T, Hq, Hkv, d, *ld, scale)
    a = lib.gocr_op_attention_packed(P, P, P, ODD, P, P, *sizes, None), _message(lib)
    b = lib.gocr_op_attention_packed_backward(P, P, P, P, P, P, P, P, P, P, *sizes, P, 0, None), _message(lib)
    return a, b


def _passes(answers):
    (a, am), (b, bm) = answers
    return a == EINVAL and "aligned" in am and b == ECAPACITY and "workspace" in bm


def _refused(answers, word):
    return all(rc == EINVAL and word in m for rc, m in answers)


def test_attention_packed_limits(lib):
    """Each limit that the header states: its last value passes, the next one is refused."""
    assert _passes(_packed(lib))
    assert _passes(_packed(lib, n=1 << 20)) and _refused(_packed(lib, n=(1 << 20) + 1), "shape")
    assert _passes(_packed(lib, T=1 << 24)) and _refused(_packed(lib, T=(1 << 24) + 1), "shape")
    assert _passes(_packed(lib, Hq=1024, Hkv=1)) and _refused(_packed(lib, Hq=1025, Hkv=1), "shape")
    # (n_seq + T) (Hq + Hkv) <= 2^31 - 1: 2^31 - 1 is prime, so the nearest products around it
    T, heads = 1 << 24, 128
    n = (2 ** 31 - 1) // heads - T
    assert n < 0  # 2^24 rows of 127 + 1 heads are already above
    assert _refused(_packed(lib, n=1, T=T, Hq=127, Hkv=1), "2^31")
    T = (2 ** 31 - 1) // heads - 1
    assert _passes(_packed(lib, n=1, T=T, Hq=127, Hkv=1)) and _refused(_packed(lib, n=2, T=T, Hq=127, Hkv=1), "2^31")
    most = 1 << 32
    for i in range(3):
        ld = [256, 128, 128]
        ld[i] = most
        assert _passes(_packed(lib, ld=ld))
        ld[i] = most + 8
        assert _refused(_packed(lib, ld=ld), "pitch")
    assert _passes(_packed(lib, scale=1e30)) and _refused(_packed(lib, scale=1.1e30), "scale")


def test_embed_and_linear_ce_limits(lib):
    def embed(T=4, H=64, V=100):
        return lib.gocr_op_embed(1, ODD, P, P, P, T, H, V, 1.0, None), _message(lib)
    for k, last, step in (("T", 1 << 28, 1), ("H", 1 << 20, 8), ("V", 1 << 28, 1)):
        assert "aligned" in embed(**{k: last})[1], k
        assert "shape" in embed(**{k: last + step})[1], k

    def ce(T=4, V=100, H=64):
        return lib.gocr_op_linear_ce(ODD, P, P, P, P, T, V, H, P, 0, None), _message(lib)
    for k, last, step in (("T", 1 << 22, 1), ("H", 1 << 15, 8), ("V", 1 << 22, 1)):
        assert "aligned" in ce(**{k: last})[1], k
        assert "shape" in ce(**{k: last + step})[1], k


def test_wrappers_refuse_sizes_past_32_bits():
    """The library takes 32-bit sizes; a longer one must not arrive as its remainder."""
    torch = pytest.importorskip("torch")
    from self_speculative_block_gb300 import gocr
    bf16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="meta")
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="meta")
    f32 = lambda *s: torch.empty(s, dtype=torch.float32, device="meta")
    many = 2 ** 32 + 8
    for call in (lambda: gocr.op_embed(i32(4), bf16(many, 8)),
                 lambda: gocr.op_embed(i32(many), bf16(4, 8)),
                 lambda: gocr.op_embed_backward(bf16(many, 8), i32(many), 10),
                 lambda: gocr.op_embed_backward(bf16(4, 8), i32(4), many),
                 lambda: gocr.op_embed_backward(bf16(4, 8), i32(4), -1),
                 lambda: gocr.op_attention_packed(bf16(many, 1, 64), bf16(many, 1, 64), bf16(many, 1, 64), i32(2)),
                 lambda: gocr.op_attention_packed(bf16(4, 1, 64), bf16(4, 1, 64), bf16(4, 1, 64), i32(many)),
                 lambda: gocr.op_attention_packed_backward(bf16(many, 1, 64), bf16(many, 1, 64), bf16(many, 1, 64),
                                                           bf16(many, 1, 64), bf16(many, 1, 64), f32(1, many), i32(2)),
                 lambda: gocr.op_linear_ce(bf16(many, 8), bf16(4, 8), i32(many)),
                 lambda: gocr.op_linear_ce(bf16(4, 8), bf16(many, 8), i32(4)),
                 lambda: gocr.op_linear_ce_backward(f32(4), bf16(4, 8), bf16(many, 8), i32(4), f32(4))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_wrappers_refuse_operands_that_want_a_gradient():
    """The calls return tensors without a graph: a gradient must not be lost silently."""
    torch = pytest.importorskip("torch")
    from self_speculative_block_gb300 import gocr
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    b = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, lse, cu = torch.zeros(4, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 4), torch.zeros(2, dtype=torch.int32)
    calls = [(gocr.op_embed, (i, b), {}, (1,)),
             (gocr.op_embed, (i, b, b[0].clone()), {}, (1, 2)),
             (gocr.op_embed_backward, (b, i, 10), {}, (0,)),
             (gocr.op_attention_packed, (q, q, q, cu), {}, (0, 1, 2)),
             (gocr.op_attention_packed_backward, (q, q, q, q, q, lse, cu), {}, (0, 1, 2, 3, 4, 5)),
             (gocr.op_linear_ce, (b, b, i), {}, (0, 1)),
             (gocr.op_linear_ce_backward, (f, b, b, i, f), {}, (0, 1, 2, 4))]
    for fn, args, kw, which in calls:
        for k in which:
            bad = [a.clone().requires_grad_() if j == k else a for j, a in enumerate(args)]
            with pytest.raises(ValueError, match="outside autograd"):
                fn(*bad, **kw)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # the next check
                fn(*bad, **kw)


@pytest.mark.parametrize("at", [257, 258, 259])
def test_arrays_of_words_are_aligned(lib, at):
    """A word that straddles its boundary would fault on the device."""
    W = ctypes.c_void_p(at)
    sizes = (2, 8, 4, 2, 64, 256, 128, 128, 0.125)
    for rc in (lib.gocr_op_embed(1, P, P, W, P, 4, 64, 100, 1.0, None),
               lib.gocr_op_embed_backward(1, P, W, P, P, 4, 64, 100, 1.0, P, BIG, None),
               lib.gocr_op_attention_packed(P, P, P, P, W, P, *sizes, None),
               lib.gocr_op_attention_packed(P, P, P, P, P, W, *sizes, None),
               lib.gocr_op_attention_packed_backward(P, P, P, P, P, W, P, P, P, P, *sizes, P, BIG, None),
               lib.gocr_op_attention_packed_backward(P, P, P, P, P, P, W, P, P, P, *sizes, P, BIG, None),
               *(lib.gocr_op_linear_ce(P, P, *(W if i == k else P for i in range(3)), 4, 100, 64, P, BIG, None) for k in range(3)),
               *(lib.gocr_op_linear_ce_backward_with_loss(*(W if i == k else P for i in range(8)), 4, 100, 64, P, BIG, None)
                 for k in (0, 3, 4, 5))):
        assert rc == EINVAL and "4-byte" in _message(lib)
