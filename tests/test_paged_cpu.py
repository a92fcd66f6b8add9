"""Argument checks of the paged KV cache operators: every refusal happens on the
host, before any device work, so it can be tested without a GPU."""
import ctypes

import pytest

EINVAL, ECAPACITY = -1, -2
P = ctypes.c_void_p(256)      # never dereferenced: each call below is refused first
ODD = ctypes.c_void_p(258)
BIG = 1 << 60


@pytest.fixture(scope="module")
def g():
    from self_speculative_block_gb300 import build, gocr
    build.build()
    gocr.load()
    return gocr


def _message(g):
    return g.load().gocr_last_error(None).decode()


def _cache(g, **kw):
    f = dict(k=256, v=256, k_page=4096, k_head=1024, k_token=64, v_page=4096, v_head=1024, v_token=64, n_pages=8,
             page_size=16, n_kv_heads=4, head_dim=64)
    f.update(kw)
    return g.PagedKV(**f)


def test_page_step_refusals(g):
    names = ("held", "start", "end", "table", "free", "n_free", "n_free_out", "held_out", "kv_len", "cu", "pos", "slots")

    def call(R=4, width=8, ps=16, n_pages=32, T=7, **ptr):
        p = lambda k: ptr.get(k, P)
        return g.load().gocr_op_page_step(p("held"), p("start"), p("end"), R, p("table"), width, ps, p("free"), n_pages,
                                          p("n_free"), p("n_free_out"), p("held_out"), p("kv_len"), p("cu"), p("pos"),
                                          p("slots"), T, None)
    for k in names:
        assert call(**{k: None}) == EINVAL and "null" in _message(g), k
        assert call(**{k: ODD}) == EINVAL and "aligned" in _message(g), k
    for ps in (0, 8, 17, 48, 512, -16):
        assert call(ps=ps) == EINVAL and "page size" in _message(g)
    for bad in (dict(R=-1), dict(R=4097), dict(width=0), dict(width=(1 << 20) + 1), dict(n_pages=0),
                dict(n_pages=1 << 27), dict(T=-1), dict(T=(1 << 24) + 1)):
        assert call(**bad) == EINVAL and "shape" in _message(g), bad


BAD_STRIDES = [dict(k_token=60), dict(k_token=63), dict(k_token=32), dict(k_head=1016), dict(v_head=64), dict(v_page=4088),
               dict(k_page=0), dict(v_token=-64), dict(k_page=1 << 33), dict(k_page=64, k_token=64),
               dict(k_head=4096 * 7 + 8)]


def test_kv_write_refusals(g):
    names = ("q", "k", "v", "pos", "slots", "q_out")

    def call(T=7, Hq=8, ld=(512, 256, 256), theta=1e4, kv=None, **ptr):
        kv = ctypes.byref(_cache(g, **(kv or {})))
        return g.load().gocr_op_kv_write_paged(*[ptr.get(k, P) for k in names], kv, T, Hq, *ld, theta, None)
    for k in names:
        assert call(**{k: None}) == EINVAL and "null" in _message(g), k
        assert call(**{k: ODD}) == EINVAL and "aligned" in _message(g), k
    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(Hq=0), dict(Hq=6), dict(Hq=1028)):
        assert call(**bad) == EINVAL and "shape" in _message(g), bad
    for bad in ((504, 256, 256), (516, 256, 256), (512, 255, 256), (512, 256, 1 << 33)):
        assert call(ld=bad) == EINVAL and "pitch" in _message(g), bad
    for bad in (0.0, 0.5, float("nan"), float("inf"), -1e4):
        assert call(theta=bad) == EINVAL and "theta" in _message(g)
    for bad in BAD_STRIDES:
        assert call(kv=bad) == EINVAL and "strides" in _message(g), bad
    for bad in (dict(head_dim=96), dict(n_kv_heads=0), dict(n_pages=0), dict(n_pages=1 << 27)):
        assert call(kv=bad) == EINVAL and "shape" in _message(g), bad
    for bad in (dict(k=None), dict(v=None)):
        assert call(kv=bad) == EINVAL and "null" in _message(g), bad
    for bad in (dict(k=264), dict(v=258)):
        assert call(kv=bad) == EINVAL and "aligned" in _message(g), bad
    assert call(kv=dict(page_size=24)) == EINVAL and "page size" in _message(g)
    assert g.load().gocr_op_kv_write_paged(P, P, P, P, P, P, None, 7, 8, 512, 256, 256, 1e4, None) == EINVAL


def test_strides_of_single_entries_count_for_nothing(g):
    """A cache of one page, or of one head: whatever stride the framework gave that dimension, the call goes on to
    the next check (here: a null pointer)."""
    def call(kv):
        return g.load().gocr_op_kv_write_paged(None, P, P, P, P, P, ctypes.byref(_cache(g, **kv)), 7, 8, 512, 256, 256,
                                               1e4, None)
    assert call(dict(n_pages=1, k_page=1, v_page=0)) == EINVAL and "null" in _message(g)
    assert call(dict(n_kv_heads=1, k_head=3, v_head=-8)) == EINVAL and "null" in _message(g)
    # a token's heads together, pages of k and v interleaved, a dimension inside another one in any order
    assert call(dict(k_token=256, k_head=64, k_page=8192, v_token=512, v_head=64, v_page=8192)) == EINVAL
    assert "null" in _message(g)
    assert call(dict(k_page=64, k_token=512, k_head=8192)) == EINVAL and "null" in _message(g)


def test_attention_paged_refusals(g):
    names = ("q", "table", "cu", "kv_len", "o", "lse", "ws")
    need = g.load().gocr_op_attention_paged_workspace(7, 8, 4, 64)
    assert need > 0
    assert [g.load().gocr_op_attention_paged_workspace(*a) for a in ((-1, 8, 4, 64), (7, 0, 4, 64), (7, 8, 0, 64))] == [0] * 3

    def call(R=4, width=8, kind=2, T=7, Hq=8, ld=512, scale=0.125, n=need, kv=None, **ptr):
        p = lambda k: ptr.get(k, P)
        kv = ctypes.byref(_cache(g, **(kv or {})))
        return g.load().gocr_op_attention_paged(p("q"), kv, p("table"), width, p("cu"), p("kv_len"), kind, p("o"),
                                                p("lse"), R, T, Hq, ld, scale, p("ws"), n, None)
    for k in names:
        assert call(**{k: None}) == EINVAL and "null" in _message(g), k
        assert call(**{k: ODD}) == EINVAL and "aligned" in _message(g), k
    for bad in (dict(R=-1), dict(R=4097), dict(width=0), dict(width=(1 << 20) + 1), dict(T=-1), dict(T=(1 << 24) + 1),
                dict(Hq=0), dict(Hq=6), dict(Hq=1028), dict(Hq=260)):
        assert call(**bad) == EINVAL and "shape" in _message(g), bad
    for bad in (504, 516, 1 << 33):
        assert call(ld=bad) == EINVAL and "pitch" in _message(g)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == EINVAL and "scale" in _message(g)
    for bad in (-1, 3):
        assert call(kind=bad) == EINVAL and "kind" in _message(g)
    for bad in BAD_STRIDES:
        assert call(kv=bad) == EINVAL and "strides" in _message(g), bad
    assert call(kv=dict(page_size=512)) == EINVAL and call(kv=dict(head_dim=32)) == EINVAL
    assert call(n=need - 1) == ECAPACITY and "workspace" in _message(g)
    # strides whose common divisor is too small for the cache's extent
    assert call(kv=dict(n_pages=1 << 26, k_page=4104, v_page=4104)) == EINVAL and "unit" in _message(g)
    assert call(kv=dict(n_pages=1 << 26, v_page=4104)) == EINVAL and "unit" in _message(g)
    # more work than 32 bits count
    big = g.load().gocr_op_attention_paged_workspace(1 << 21, 8, 4, 64)
    assert call(T=1 << 21, R=4096, width=1 << 16, n=big) == EINVAL and "shape" in _message(g)


def test_attention_paged_workspaces_serve_fewer_rows(g):
    for heads in ((1, 1, 64), (12, 4, 128), (64, 1, 128)):
        sizes = [g.load().gocr_op_attention_paged_workspace(T, *heads) for T in (0, 1, 2, 33, 64, 100, 1000, 1 << 20)]
        assert sizes == sorted(sizes)


def test_paged_wrappers_check_tensors(g):
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    step = lambda **kw: g.op_page_step(**{**dict(held=i(4), start=i(4), end=i(4), table=i(4, 8), free_pages=i(32),
                                                 n_free=i(1), page_size=16, rows=9), **kw})
    for kw, what in ((dict(), "CUDA"), (dict(held=i(3)), "held must be"), (dict(table=i(4)), "dimensions"),
                     (dict(end=i(4).long()), "int32"), (dict(n_free=i(2)), "n_free"), (dict(rows=-1), "size"),
                     (dict(rows=1 << 31), "size"), (dict(table=i(8, 4).T), "contiguous"), (dict(page_size=1 << 32), "size")):
        with pytest.raises(ValueError, match=what):
            step(**kw)
    write = lambda **kw: g.op_kv_write_paged(**{**dict(q=b(5, 8, 64), k=b(5, 4, 64), v=b(5, 4, 64), pos=i(5), slots=i(5),
                                                       k_cache=b(8, 4, 16, 64), v_cache=b(8, 4, 16, 64)), **kw})
    for kw, what in ((dict(), "CUDA"), (dict(k=b(5, 8, 64)), "k must be"), (dict(q=b(5, 8, 128)), "heads of"),
                     (dict(v_cache=b(7, 4, 16, 64)), "v_cache"), (dict(k_cache=b(8, 4, 64, 16).transpose(2, 3)), "contiguous"),
                     (dict(slots=i(4)), "slots"), (dict(k_cache=b(8, 4, 16, 64).float()), "bfloat16"),
                     (dict(q=b(5, 8, 64).requires_grad_()), "requires grad")):
        with pytest.raises(ValueError, match=what):
            write(**kw)
    attend = lambda **kw: g.op_attention_paged(**{**dict(q=b(5, 8, 64), k_cache=b(8, 4, 16, 64), v_cache=b(8, 4, 16, 64),
                                                         table=i(2, 3), cu_rows=i(3), kv_len=i(2)), **kw})
    for kw, what in ((dict(), "CUDA"), (dict(cu_rows=i(2)), "cu_rows"), (dict(kv_len=i(3)), "kv_len"),
                     (dict(table=i(6)), "dimensions"), (dict(q=b(5, 8, 128)), "heads of")):
        with pytest.raises(ValueError, match=what):
            attend(**kw)
