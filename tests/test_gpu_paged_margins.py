"""Lengths, tables and row ranges that contradict one another: nothing beside the arrays of a call is written."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EDGE = 4096  # elements on both sides


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    from self_speculative_block_gb300 import build, gocr
    build.build()
    gocr.load()
    return gocr


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Fenced:
    """Arrays within larger ones of one value."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype, fill):
        n = 1
        for s in shape:
            n *= s
        whole = torch.full((n + 2 * EDGE,), fill, dtype=dtype, device="cuda")
        self.all.append((whole, fill))
        return whole[EDGE:EDGE + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for whole, fill in self.all:
            assert (whole[:EDGE] == fill).all() and (whole[-EDGE:] == fill).all()


def _attend(g, cu, kv_len, table, T, Hq, Hkv, d, ps, n_pages, kind):
    f = Fenced()
    r = torch.Generator(device="cuda").manual_seed(1)
    kc, vc = (torch.randn((n_pages, Hkv, ps, d), generator=r, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((T, Hq, d), generator=r, device="cuda").bfloat16()
    o, lse = f((T, Hq, d), torch.bfloat16, 7.0), f((Hq, T), torch.float32, 7.0)
    ws = f((g.load().gocr_op_attention_paged_workspace(T, Hq, Hkv, d),), torch.uint8, 0)
    g.op_attention_paged(q, kc, vc, table, i32(cu), i32(kv_len), kind=kind, o=o, lse=lse, workspace=ws)
    g.op_status()
    f.check()
    return o


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (12, 4, 128), (64, 1, 128)])
@pytest.mark.parametrize("cu", [[0, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 5, 300], [300, 5, 0], [0, 300, 5], [7, 7, 299],
                                [299, 300, 2 ** 31 - 1], [300, 300, 300], [0, 300, -1, 300, 0, 300]])
def test_attention_paged_row_ranges(g, cu, Hq, Hkv, d, kind):
    R = len(cu) - 1
    table = torch.arange(R * 40, dtype=torch.int32, device="cuda").view(R, 40) % 50
    for kv_len in ([600] * R, [17, 2 ** 31 - 1, 0, -5, 640][:R], [1] * R):
        o = _attend(g, cu, kv_len, table, 300, Hq, Hkv, d, 16, 50, kind)
        lo = min(max(min(cu), 0), 300)
        assert (o[:lo] == 7.0).all()


def test_attention_paged_more_work_than_32_bits_count(g):
    """2,048 requests of the same 1,024 rows over 13,421,760 keys each: 2^32 + 24,576 units of work."""
    R, T, kv, ps = 4096, 1024, 13421760, 256
    table = torch.zeros((R, -(-kv // ps)), dtype=torch.int32, device="cuda")
    _attend(g, [T * (r & 1) for r in range(R + 1)], [kv] * R, table, T, 1, 1, 64, ps, 3, g.FWD_VERIFY)


@pytest.mark.parametrize("n_free", [-2 ** 31, -3, 0, 8, 2 ** 31 - 1])
@pytest.mark.parametrize("lens", [([64, 0, 20], [0, 0, 20], [64, 0, 64]), ([64, 64, 64], [0, 0, 0], [0, 0, 0]),
                                  ([0, 0, 0], [0, 0, 0], [64, 64, 64]), ([64, 64, 0], [0, 64, 0], [0, 64, 64]),
                                  ([2 ** 31 - 1, -2 ** 31, 64], [0, -2 ** 31, 64], [2 ** 31 - 1, 2 ** 31 - 1, 65])])
def test_page_step_state(g, lens, n_free):
    n_pages, ps, R, T = 8, 16, 3, 128
    f = Fenced()
    (held, start, end), below = (i32(x) for x in lens), i32([n_free])
    table, free = f((R, 4), torch.int32, 77), f((n_pages,), torch.int32, 77)
    table.copy_(i32([[99, -7, 5, 2 ** 31 - 1], [3, 4, -2 ** 31, 8], [0, 1, 2, 3]]))
    free.copy_(i32([2 ** 31 - 1, -5, 8, 1000, 7, 6, -1, 3]))
    height, out_held, kv_len, cu, pos, slots = (f((n,), torch.int32, 77) for n in (1, R, R, R + 1, T, T))
    p = lambda t: t.data_ptr()
    rc = g.load().gocr_op_page_step(p(held), p(start), p(end), R, p(table), 4, ps, p(free), n_pages, p(below),
                                    p(height), p(out_held), p(kv_len), p(cu), p(pos), p(slots), T,
                                    torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    f.check()
    assert 0 <= int(height) <= n_pages
    assert int(slots.max()) < n_pages * ps and int(slots.min()) >= -1
    c = cu.tolist()
    assert c[0] == 0 and c == sorted(c) and c[-1] <= T
    assert int(kv_len.min()) >= 0 and int(kv_len.max()) <= 4 * ps
