"""The page step where its counts and its shared memory are largest."""
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


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("R", [257, 1024, 4096])
def test_page_step_more_rows_than_32_bits_count(g, R):
    """Requests of 2^23 rows each, 2^33 in all: the first two fill the 2^24 rows, every other one is refused."""
    n, ps = 1 << 23, 256
    each = n // ps
    n_pages, T = 2 * each + 5, 2 * n
    table = torch.full((R, each), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(n_pages, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.int32)
    zero = torch.zeros((R,), dtype=torch.int32, device="cuda")
    s = g.op_page_step(zero, zero, zero + n, table, order.clone(), i32([n_pages]), ps, T)
    pages = order.flip(0)[:2 * each].view(2, each)
    assert torch.equal(table[:2], pages) and (table[2:] == -1).all() and int(s.n_free) == 5
    first = torch.arange(R, device="cuda") < 2
    for x in (s.held, s.kv_len):
        assert torch.equal(x, torch.where(first, n, 0).to(torch.int32))
    assert s.cu_rows[:3].tolist() == [0, n, T] and (s.cu_rows[2:] == T).all()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(s.pos.view(2, n), pos.expand(2, n))
    assert torch.equal(s.slots.view(2, n), pages.repeat_interleave(ps, 1) * ps + pos % ps)
