"""The page step where its counts and its shared memory are largest."""
import os
import subprocess
import sys

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


def test_page_step_ends_behind_rows_that_do_not_fit(g):
    """From the first request on whose rows end behind the last row, none gives anything back or takes anything; asked
    again with what the step says they hold, they do."""
    ps, order = 16, list(range(12))
    table, free = torch.full((4, 4), -1, dtype=torch.int32, device="cuda"), i32(order)
    s = g.op_page_step(i32([0] * 4), i32([0] * 4), i32([16, 32, 40, 33]), table, free, i32([12]), ps, 121)
    assert int(s.n_free) == 3 and s.held.tolist() == [16, 32, 40, 33]
    before = table.tolist()
    # the first grows within the rows, the second does not fit, the third ends, the fourth is rolled back
    s = g.op_page_step(s.held, i32([16, 32, 0, 10]), i32([18, 35, 0, 10]), table, free, s.n_free, ps, 4)
    assert s.held.tolist() == [18, 32, 40, 33] and s.kv_len.tolist() == [18, 0, 0, 0] and int(s.n_free) == 2
    assert s.cu_rows.tolist() == [0, 2, 4, 4, 4] and s.pos.tolist() == [16, 17, -1, -1]
    before[0][1] = 2
    assert table.tolist() == before
    s = g.op_page_step(s.held, i32([18, 32, 0, 10]), i32([18, 32, 0, 10]), table, free, s.n_free, ps, 4)
    assert s.held.tolist() == [18, 32, 0, 10] and int(s.n_free) == 2 + 3 + 2
    assert free[:7].tolist() == [0, 1, before[3][2], before[3][1], before[2][2], before[2][1], before[2][0]]


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# a page each, the last request none: whatever shared memory the sizes before have asked for stays set
EVERY_REQUEST = """
import torch
from self_speculative_block_gb300 import gocr as g
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
for R in (4090, 4091, 4092, 4093, 4094, 4095, 4096):
    table = torch.full((R, 2), -1, dtype=torch.int32, device="cuda")
    zero = torch.zeros((R,), dtype=torch.int32, device="cuda")
    free = torch.arange(R - 1, dtype=torch.int32, device="cuda")
    s = g.op_page_step(zero, zero, zero + 3, table, free, i32([R - 1]), 16, 3 * R)
    page = torch.arange(R - 1, device="cuda", dtype=torch.int32).flip(0)
    assert torch.equal(table[:-1, 0], page) and int(table[-1, 0]) == -1 and (table[:, 1] == -1).all(), R
    assert int(s.n_free) == 0 and (s.kv_len[:-1] == 3).all() and int(s.kv_len[-1]) == 0, R
    assert torch.equal(s.slots[:-3].view(R - 1, 3), page[:, None] * 16 + i32([0, 1, 2])) and (s.slots[-3:] == -1).all(), R
print("served")
"""


def test_page_step_most_requests_in_a_new_process(g):
    """4,090 to 4,096 requests, the fewest first, where no larger call has raised the kernel's limit before."""
    r = subprocess.run([sys.executable, "-c", EVERY_REQUEST], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "served", r.stdout + r.stderr
