"""gocr_op_status: a wait that runs out is reported, once to every thread that
asks, and a report is neither lost nor taken by another thread."""
import threading

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


def _status(g):
    """None, or the message."""
    try:
        g.op_status()
    except g.GocrError as e:
        return str(e)


def _give_up(g, us=200):
    """A kernel on the current stream whose wait runs out after `us` microseconds."""
    assert g.load().gocr_op_wait_probe(us, torch.cuda.current_stream().cuda_stream) == g.GOCR_OK


def test_a_wait_that_gives_up_is_reported_once(g):
    _status(g)
    assert _status(g) is None
    _give_up(g)
    assert "gave up" in _status(g)
    assert _status(g) is None


def test_another_stream_keeps_its_outputs(g):
    """The context goes on after a report."""
    _status(g)
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    table = torch.randn((4, 64), device="cuda")
    _give_up(g)
    y = g.op_embed(ids, table)
    assert "gave up" in _status(g)
    assert torch.equal(y, table)


def test_no_thread_takes_another_ones_report(g):
    _status(g)
    ready, failed, seen = threading.Barrier(2), threading.Event(), []

    def other():
        _status(g)                  # whatever came before
        ready.wait(30)
        assert failed.wait(30)
        seen.append(_status(g))     # asks after the first thread has asked

    t = threading.Thread(target=other)
    t.start()
    ready.wait(30)
    _give_up(g)
    mine = _status(g)
    failed.set()
    t.join(60)
    assert "gave up" in mine and seen and seen[0] is not None and "gave up" in seen[0]


def test_reports_between_two_questions_are_not_lost(g):
    """A second stream's kernel gives up while the first stream's status is being read."""
    _status(g)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _give_up(g, 20_000)
    first = _status(g)              # of the current stream: does not wait for the other
    s.synchronize()
    second = _status(g)
    assert (first is None) != (second is None)


def test_status_of_a_capturing_stream_is_refused_and_the_capture_goes_on(g):
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    table = torch.randn((4, 64), device="cuda")
    g.op_embed(ids, table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = g.op_embed(ids, table)
        assert g.load().gocr_op_status(torch.cuda.current_stream().cuda_stream) == -1  # GOCR_EINVAL
        z = g.op_embed(ids, table, scale=2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, table) and torch.equal(z, 2 * table)
