"""The library's workspace: one buffer a stream, and beside it only those that a captured call used."""

import pytest
import torch

pytestmark = pytest.mark.gpu

MB = 1 << 20


@pytest.fixture(autouse=True)
def no_workspaces():
    """torch hands its streams out again: one may hold a workspace of a test before."""
    import split_kv_decode_flashdecoding_b200 as fd
    fd.fd_shutdown()


def _used():
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return (total - free) / MB


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_a_workspace_that_grows_gives_its_old_buffer_back():
    import split_kv_decode_flashdecoding_b200 as fd
    s = torch.cuda.Stream()
    fd.fd_reserve_workspace(2 * MB, stream=s)
    before = _used()
    fd.fd_reserve_workspace(600 * MB, stream=s)
    assert 590 <= _used() - before <= 610
    fd.fd_reserve_workspace(700 * MB, stream=s)
    assert 690 <= _used() - before <= 710
    fd.fd_reserve_workspace(100 * MB, stream=s)  # held already
    assert 690 <= _used() - before <= 710


def test_flags_outlive_a_workspace_that_grows():
    import split_kv_decode_flashdecoding_b200 as fd
    s = torch.cuda.Stream()
    refs, table = _i32([0] * 4), _i32([[-1, -1]])
    fd.fd_pages_reserve(refs, table, _i32([100]), 8, stream=s)
    fd.fd_reserve_workspace(16 * MB, stream=s)
    fd.fd_reserve_workspace(32 * MB, stream=s)
    assert fd.fd_poll_status(stream=s) == fd.FD_FLAG_LEN_CLAMPED
    assert fd.fd_poll_status(stream=s) == 0


def test_a_buffer_that_a_graph_uses_stays():
    import split_kv_decode_flashdecoding_b200 as fd
    s = torch.cuda.Stream()
    refs, table, want = _i32([0] * 40), _i32([[-1] * 4] * 8), _i32([17] * 8)
    torch.cuda.synchronize()
    graphs = []
    for size in (300, 700):
        fd.fd_reserve_workspace(size * MB, stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fd.fd_pages_reserve(refs, table, want, 8)
        graphs.append(g)
    before = _used()
    fd.fd_reserve_workspace(1500 * MB, stream=s)  # both graphs' buffers stay beside it
    assert 1490 <= _used() - before <= 1510
    fd.fd_reserve_workspace(1600 * MB, stream=s)  # that one no graph uses
    assert 1590 <= _used() - before <= 1610
    for g in graphs:
        refs.zero_(), table.fill_(-1), want.fill_(17)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert table.tolist() == [[3 * b, 3 * b + 1, 3 * b + 2, -1] for b in range(8)]
        assert fd.fd_poll_status(stream=s) == 0
        want.fill_(1000)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert fd.fd_poll_status(stream=s) == fd.FD_FLAG_LEN_CLAMPED  # the graph's own status word is polled
