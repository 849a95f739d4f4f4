"""fd_poll_status works on the polled stream: it does not wait for other streams' work, and what it
clears is cleared before the stream's next call runs."""

import time

import pytest
import torch

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("static", [False, True])
def test_poll_does_not_wait_for_the_default_stream(static):
    import split_kv_decode_flashdecoding_b200 as fd
    s = torch.cuda.Stream()
    refs, table, want = _i32([0] * 4), _i32([[-1, -1]]), _i32([9])
    q, kv = torch.randn((1, 8, 64), device="cuda"), torch.randn((1, 8, 40, 64), device="cuda")
    out, lse, lens = torch.empty_like(q), torch.empty((1, 8), device="cuda"), _i32([40])
    if static:  # the static scratch holds a status word of its own
        fd.fd_decode_attention_static(q, kv, kv, lens, 0, out, lse)
    torch.cuda.synchronize()
    fd.fd_poll_status(stream=s)  # what a test before left on this stream
    fd.fd_pages_reserve(refs, table, want, 8, stream=s)
    assert fd.fd_poll_status(stream=s) == 0
    torch.cuda._sleep(1_000_000_000)  # half a second of the default stream
    busy = torch.cuda.Event()
    busy.record()
    t0 = time.perf_counter()
    flags = fd.fd_poll_status(stream=s)
    waited, still = time.perf_counter() - t0, not busy.query()
    torch.cuda.synchronize()
    assert flags == 0 and still and waited < 0.2


def test_flags_of_calls_in_a_row():
    import split_kv_decode_flashdecoding_b200 as fd
    s = torch.cuda.Stream()
    refs, table = _i32([0] * 4), _i32([[-1, -1]])
    good, bad = _i32([9]), _i32([100])
    torch.cuda.synchronize()
    fd.fd_poll_status(stream=s)
    for _ in range(200):
        fd.fd_pages_reserve(refs, table, bad, 8, stream=s)
        assert fd.fd_poll_status(stream=s) == fd.FD_FLAG_LEN_CLAMPED
        fd.fd_pages_reserve(refs, table, good, 8, stream=s)
        assert fd.fd_poll_status(stream=s) == 0
