"""Serving calls on a torch stream other than the current one: memory that the caching allocator hands
out for the call, or takes back from its arguments, is not used by both streams at once. A stream is held
up by a spin where the order would show."""

import types

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

SPIN = 200_000_000  # a tenth of a second


def _fd():
    import split_kv_decode_flashdecoding_b200 as fd
    return fd


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rand(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


class Prompt:
    def __init__(self):
        self.args = _rand(300, 16, 128), _rand(300, 2, 128, seed=2), _rand(300, 2, 128, seed=3), _i32([100, 200])

    def __call__(self, args, **kw):
        return _fd().fd_prompt_attention(*args, **kw)


class Tree:
    def __init__(self):
        see = [ref.random_tree(torch.Generator().manual_seed(4), n) for n in (30, 20)]
        self.args = (_rand(50, 16, 128), _rand(2, 2, 200, 128, seed=2), _rand(2, 2, 200, 128, seed=3), _i32([150, 90]), _i32([30, 20]),
                     ref.mask_words(see, 1).cuda())

    def __call__(self, args, **kw):
        return _fd().fd_tree_attention(*args, **kw)


def _copies(args):
    return tuple(x.clone() for x in args)


@pytest.mark.parametrize("kind", [Prompt, Tree])
def test_new_results_are_free_of_the_current_streams_work(kind):
    call = kind()
    want = call(call.args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(call.args, stream=s)  # the workspace of the stream
    torch.cuda.synchronize()
    held = [torch.empty_like(x) for x in want]
    torch.cuda._sleep(SPIN)
    for x in held:
        x.fill_(7.0)      # runs long after the call below
    del held, x           # memory of the results' sizes, free for the current stream
    got = call(call.args, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("kind", [Prompt, Tree])
def test_arguments_may_be_dropped_after_the_call(kind):
    call = kind()
    want = call(call.args)
    out, lse = (torch.empty_like(x) for x in want)
    s = torch.cuda.Stream()
    call(call.args, stream=s)
    args = _copies(call.args)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    call(args, out=out, lse=lse, stream=s)
    shapes = [(x.shape, x.dtype) for x in args]
    del args
    other = [torch.full(n, 1, dtype=t, device="cuda") for n, t in shapes]  # overwrites what the current stream was given back
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and len(other) > 0


@pytest.mark.parametrize("kind", [Prompt, Tree])
def test_results_may_be_dropped_while_the_current_stream_reads_them(kind):
    call = kind()
    want = call(call.args)
    zero = list(_copies(call.args))
    zero[2] = torch.zeros_like(zero[2])  # v: all results 0
    s = torch.cuda.Stream()
    call(call.args, stream=s)
    torch.cuda.synchronize()
    got = call(call.args, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SPIN)
    copies = [x.clone() for x in got]    # not before the spin is over
    del got
    for _ in range(4):
        call(zero, stream=s)             # might write to the memory that is still to be copied
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, copies))


def test_page_operators_arguments_may_be_dropped():
    fd = _fd()
    s = torch.cuda.Stream()
    k_pages, v_pages = (torch.zeros((12, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    refs, table, lens = _i32([0] * 12), _i32([[-1] * 4] * 3), _i32([40, 20, 0])
    x = _rand(60, 2, 128, seed=9)
    fd.fd_reserve_workspace(1 << 20, stream=s)
    args = [x.clone(), x.neg(), _i32([40, 20, 0]), _i32([0, 0, 0]), _i32([0]), _i32([2]), _i32([32, 2, 0]),
            _i32([[1, 4, 6], [0, 0, 0], [0, 0, 0]]), _i32([3, -1, -1]), _i32([1])]
    k, v, want, zero, src, dst, start, keep, kept, gone = args
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    fd.fd_pages_reserve(refs, table, want, 16, stream=s)
    fd.fd_pages_append(k, v, k_pages, v_pages, table, zero, want, stream=s)
    fd.fd_pages_fork(k_pages, v_pages, refs, table, lens, src, dst, stream=s)
    fd.fd_pages_free(refs, table, lens, gone, stream=s)
    fd.fd_pages_compact(k_pages, v_pages, refs, table, lens, start, keep, kept, stream=s)
    shapes = [(y.shape, y.dtype) for y in args]
    del args, k, v, want, zero, src, dst, start, keep, kept, gone
    other = [torch.full(n, 1, dtype=t, device="cuda") for n, t in shapes for _ in range(2)]
    torch.cuda.synchronize()
    assert len(other) > 0 and fd.fd_poll_status(stream=s) == 0
    assert lens.tolist() == [35, 0, 40] and table.tolist() == [[0, 1, 2, -1], [-1] * 4, [0, 1, 5, -1]]
    assert refs.tolist() == [2, 2, 1, 0, 0, 1] + [0] * 6
    for pool, y in ((k_pages, x), (v_pages, x.neg())):
        assert torch.equal(pool[2, :, :3].transpose(0, 1), y[[33, 36, 38]]) and torch.equal(pool[5, :, :8].transpose(0, 1), y[32:40])


def test_kinds_of_streams():
    fd = _fd()
    call = Prompt()
    want = call(call.args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream), torch.cuda.default_stream(), 0):
        got = call(call.args, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), stream
    with torch.cuda.stream(s):
        got = call(call.args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(TypeError):
        call(call.args, stream="s")
    elsewhere = types.SimpleNamespace(stream_id=0, device_index=torch.cuda.current_device() + 1, device_type=s.device_type)
    with pytest.raises(ValueError, match="the stream is not one of cuda:0"):
        call(call.args, stream=elsewhere)
    assert fd.fd_poll_status() == 0 and fd.fd_poll_status(stream=s) == 0


def test_a_call_on_another_stream_in_a_graph():
    fd = _fd()
    call = Prompt()
    want = call(call.args)
    s, side = torch.cuda.Stream(), torch.cuda.Stream()
    for x in (s, side):
        fd.fd_reserve_workspace(fd.fd_prompt_workspace_bytes(2, 300, 16, 2, 128), stream=x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        side.wait_stream(s)
        got = call(call.args, stream=side)
        s.wait_stream(side)
        copies = [x.clone() for x in got]
    for _ in range(3):
        for x in copies:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, copies))
