"""Host threads that call on one stream at the same time: a call's kernels stay together, and a workspace
that one thread grows is not taken from another's call."""

import threading

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


def _fd():
    import split_kv_decode_flashdecoding_b200 as fd
    return fd


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rand(*shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


class Decode:
    """Planner, splits and combine: three kernels that meet in the workspace."""

    def __init__(self):
        self.q, self.k, self.v = _rand(300, 16, 128, seed=1), _rand(300, 2, 64, 128, seed=2), _rand(300, 2, 64, 128, seed=3)
        self.lens = _i32([(11 * b) % 65 for b in range(300)])

    def call(self, stream):
        return _fd().fd_decode_attention(self.q, self.k, self.v, self.lens, 3, stream=stream)


class Rows:
    """One kernel whose pieces meet in the workspace."""

    def __init__(self):
        self.args = _rand(1700, 8, 128, seed=4), _rand(1700, 1, 128, seed=5), _rand(1700, 1, 128, seed=6), _i32([1600, 100])

    def call(self, stream):
        return _fd().fd_prompt_attention(*self.args, stream=stream)


class Pages:
    """Fork and compact: two kernels each, the second of which reads what the first left there."""

    def __init__(self):
        fd = _fd()
        self.k, self.v = _rand(400, 2, 8, 128, seed=7), _rand(400, 2, 8, 128, seed=8)
        self.refs, self.table = torch.zeros(400, dtype=torch.int32, device="cuda"), torch.full((60, 8), -1, dtype=torch.int32, device="cuda")
        self.lens = _i32([3 + b for b in range(30)] + [0] * 30)
        fd.fd_pages_reserve(self.refs, self.table, self.lens, 8)
        self.src, self.dst = _i32(list(range(30))), _i32(list(range(59, 29, -1)))
        self.zero, self.keep, self.kept = _i32([0] * 60), _i32([[2, 5]] * 60), _i32([-1] * 30 + [1] * 30)

    def call(self, stream):
        fd = _fd()
        with torch.cuda.stream(stream):
            state = [x.clone() for x in (self.k, self.v, self.refs, self.table, self.lens)]
        fd.fd_pages_fork(*state, self.src, self.dst, stream=stream)
        # what the forks keep is their third token: on a shared page, unless it is their only one
        fd.fd_pages_compact(*state, self.zero, self.keep, self.kept, stream=stream)
        return state


@pytest.mark.parametrize("grow", [False, True])
def test_calls_of_several_threads_on_one_stream(grow):
    fd = _fd()
    kinds = [Decode(), Rows(), Pages()]
    alone = torch.cuda.Stream()
    torch.cuda.synchronize()
    fd.fd_poll_status(stream=alone)  # what a test before left on this stream
    want = [k.call(alone) for k in kinds]
    torch.cuda.synchronize()
    flags = fd.fd_poll_status(stream=alone)
    assert flags == fd.FD_FLAG_BAD_PAGE  # of the forks whose third token stands on a shared page
    s = torch.cuda.Stream()
    got, errors = [[] for _ in kinds], []

    def work(i):
        try:
            for _ in range(25):
                got[i].append(kinds[i].call(s))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    def enlarge():
        try:
            for n in range(1, 20):
                fd.fd_reserve_workspace(n * (7 << 20), stream=s)
                fd.fd_poll_status(stream=s)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(kinds)) for _ in range(2)]
    threads += [threading.Thread(target=enlarge)] if grow else []
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for results, expected in zip(got, want):
        assert len(results) == 50
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, expected))
    p = kinds[1]
    ref.check_rows(*want[1], ref.prompt(*p.args[:3], [1600, 100]), "rows")
