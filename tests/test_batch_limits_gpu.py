"""Calls at the batches and list lengths where a kernel's shared memory passes 48 KB, up to the largest
allowed, 4096: page operators against their definitions on the host, planners against the host planner
and the 64-bit reference."""

import pytest
import torch

import serving_ref as ref
from test_pages_gpu import Both, _fd, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [4053, 4054, 4095, 4096])
def test_reserve_of_many_sequences(batch):
    s = Both(batch + 50, 1, 8, 64, batch, 2)
    want = [1 + (5 * b) % 3 for b in range(batch)]
    assert s.reserve(want)
    s.same()
    assert not s.reserve([16] * batch)
    s.same(_fd().FD_FLAG_POOL_FULL)


@pytest.mark.parametrize("count,batch", [(2047, 4094), (2048, 4096), (2960, 256), (3056, 64), (3055, 100), (4096, 4096)])
def test_fork_of_many_pairs(count, batch):
    fd = _fd()
    half = min(batch // 2, 2048)
    s = Both(2 * half + 20, 1, 8, 64, batch, 2)
    lens = [1 + (3 * b) % 16 for b in range(half)] + [0] * (batch - half)
    s.reserve([8 if n else 0 for n in lens])  # a page each: sequences of more than 8 tokens lack one
    s.set_lens(lens)
    src, dst = [i % half for i in range(count)], [half + i % (batch - half) for i in range(count)]
    s.fork(src, dst)
    flags = fd.FD_FLAG_BAD_PAGE | (fd.FD_FLAG_BAD_INDEX if count > batch - half else 0)
    s.same(flags)


def test_page_operators_at_the_largest_batch():
    s = Both(9000, 2, 8, 64, 4096, 3)
    lens = [(7 * b) % 17 for b in range(4096)]
    s.reserve(lens)
    s.append([0] * 4096, lens)
    s.set_lens(lens)
    s.same()
    s.compact([0] * 4096, [[n - 1] if n else None for n in lens])
    s.same()
    s.free(list(range(4095, -1, -1)))
    s.same()
    assert not s.refs.any()


@pytest.mark.parametrize("batch", [1746, 1747, 1755, 1756, 4096])
def test_decode_planner(batch):
    fd = _fd()
    lens = [(37 * b) % 3000 for b in range(batch)]
    info, splits, items = fd.fd_split_plan(lens, 2, 3000)
    total, got, rows = fd.fd_split_plan_device(_i32(lens), 2, 3000, items_capacity=info["total_items"])
    assert int(total) == info["total_items"] and got.tolist() == splits
    assert sorted(map(tuple, rows.tolist())) == sorted(items)


@pytest.mark.parametrize("batch", [868, 869, 877, 878, 4096])
def test_chunk_planner(batch):
    fd = _fd()
    gen = torch.Generator(device="cuda").manual_seed(batch)
    hq, hkv, d, cap = 2, 1, 64, 16
    prefix, new = [(5 * b) % 9 for b in range(batch)], [(3 * b) % 4 for b in range(batch)]
    q = torch.randn((sum(new), hq, d), generator=gen, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((batch, hkv, cap, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, lse = fd.fd_chunk_prefill_attention(q, k, v, _i32(prefix), _i32(new))
    torch.cuda.synchronize()
    assert fd.fd_poll_status() == 0
    some = [b for b in range(batch) if new[b] and (batch < 1000 or b % 7 == 0)]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    for b in some:
        n, p = new[b], prefix[b]
        rows = slice(starts[b], starts[b] + n)
        see = torch.ones((n, p + n), dtype=torch.bool, device="cuda").tril(p)
        want = ref.attend(q[rows], k[b, :, :p + n].transpose(0, 1), v[b, :, :p + n].transpose(0, 1), see)
        ref.check_rows(out[rows], lse[rows], want, f"request {b}")
