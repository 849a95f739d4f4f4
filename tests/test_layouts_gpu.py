"""Layouts that the serving calls allow beside the usual ones: broadcast and overlapping rows and heads,
strided results, tensors of more than 2^31 elements; and the references that a run leaves."""

import pytest
import torch

import serving_ref as ref
from test_pages_gpu import Both, _i32

pytestmark = pytest.mark.gpu

LENS = [200, 57]
T = sum(LENS)


def _fd():
    import split_kv_decode_flashdecoding_b200 as fd
    return fd


def _rand(*shape, seed=5):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


LAYOUTS = {
    "broadcast kv heads": lambda: (_rand(T, 8, 128), _rand(T, 1, 128, seed=6).expand(T, 4, 128), _rand(T, 1, 128, seed=7).expand(T, 4, 128)),
    "broadcast q heads": lambda: (_rand(T, 1, 128).expand(T, 8, 128), _rand(T, 1, 128, seed=6), _rand(T, 1, 128, seed=7)),
    "one key for all": lambda: (_rand(T, 8, 128), _rand(1, 2, 128, seed=6).expand(T, 2, 128), _rand(1, 2, 128, seed=7).expand(T, 2, 128)),
    "overlapping rows": lambda: (_rand(T, 8, 128), _rand(T + 20, 128, seed=6).as_strided((T, 2, 128), (128, 256, 1)),
                                 _rand(T + 20, 128, seed=7).as_strided((T, 2, 128), (128, 512, 1))),
}


@pytest.mark.parametrize("layout", LAYOUTS)
def test_prompt_layouts(layout):
    q, k, v = LAYOUTS[layout]()
    out, lse = _fd().fd_prompt_attention(q, k, v, _i32(LENS))
    assert _fd().fd_poll_status() == 0
    ref.check_rows(out, lse, ref.prompt(q, k, v, LENS), layout)


def test_results_into_a_part_of_a_tensor():
    q, k, v = _rand(T, 8, 128), _rand(T, 2, 128, seed=6), _rand(T, 2, 128, seed=7)
    wide = torch.full((T, 11, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = _fd().fd_prompt_attention(q, k, v, _i32(LENS), out=wide[:, 1:9, 16:144])
    ref.check_rows(out, lse, ref.prompt(q, k, v, LENS))
    for rest in (wide[:, 0], wide[:, 9:], wide[:, :, :16], wide[:, :, 144:]):
        assert bool((rest == 3.0).all())


def test_tree_over_a_broadcast_cache():
    k, v = (_rand(1, 1, 90, 128, seed=s).expand(3, 2, 90, 128) for s in (6, 7))
    q, prefix, new = _rand(9, 8, 128), [80, 5, 0], [3, 3, 3]
    see = [torch.ones(3, 3, dtype=torch.bool).tril()] * 3
    out, lse = _fd().fd_tree_attention(q, k, v, _i32(prefix), _i32(new), ref.mask_words(see, 1).cuda())
    caches = [(k[b].transpose(0, 1), v[b].transpose(0, 1)) for b in range(3)]
    ref.check_rows(out, lse, ref.tree(q, caches, prefix, new, see))


def test_append_of_a_broadcast_row():
    s = Both(4, 2, 16, 128, 1, 2)
    s.reserve([20])
    x = _rand(1, 2, 128).expand(9, 2, 128)
    _fd().fd_pages_append(x, x, s.k, s.v, s.table, _i32([3]), _i32([9]))
    s.host.append(x.cpu(), x.cpu(), [3], [9])
    s.same()


def test_prompts_behind_2_to_the_31_elements():
    n = 265
    q, k, v = _rand(n * 1024, 64, 128), _rand(n * 1024, 4, 128, seed=6), _rand(n * 1024, 4, 128, seed=7)
    assert q.numel() > 1 << 31
    out, lse = _fd().fd_prompt_attention(q, k, v, _i32([1024] * n))
    for b in (0, 262, 264):
        rows = slice(1024 * b, 1024 * b + 1024)
        ref.check_rows(out[rows], lse[rows], ref.prompt(q[rows], k[rows], v[rows], [1024]), f"prompt {b}")


def test_tree_over_a_cache_of_more_than_2_to_the_31_elements():
    batch, cap = 36, 65536
    k, v, q = _rand(batch, 8, cap, 128), _rand(batch, 8, cap, 128, seed=6), _rand(4 * batch, 16, 128, seed=7)
    assert k.numel() > 1 << 31
    prefix, see = [60000 - 100 * b for b in range(batch)], [torch.ones(4, 4, dtype=torch.bool).tril()] * batch
    out, lse = _fd().fd_tree_attention(q, k, v, _i32(prefix), _i32([4] * batch), ref.mask_words(see, 1).cuda())
    for b in (0, 33, 35):
        rows = slice(4 * b, 4 * b + 4)
        want = ref.tree(q[rows], [(k[b].transpose(0, 1), v[b].transpose(0, 1))], [prefix[b]], [4], [see[b]])
        ref.check_rows(out[rows], lse[rows], want, f"tree {b}")


@pytest.mark.parametrize("size", [8, 16, 128])
def test_references_of_a_run(size):
    s = Both(120, 2, size, 64, 6, 48)
    held = [150, 1, 77, 0, 0, 0]
    s.reserve(held)
    s.append([0] * 6, held)
    s.set_lens(held)
    s.fork([0, 0, 2], [3, 4, 5])
    for step in range(3):
        held = list(s.host.lens)
        new = [(7 * b + 5 * step) % 19 + 1 for b in range(6)]
        s.reserve([a + n for a, n in zip(held, new)])
        s.append(held, new)
        s.compact(held, [list(range(step, n, 3)) for n in new])
        s.same()
        assert int(s.refs.sum()) == sum(-(-n // size) for n in s.host.lens)
    assert size > 64 or int((s.refs > 1).sum()) > 0
