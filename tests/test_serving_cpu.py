"""CPU checks of the serving operators: their references against the float64 oracle and by hand, and
the argument errors, which return before anything touches a GPU."""

import ctypes

import numpy as np
import pytest
import torch

import serving_ref as ref
import split_kv_decode_flashdecoding_b200 as fd
from oracle import attention as oracle

INV, UNS = fd.FD_ERR_INVALID_ARGUMENT, fd.FD_ERR_UNSUPPORTED


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def test_prompt_reference_is_the_oracles_chunk_without_a_prefix():
    lens, hq, hkv, d = [5, 1, 9], 4, 2, 64
    q, k, v = (_rand(sum(lens), h, d, seed=i) for i, h in enumerate((hq, hkv, hkv)))
    cap = max(lens)
    kc, vc = np.zeros((3, hkv, cap, d), np.float32), np.zeros((3, hkv, cap, d), np.float32)
    at = 0
    for b, n in enumerate(lens):
        kc[b, :, :n], vc[b, :, :n] = (x[at:at + n].transpose(0, 1).numpy() for x in (k, v))
        at += n
    o, l = oracle.chunk_prefill_attention(q.numpy(), kc, vc, [0, 0, 0], lens)
    r = ref.prompt(q, k, v, lens)
    assert np.abs(r.out.numpy() - o).max() < 1e-12 and np.abs(r.lse.numpy() - l).max() < 1e-12


def test_tree_reference_of_a_line_is_the_oracles_verification():
    hq, hkv, d, pre, new = 4, 2, 64, [7, 0, 3], [4, 2, 1]
    q = _rand(sum(new), hq, d)
    kc, vc = _rand(3, hkv, 11, d, seed=1), _rand(3, hkv, 11, d, seed=2)
    o, l = oracle.chunk_prefill_attention(q.numpy(), kc.numpy(), vc.numpy(), pre, new)
    line = [torch.ones(n, n, dtype=torch.bool).tril() for n in new]
    r = ref.tree(q, [(kc[b].transpose(0, 1), vc[b].transpose(0, 1)) for b in range(3)], pre, new, line)
    assert np.abs(r.out.numpy() - o).max() < 1e-12 and np.abs(r.lse.numpy() - l).max() < 1e-12


def test_mask_words_and_empty_rows():
    see = [torch.zeros(3, 3, dtype=torch.bool), torch.eye(33, dtype=torch.bool)]
    w = ref.mask_words(see, 2)
    assert w[:3].abs().sum() == 0
    assert w[3 + 31, 0] == -(1 << 31) and w[3 + 32, 1] == 1 and w[3, 0] == 1
    r = ref.attend(_rand(1, 2, 64), _rand(4, 1, 64), _rand(4, 1, 64), torch.zeros(1, 4, dtype=torch.bool))
    assert not r.out.any() and bool((r.lse == -float("inf")).all())


def test_pool_reference_by_hand():
    k = torch.arange(6.0).view(6, 1, 1, 1).expand(6, 1, 4, 64).clone()
    pool = ref.Pool(k, -k, [0] * 6, [[-1] * 3 for _ in range(3)], [0] * 3)
    assert pool.reserve([6, 0, 3])
    assert pool.table == [[0, 1, -1], [-1] * 3, [2, -1, -1]] and pool.refs == [1, 1, 1, 0, 0, 0]
    rows = torch.arange(100.0, 109.0)[:, None, None].expand(9, 1, 64)
    pool.append(rows, rows, [0, 0, 0], [6, 0, 3])
    assert pool.k[0, 0, :, 0].tolist() == [100, 101, 102, 103] and pool.k[1, 0, :2, 0].tolist() == [104, 105]
    pool.lens = [6, 0, 3]
    pool.fork([0], [1])
    assert pool.table[1] == [0, 3, -1] and pool.refs == [2, 1, 1, 1, 0, 0] and pool.lens == [6, 6, 3]
    assert pool.k[3, 0, :, 0].tolist() == [104, 105, 3, 3]
    pool.compact([4, 0, 1], [[1], [0], [1]], [1, -1, 1])
    assert pool.k[1, 0, :2, 0].tolist() == [105, 105] and pool.k[2, 0, :3, 0].tolist() == [106, 108, 108]
    assert pool.lens == [5, 6, 2]
    pool.compact([0, 0, 0], [[], [0, 2], [0]], [0, 2, 1])  # the second writes a shared page: refused
    assert pool.lens == [0, 6, 1] and pool.table == [[-1] * 3, [0, 3, -1], [2, -1, -1]]
    assert pool.refs == [1, 0, 1, 1, 0, 0]
    pool.free([1, 1, 2])
    assert pool.refs == [0] * 6 and pool.lens == [0, 0, 0]
    assert not pool.reserve([13, 12, 1])  # 3 + 3 pages: the third sequence gets none
    assert pool.table == [[0, 1, 2], [3, 4, 5], [-1] * 3]


# ---- argument errors ----------------------------------------------------------------------------

def _fake(shape, dtype=fd.FD_BF16, strides=None, ptr=0x100000):
    t = fd.FdTensor()
    t.data, t.dtype, t.ndim = ptr, dtype, len(shape)
    if strides is None:
        strides = [int(np.prod(shape[i + 1:])) for i in range(len(shape))]
    for i, (n, s) in enumerate(zip(shape, strides)):
        t.shape[i], t.stride[i] = n, s
    return t


def _i(ptr=0x200000):
    return ctypes.cast(ctypes.c_void_p(ptr), ctypes.POINTER(ctypes.c_int32)) if ptr else None


def _f(ptr=0x300000):
    return ctypes.cast(ctypes.c_void_p(ptr), ctypes.POINTER(ctypes.c_float)) if ptr else None


def _ref(t):
    return ctypes.byref(t) if t is not None else None


def _prompt(q=(9, 8, 128), k=(9, 2, 128), v=None, out=None, lens=_i(), batch=2, lse=_f(), **kw):
    q = _fake(q) if isinstance(q, tuple) else q
    k = _fake(k) if isinstance(k, tuple) else k
    v = _fake((9, 2, 128)) if v is None else v
    out = _fake((9, 8, 128)) if out is None else out
    return fd.lib.fd_prompt_attention(_ref(q), _ref(k), _ref(v), lens, batch, _ref(out), lse, None)


def test_prompt_refusals():
    assert fd.lib.fd_prompt_attention(None, None, None, None, 1, None, None, None) == INV
    assert _prompt(q=(9, 7, 128), out=_fake((9, 7, 128))) == INV               # heads do not divide
    assert _prompt(q=_fake((9, 8, 128), fd.FD_F32)) == UNS
    assert _prompt(k=_fake((9, 2, 128), fd.FD_E4M3)) == UNS
    assert _prompt(k=(8, 2, 128)) == INV                                       # another row count
    assert _prompt(v=_fake((9, 1, 128))) == INV
    assert _prompt(out=_fake((9, 8, 64))) == INV
    assert _prompt(q=_fake((9, 8, 128), ptr=0x100008)) == UNS                  # data not 16-byte aligned
    assert _prompt(k=_fake((9, 2, 128), strides=[260, 128, 1])) == UNS         # stride not 16 bytes
    assert _prompt(k=_fake((9, 2, 128), strides=[512, 256, 2])) == UNS         # last dimension strided
    assert _prompt(batch=-1) == INV
    assert _prompt(batch=5000) == UNS
    assert _prompt(lens=None) == INV
    assert _prompt(lse=None) == INV
    q, kv = _fake((9, 34, 128)), _fake((9, 2, 128))
    assert _prompt(q=q, k=kv, out=_fake((9, 34, 128))) == UNS                  # groups of 17
    q, kv = _fake((9, 8, 96)), _fake((9, 2, 96))
    assert _prompt(q=q, k=kv, v=kv, out=_fake((9, 8, 96))) == UNS              # head_dim
    assert _prompt(batch=0) == fd.FD_OK                                        # nothing to do
    e = _fake((0, 8, 128), ptr=None)
    kv = _fake((0, 2, 128), ptr=None)
    assert _prompt(q=e, k=kv, v=kv, out=e) == fd.FD_OK


def _tree(q=(9, 8, 128), k=(3, 2, 50, 128), v=None, pre=_i(), new=_i(), mask=_i(), words=1, out=None, lse=_f()):
    q = _fake(q) if isinstance(q, tuple) else q
    k = _fake(k) if isinstance(k, tuple) else k
    v = k if v is None else v
    out = _fake((9, 8, 128)) if out is None else out
    return fd.lib.fd_tree_attention(_ref(q), _ref(k), _ref(v), pre, new, mask, words, _ref(out), lse, None)


def test_tree_refusals():
    assert _tree(words=0) == INV
    assert _tree(words=9) == UNS
    assert _tree(pre=None) == INV and _tree(new=None) == INV and _tree(mask=None) == INV and _tree(lse=None) == INV
    assert _tree(k=(3, 3, 50, 128)) == INV
    assert _tree(k=_fake((3, 2, 50, 128), fd.FD_E4M3)) == UNS
    assert _tree(k=_fake((3, 2, 50, 128), strides=[25600, 128, 256, 1])) == UNS  # token rows apart
    assert _tree(v=_fake((3, 2, 51, 128))) == INV
    assert _tree(v=_fake((3, 2, 50, 128), strides=[12808, 6400, 128, 1])) == UNS
    assert _tree(k=(3, 2, 0, 128)) == INV
    assert _tree(out=_fake((8, 8, 128))) == INV
    q, p, o = _fake((9, 8, 128)), _fake((7, 2, 16, 128)), _fake((9, 8, 128))

    def paged(pages=p, table=_i(), per=4, batch=3, words=1):
        return fd.lib.fd_tree_attention_paged(_ref(q), _ref(pages), _ref(pages), table, per, batch, _i(), _i(), _i(),
                                              words, _ref(o), _f(), None)
    assert paged(table=None) == INV
    assert paged(per=0) == INV
    assert paged(per=1 << 28) == UNS
    assert paged(batch=-1) == INV
    assert paged(pages=_fake((7, 2, 24, 128))) == UNS
    assert paged(pages=_fake((0, 2, 16, 128))) == INV
    assert paged(words=9) == UNS
    assert paged(batch=0) == fd.FD_OK


def test_page_operator_refusals():
    pages, new = _fake((7, 2, 16, 128)), _fake((9, 2, 128))

    def append(k=new, v=new, pk=pages, pv=None, table=_i(), per=4, batch=3, start=_i(), lens=_i()):
        return fd.lib.fd_pages_append(_ref(k), _ref(v), _ref(pk), _ref(pk if pv is None else pv), table, per, batch,
                                      start, lens, None)
    assert append(k=_fake((9, 3, 128))) == INV
    assert append(v=_fake((8, 2, 128))) == INV
    assert append(k=_fake((9, 2, 128), fd.FD_F32)) == INV
    assert append(pk=_fake((7, 2, 16, 128), fd.FD_E4M3)) == INV
    assert append(pv=_fake((7, 2, 16, 128), fd.FD_F32)) == INV
    assert append(pk=_fake((7, 2, 12, 128))) == UNS and append(pk=_fake((7, 2, 16, 96))) == UNS
    assert append(table=None) == INV and append(start=None) == INV and append(lens=None) == INV
    assert append(per=0) == INV and append(batch=4097) == UNS and append(batch=-1) == INV
    assert append(k=_fake((9, 2, 128), strides=[264, 132, 1])) == UNS
    assert append(batch=0) == fd.FD_OK
    codes = _fake((7, 2, 16, 128), fd.FD_E4M3)

    def fp8(k=new, pk=codes, ks=1.0, vs=1.0):
        return fd.lib.fd_pages_append_fp8(_ref(k), _ref(k), _ref(pk), _ref(pk), ks, vs, _i(), 4, 3, _i(), _i(), None)
    assert fp8(pk=pages) == INV
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert fp8(ks=bad) == INV and fp8(vs=bad) == INV
    assert fp8(k=_fake((9, 2, 128), fd.FD_E4M3)) == INV

    def reserve(refs=_i(), n=7, table=_i(), per=4, batch=3, want=_i(), size=16):
        return fd.lib.fd_pages_reserve(refs, n, table, per, batch, want, size, None)
    assert reserve(refs=None) == INV and reserve(table=None) == INV and reserve(want=None) == INV
    assert reserve(n=0) == INV and reserve(size=0) == INV and reserve(per=0) == INV and reserve(batch=4097) == UNS
    assert reserve(per=1 << 27, size=16) == UNS and reserve(batch=0) == fd.FD_OK

    def fork(pk=pages, refs=_i(), table=_i(), per=4, batch=3, lens=_i(), src=_i(), dst=_i(), count=2):
        return fd.lib.fd_pages_fork(_ref(pk), _ref(pk), refs, table, per, batch, lens, src, dst, count, None)
    assert fork(refs=None) == INV and fork(lens=None) == INV and fork(src=None) == INV and fork(dst=None) == INV
    assert fork(count=-1) == INV and fork(count=4097) == UNS and fork(batch=0) == INV and fork(count=0) == fd.FD_OK
    assert fork(pk=_fake((7, 2, 16, 128), strides=[4100, 2048, 128, 1])) == UNS

    def free(refs=_i(), n=7, table=_i(), per=4, batch=3, lens=_i(), seqs=_i(), count=2):
        return fd.lib.fd_pages_free(refs, n, table, per, batch, lens, seqs, count, None)
    assert free(refs=None) == INV and free(seqs=None) == INV and free(lens=None) == INV and free(table=None) == INV
    assert free(n=0) == INV and free(count=-1) == INV and free(count=4097) == UNS and free(count=0) == fd.FD_OK

    def compact(pk=pages, refs=_i(), lens=_i(), start=_i(), keep=_i(), most=5, kept=_i(), batch=3):
        return fd.lib.fd_pages_compact(_ref(pk), _ref(pk), refs, _i(), 4, batch, lens, start, keep, most, kept, None)
    assert compact(refs=None) == INV and compact(keep=None) == INV and compact(kept=None) == INV
    assert compact(most=-1) == INV and compact(start=None) == INV and compact(lens=None) == INV
    assert compact(batch=0) == fd.FD_OK


def test_binding_refuses_wrong_integer_tensors():
    q, kv = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    for lens in (torch.tensor([4]), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            fd.fd_prompt_attention(q, kv, kv, lens)
    pages = torch.zeros(3, 1, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fd.fd_pages_append(kv, kv, pages, pages, torch.zeros(2, 3, dtype=torch.int32),
                           torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        fd.fd_prompt_attention(q, kv, kv, torch.zeros(1, dtype=torch.int32), lse=torch.zeros(2, 4).T)


def test_workspace_sizes():
    assert fd.fd_prompt_workspace_bytes(3, 100, 8, 2, 128) >= 256
    assert fd.fd_tree_workspace_bytes(3, 100, 8, 2, 500, 128) >= 256
    assert fd.fd_prompt_workspace_bytes(-1, 100, 8, 2, 128) == 0
    assert fd.fd_tree_workspace_bytes(3, -1, 8, 2, 500, 128) == 0


def test_capacities_near_2_to_the_31_are_refused():
    big = 2**31 - 1023
    assert _prompt(q=_fake((big, 8, 128), strides=[0, 128, 1]), out=_fake((big, 8, 128), strides=[0, 128, 1])) == UNS

    def tree(pages, page_size):
        kv = _fake((4, 2, page_size, 64))
        q = _fake((3, 4, 64))
        return fd.lib.fd_tree_attention_paged(_ref(q), _ref(kv), _ref(kv), _i(), pages, 1, _i(), _i(), _i(), 1, _ref(q), _f(), None)

    assert tree((2**31 - 1024) // 8 + 1, 8) == UNS and tree(2**31 // 128 - 1, 128) == UNS


def test_binding_names_what_it_refuses():
    q, n = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    pages, table = torch.zeros(3, 1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors are needed, not cpu"):
        fd.fd_prompt_attention(q, q, q, n)
    with pytest.raises(ValueError, match="seq_lens must be a contiguous int32 tensor"):
        fd.fd_prompt_attention(q, q, q, n.float())
    with pytest.raises(ValueError, match=r"q must be \[T, Hq, D\]"):
        fd.fd_prompt_attention(q[0], q, q, n)
    with pytest.raises(ValueError, match=r"block_table must be \[B, pages_per_seq\]"):
        fd.fd_pages_reserve(n, n, n, 16)
    with pytest.raises(ValueError, match="page_size is out of range"):
        fd.fd_pages_reserve(n, table, n, 2**31)
    with pytest.raises(ValueError, match="tree_mask must be a contiguous int32 tensor"):
        fd.fd_tree_attention_paged(q, pages, pages, table, n, n, torch.zeros(3, 1, dtype=torch.int32))
    with pytest.raises(TypeError, match="v must be a tensor"):
        fd.fd_prompt_attention(q, q, None, n)
    with pytest.raises(TypeError):
        fd.fd_pages_reserve(n, table, n, 1.5)
    with pytest.raises(TypeError):
        fd.fd_pages_append_fp8(q, q, pages, pages, "1", 1.0, table, n, n)
