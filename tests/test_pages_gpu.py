"""The page operators on the GPU against their definitions on the host (serving_ref.Pool): every
table entry, reference, length and byte of the pools is compared."""

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


def _fd():
    import split_kv_decode_flashdecoding_b200 as fd
    return fd


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """The same state on the GPU and in the reference."""

    def __init__(self, pages, hkv, size, d, seqs, columns, dtype=torch.bfloat16, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn((2, pages, hkv, size, d), generator=gen, device="cuda")
        x = x.to(dtype) if dtype != torch.uint8 else (x * 40).to(torch.float8_e4m3fn).view(torch.uint8)
        self.k, self.v = x[0].clone(), x[1].clone()
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((seqs, columns), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.host = ref.Pool(self.k, self.v, [0] * pages, [[-1] * columns for _ in range(seqs)], [0] * seqs)
        self.size, self.gen = size, gen

    def same(self, flags=0, what=""):
        fd = _fd()
        assert fd.fd_poll_status() == flags, what
        h = self.host
        assert self.table.tolist() == h.table, what
        assert self.refs.tolist() == h.refs, what
        assert self.lens.tolist() == h.lens, what
        assert torch.equal(self.k.cpu(), h.k) and torch.equal(self.v.cpu(), h.v), what

    def set_lens(self, lens):
        self.lens.copy_(_i32(lens))
        self.host.lens = list(lens)

    def reserve(self, want):
        _fd().fd_pages_reserve(self.refs, self.table, _i32(want), self.size)
        return self.host.reserve(want)

    def append(self, start, new, pad=0):
        t, (_, hkv, _, d) = sum(max(n, 0) for n in new) + pad, self.k.shape
        x = torch.randn((2, t, hkv, d), generator=self.gen, device="cuda").to(self.k.dtype)
        _fd().fd_pages_append(x[0], x[1], self.k, self.v, self.table, _i32(start), _i32(new))
        self.host.append(x[0].cpu(), x[1].cpu(), start, new)

    def fork(self, src, dst):
        _fd().fd_pages_fork(self.k, self.v, self.refs, self.table, self.lens, _i32(src), _i32(dst))
        self.host.fork(src, dst)

    def free(self, seqs):
        _fd().fd_pages_free(self.refs, self.table, self.lens, _i32(seqs))
        self.host.free(seqs)

    def compact(self, start, keep):
        m = [-1 if x is None else len(x) for x in keep]
        rows = [(x or []) + [0] * (max(m + [1]) - len(x or [])) for x in keep]
        _fd().fd_pages_compact(self.k, self.v, self.refs, self.table, self.lens, _i32(start), _i32(rows), _i32(m))
        self.host.compact(start, rows, m)


@pytest.mark.parametrize("size", [8, 16, 64, 128, 384])
@pytest.mark.parametrize("hkv,d,dtype", [(1, 64, torch.bfloat16), (3, 128, torch.bfloat16), (2, 64, torch.float32), (2, 128, torch.float32)])
def test_append(size, hkv, d, dtype):
    s = Both(40, hkv, size, d, 5, 12, dtype)
    want = [size, 1, 0, 3 * size + 2, 2 * size]
    s.reserve(want)
    s.append([0, 0, 0, 1, size - 1], [size, 1, 0, 3 * size + 1, size + 1], pad=3)
    s.same()


def test_append_of_many_rows_and_sequences():
    s = Both(3000, 2, 16, 128, 1200, 4)
    lens = [(7 * i) % 33 for i in range(1200)]
    s.reserve(lens)
    s.append([0] * 1200, lens)
    s.same()
    s.append([max(n - 1, 0) for n in lens], [min(n, 1) for n in lens])
    s.same()


def test_append_takes_slices_of_a_fused_projection():
    fd = _fd()
    s = Both(10, 2, 16, 64, 2, 4)
    s.reserve([30, 5])
    x = torch.randn((35, 7, 64), generator=s.gen, device="cuda").to(torch.bfloat16)
    fd.fd_pages_append(x[:, 3:5], x[:, 5:7], s.k, s.v, s.table, _i32([0, 0]), _i32([30, 5]))
    s.host.append(x[:, 3:5].cpu(), x[:, 5:7].cpu(), [0, 0], [30, 5])
    s.same()


def test_append_skips_what_has_no_place():
    fd = _fd()
    s = Both(10, 2, 16, 64, 3, 2)
    s.reserve([16, 20, 32])
    s.append([10, -1, 30], [10, 2, 4])  # past the pages, a negative start, past the row
    s.same(fd.FD_FLAG_BAD_PAGE | fd.FD_FLAG_LEN_CLAMPED)
    s.append([0, 0, 0], [2, -3, 1])     # a negative count is none
    s.same()
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    fd.fd_pages_append(x, x, s.k, s.v, s.table, _i32([0, 0, 0]), _i32([2, 1, 1]))
    s.same(fd.FD_FLAG_LEN_CLAMPED, "more rows than there are: nothing is written")


@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_append_fp8(src, d):
    fd = _fd()
    for scale in (1.0, 0.37, 1e-3, 1e-38, 1e-40, 1e30):
        s = Both(20, 2, 32, d, 3, 8, torch.uint8)
        s.reserve([40, 3, 64])
        x = torch.randn((2, 107, 2, d), generator=s.gen, device="cuda") * 100
        x[0, :5, 0, :8] = torch.tensor([0.0, -0.0, 448.0, 449.0, -1e9, float("inf"), float("-inf"), 2.0 ** -10], device="cuda")
        x[1, 7, 1, 3] = float("nan")
        x = x.to(src)
        ks, vs = scale, 2 * scale
        fd.fd_pages_append_fp8(x[0], x[1], s.k, s.v, ks, vs, s.table, _i32([0, 0, 0]), _i32([40, 3, 64]))
        codes = []
        for y, z in ((x[0], ks), (x[1], vs)):
            q = (y.float() / torch.tensor(z, dtype=torch.float32, device="cuda")).clamp(-448, 448)
            codes.append(q.to(torch.float8_e4m3fn).view(torch.uint8).cpu())
        s.host.append(codes[0], codes[1], [0, 0, 0], [40, 3, 64])
        s.same(what=str(scale))
        s.k, s.v = s.k.view(torch.float8_e4m3fn), s.v.view(torch.float8_e4m3fn)
        fd.fd_pages_append_fp8(x[0], x[1], s.k, s.v, ks, vs, s.table, _i32([0, 0, 0]), _i32([40, 3, 64]))


@pytest.mark.parametrize("pages", [1, 7, 100, 20000, 70001])
def test_reserve(pages):
    s = Both(pages, 1, 8, 64, 40, 30)
    g = torch.Generator().manual_seed(pages)
    for r in range(4):
        want = torch.randint(-5, 260, (40,), generator=g).tolist()
        want = [min(w, max(1, pages // 4)) for w in want] if r < 2 else want
        ok = s.reserve(want)
        flags = (0 if ok else _fd().FD_FLAG_POOL_FULL) | (_fd().FD_FLAG_LEN_CLAMPED if max(want) > 240 else 0)
        s.same(flags, f"round {r}")
        s.free([3, 17, r])
        s.same()


def test_reserve_when_references_are_not_16_byte_aligned():
    fd = _fd()
    big = torch.zeros(50, dtype=torch.int32, device="cuda")
    big[3:9] = 1
    table = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    fd.fd_pages_reserve(big[3:], table, _i32([33, 8]), 8)
    assert table[0, :5].tolist() == [6, 7, 8, 9, 10] and table[1, 0] == 11 and int(big.sum()) == 12
    assert bool((big[:3] == 0).all())


def test_reserve_that_runs_out_serves_the_first_sequences():
    fd = _fd()
    s = Both(6, 1, 8, 64, 4, 8)
    assert not s.reserve([16, 40, 8, 0])
    s.same(fd.FD_FLAG_POOL_FULL)
    assert s.table[0, :3].tolist() == [0, 1, -1] and bool((s.table[1:] == -1).all())


@pytest.mark.parametrize("size,hkv,d,dtype", [(16, 2, 128, torch.bfloat16), (128, 1, 64, torch.float32), (8, 3, 64, torch.uint8)])
def test_fork_and_free(size, hkv, d, dtype):
    s = Both(120, hkv, size, d, 12, 9, dtype)
    lens = [3 * size, 2 * size + 3, 1, 0]
    s.reserve(lens + [0] * 8)
    s.set_lens(lens + [0] * 8)
    s.fork([0, 1, 1, 2, 3], [4, 5, 6, 7, 8])
    s.same()
    s.reserve([n + 1 for n in s.host.lens])
    s.same()
    s.fork([5, 4], [9, 10])  # the reserve gave 9 and 10 a page: they are not empty
    s.same(_fd().FD_FLAG_BAD_INDEX)
    s.free([9, 10])
    s.fork([5, 4], [9, 10])  # forks of forks; 4's reserved page is not shared
    s.same()
    s.free([1, 4, 5])
    s.same()
    s.free([0, 6, 7, 8, 9, 10, 2, 3, 11])
    s.same()
    assert int(s.refs.sum()) == 0


def test_fork_refuses():
    fd = _fd()
    s = Both(20, 2, 8, 64, 6, 4)
    s.reserve([20, 8, 0, 0, 0, 0])
    s.set_lens([20, 8, 0, 0, 0, 0])
    s.fork([0, 0, 9, 0, -1, 0], [2, 2, 3, 1, 3, 6])  # twice the same, no such source, a full row, ...
    s.same(fd.FD_FLAG_BAD_INDEX)
    s.set_lens([25, 8, 20, 0, 0, 0])                  # more tokens than pages
    s.fork([0], [4])
    s.same(fd.FD_FLAG_BAD_PAGE)
    s.set_lens([20, 8, 20, 0, 0, 0])
    s.table[1, 0] = 20
    s.host.table[1][0] = 20
    s.fork([1, 0], [4, 5])
    s.same(fd.FD_FLAG_BAD_PAGE)
    assert s.host.lens == [20, 8, 20, 0, 0, 20]
    s.table[1, 0] = -2                                # any negative entry is none
    s.host.table[1][0] = -2
    s.fork([1], [4])
    s.same(fd.FD_FLAG_BAD_PAGE)


def test_fork_when_pages_run_out():
    fd = _fd()
    s = Both(5, 1, 8, 64, 6, 4)
    s.reserve([12, 8, 0, 0, 0, 0])
    s.set_lens([12, 8, 0, 0, 0, 0])
    s.fork([0, 0, 1, 0], [2, 3, 4, 5])  # two pages are left: the last pair gets none
    s.same(fd.FD_FLAG_POOL_FULL)
    assert s.host.lens == [12, 8, 12, 12, 8, 0]


def test_free_of_repeated_and_wrong_indices():
    fd = _fd()
    s = Both(30, 1, 8, 64, 300, 2)
    s.reserve([8, 16] + [0] * 298)
    s.set_lens([8, 16] + [0] * 298)
    s.free([1, 1, 1, 0, 1])
    s.same()
    s.reserve([8, 16] + [0] * 298)
    s.free([-1, 300, 1] + [5] * 200 + [1])
    s.same(fd.FD_FLAG_BAD_INDEX)
    s.table[0, 0], s.host.table[0][0] = 99, 99
    s.free([0])
    s.same(fd.FD_FLAG_BAD_PAGE)


@pytest.mark.parametrize("size,hkv,d,dtype", [(16, 2, 128, torch.bfloat16), (8, 1, 64, torch.uint8), (128, 2, 128, torch.float32)])
def test_compact(size, hkv, d, dtype):
    s = Both(300, hkv, size, d, 7, 40, dtype)
    start, new = [0, 5, 100, 33, 0, 7, 20], [64, 64, 17, 1, 200, 0, 8]
    s.reserve([a + n for a, n in zip(start, new)])
    s.set_lens(start)
    if dtype != torch.uint8:
        s.append(start, new)
    g = torch.Generator().manual_seed(5)
    pick = lambda n, m: torch.randperm(n, generator=g)[:m].sort().values.tolist()  # noqa: E731
    s.compact(start, [pick(64, 31), [63], list(range(17)), [], pick(200, 150), [], None])
    s.same()
    s.compact([0] * 7, [[], None, [1, 2, 3], pick(33, 20), pick(150, 149), None, None])
    s.same()


def test_compact_of_a_long_list():
    s = Both(700, 2, 16, 128, 3, 320)
    s.reserve([5000, 10, 4096])
    s.append([0, 0, 0], [5000, 10, 4096])
    g = torch.Generator().manual_seed(6)
    keep = [torch.randperm(5000, generator=g)[:3333].sort().values.tolist(), [9], list(range(1, 4096))]
    s.compact([0, 0, 0], keep)
    s.same()


@pytest.mark.parametrize("shift", [1, 127, 128, 129, 500])
def test_compact_that_closes_one_gap(shift):
    # every row moves by the same distance, below, at and above the rows that move together
    s = Both(300, 1, 16, 128, 2, 260)
    n = 1500
    s.reserve([n + shift, 0])
    s.append([0, 0], [n + shift, 0])
    s.compact([0, 0], [list(range(shift, n + shift)), None])
    s.same()


def test_compact_refuses():
    fd = _fd()
    s = Both(40, 1, 8, 64, 4, 4)
    s.reserve([30, 30, 30, 30])
    s.set_lens([30, 30, 30, 30])
    s.append([0] * 4, [30] * 4)
    s.compact([0, 0, -1, 0], [[3, 3], [4, 2], [1], [5, 6]])   # not increasing twice, a negative start
    s.same(fd.FD_FLAG_BAD_INDEX)
    s.compact([0, 28, 0, 0], [[-1, 2], [4], [32], [1, 2]])    # below 0, past the row twice
    s.same(fd.FD_FLAG_BAD_INDEX)
    s.reserve([0] * 4)
    s.free([3])
    s.fork([0], [3])
    s.same()
    s.compact([0, 0, 24, 26], [[1], None, None, [1]])         # a shared page; the fork's own last page
    s.same(fd.FD_FLAG_BAD_PAGE)
    assert s.host.lens[3] == 27
    s.compact([0, 0, 0, 0], [None, [25], None, None])
    s.same()
    s.compact([0, 0, 0, 0], [None, [9], None, None])          # no page there any more
    s.same(fd.FD_FLAG_BAD_PAGE)


def test_a_step_in_a_graph():
    fd = _fd()
    s = Both(64, 2, 16, 128, 4, 8)
    s.reserve([20, 5, 33, 0])
    s.set_lens([20, 5, 33, 0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want, start, new = _i32([24, 9, 37, 0]), _i32([20, 5, 33, 0]), _i32([4, 4, 4, 0])
    keep, kept = _i32([[1, 3], [0, 2], [3, 0], [0, 0]]), _i32([2, 2, 1, 0])
    x = torch.randn((2, 12, 2, 128), generator=s.gen, device="cuda").to(torch.bfloat16)
    with torch.cuda.stream(st):
        fd.fd_reserve_workspace(1 << 16, stream=st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            fd.fd_pages_reserve(s.refs, s.table, want, 16)
            fd.fd_pages_append(x[0], x[1], s.k, s.v, s.table, start, new)
            fd.fd_pages_compact(s.k, s.v, s.refs, s.table, s.lens, start, keep, kept)
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
        s.host.reserve([24, 9, 37, 0])
        s.host.append(x[0].cpu(), x[1].cpu(), [20, 5, 33, 0], [4, 4, 4, 0])
        s.host.compact([20, 5, 33, 0], [[1, 3], [0, 2], [3, 0], [0, 0]], [2, 2, 1, 0])
        torch.cuda.synchronize()
        s.same()
    assert fd.fd_poll_status(stream=st) == 0
