"""Page operators that write cache_lens, directly followed by a decode call on the same stream: the
decode call has to see the lengths, tables and rows that the operator leaves. Nothing here waits for
the GPU between the two. Sequences shrink or grow by a large factor, so a plan from older lengths
would differ in every sequence."""

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

HQ, HKV, D, SIZE, PAGES, COLUMNS = 16, 2, 128, 16, 2600, 160


def _fd():
    import split_kv_decode_flashdecoding_b200 as fd
    return fd


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """`full` sequences of up to 2400 tokens, then as many empty ones; one page operator and one decode."""

    def __init__(self, op, fp8, full=16):
        fd = _fd()
        gen = torch.Generator(device="cuda").manual_seed(77)
        self.op, self.fp8, self.n = op, fp8, 2 * full
        lens = [2400 - 97 * i for i in range(full)] + [0] * full
        x = torch.randn((2, PAGES, HKV, SIZE, D), generator=gen, device="cuda")
        self.k, self.v = (y.to(torch.float8_e4m3fn) if fp8 else y.to(torch.bfloat16) for y in x)
        self.q = torch.randn((self.n, HQ, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.refs, self.lens = torch.zeros(PAGES, dtype=torch.int32, device="cuda"), _i32(lens)
        self.table = torch.full((self.n, COLUMNS), -1, dtype=torch.int32, device="cuda")
        fd.fd_pages_reserve(self.refs, self.table, self.lens, SIZE)
        self.state = [self.k, self.v, self.refs, self.table, self.lens]
        self.start = [x.clone() for x in self.state]
        # what compact keeps: the first sequence's last tokens, 1 to a few of the next ones, all of some
        kept = [3, 1, 2303 - 97, 40] + [(53 * i) % 1300 for i in range(full - 4)] + [-1] * full
        keep = torch.zeros((self.n, 2400), dtype=torch.int32)
        for b, m in enumerate(kept):
            if m > 0:
                keep[b, :m] = torch.arange(lens[b] - m, lens[b], dtype=torch.int32)
        self.keep, self.kept, self.zero = keep.cuda(), _i32(kept), torch.zeros(self.n, dtype=torch.int32, device="cuda")
        self.src, self.dst = _i32(list(range(full))), _i32(list(range(self.n - 1, full - 1, -1)))
        self.gone = _i32(list(range(0, full, 2)))
        self.one = _i32([1] * full + [0] * full)
        self.new = torch.randn((2, full, HKV, D), generator=gen, device="cuda").to(torch.bfloat16)

    def restore(self):
        for x, y in zip(self.state, self.start):
            x.copy_(y)

    def operate(self):
        fd = _fd()
        if "compact" in self.op:
            fd.fd_pages_compact(self.k, self.v, self.refs, self.table, self.lens, self.zero, self.keep, self.kept)
        if "free" in self.op:
            fd.fd_pages_free(self.refs, self.table, self.lens, self.gone)
        if "fork" in self.op:
            fd.fd_pages_fork(self.k, self.v, self.refs, self.table, self.lens, self.src, self.dst)
        if "reserve" in self.op:  # behind the writer, and itself a kernel that lets the next one start early
            fd.fd_pages_reserve(self.refs, self.table, self.one, SIZE)
        if "append" in self.op:   # likewise; position 0 of every sequence that has a page
            if self.fp8:
                fd.fd_pages_append_fp8(self.new[0], self.new[1], self.k, self.v, 1.0, 1.0, self.table, self.zero, self.one)
            else:
                fd.fd_pages_append(self.new[0], self.new[1], self.k, self.v, self.table, self.zero, self.one)

    def decode(self, out=None, lse=None):
        fd = _fd()
        if self.fp8:
            return fd.fd_decode_attention_paged_fp8(self.q, self.k, self.v, 1.0, 1.0, self.table, self.lens, out=out, lse=lse)
        return fd.fd_decode_attention_paged(self.q, self.k, self.v, self.table, self.lens, out=out, lse=lse)

    def slowly(self):
        """The same step with the host waiting in between, and its result checked where q is exact."""
        self.restore()
        torch.cuda.synchronize()
        self.operate()
        torch.cuda.synchronize()
        out, lse = self.decode()
        torch.cuda.synchronize()
        if not self.fp8:
            for b, n in enumerate(self.lens.tolist()):
                ids = self.table[b, :-(-n // SIZE)].long()
                k, v = (x[ids].transpose(1, 2).reshape(-1, HKV, D)[:n] for x in (self.k, self.v))
                see = torch.ones((1, n), dtype=torch.bool, device="cuda")
                ref.check_rows(out[b:b + 1], lse[b:b + 1], ref.attend(self.q[b:b + 1], k, v, see), f"sequence {b}")
        return out, lse


OPS = ["compact", "free", "fork", "compact fork", "free fork", "compact reserve append", "free reserve append"]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("op", OPS)
def test_decode_behind_a_page_operator(op, fp8):
    fd = _fd()
    s = Step(op, fp8)
    want = s.slowly()
    got = [(torch.empty_like(want[0]), torch.empty_like(want[1])) for _ in range(40)]
    for out, lse in got:
        s.restore()
        s.operate()
        s.decode(out, lse)
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), f"pass {i}"
    assert fd.fd_poll_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("op", OPS)
def test_decode_behind_a_page_operator_in_a_graph(op, fp8):
    fd = _fd()
    s = Step(op, fp8)
    want = s.slowly()
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        need = fd.fd_decode_workspace_bytes(s.n, HQ, HKV, COLUMNS * SIZE, D, 0, fd.fd_decode_num_ctas(0, torch.bfloat16, HQ // HKV, D))
        fd.fd_reserve_workspace(need, stream=st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            s.restore()
            s.operate()
            s.decode(out, lse)
    torch.cuda.synchronize()
    for i in range(40):
        out.fill_(9.0), lse.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), f"replay {i}"
    assert fd.fd_poll_status(stream=st) == 0
