"""Rows of the block table in which something stands behind the first negative entry: the page
operators ignore it, also once a later reserve has filled the gap in front of it."""

import pytest
import torch

import serving_ref as ref
from test_pages_gpu import Both, _fd, _i32

pytestmark = pytest.mark.gpu


class Rows(Both):
    """The state of Both, with `behind` in every column of every row; compared by the rows' pages."""

    def __init__(self, *args, behind=0, **kw):
        super().__init__(*args, **kw)
        self.table[:, 1:] = behind
        self.host.table = [[-1] + [behind] * (len(r) - 1) for r in self.host.table]

    def reserve(self, want):
        have = [len(self.host.pages(b)) for b in range(len(want))]
        _fd().fd_pages_reserve(self.refs, self.table, _i32(want), self.size)
        for b, n in enumerate(want):  # the sequence ends behind its new pages
            row, pages = self.host.table[b], -(-n // self.size)
            if pages > have[b] and pages < len(row):
                row[pages] = -1
        return self.host.reserve(want)

    def pages(self):
        return [self.host.pages(b) for b in range(len(self.host.table))]

    def same(self, flags=0, what=""):
        assert _fd().fd_poll_status() == flags, what
        rows = []
        for row in self.table.tolist():
            n = next((c for c, p in enumerate(row) if p < 0), len(row))
            rows.append(row[:n])
        assert rows == self.pages(), what
        assert self.refs.tolist() == self.host.refs, what
        assert self.lens.tolist() == self.host.lens, what
        assert torch.equal(self.k.cpu(), self.host.k) and torch.equal(self.v.cpu(), self.host.v), what


def test_reserve_ends_the_row():
    fd = _fd()
    refs, table = _i32([1, 0, 0, 1, 0, 0, 0, 1]), _i32([[3, -1, 7, 7], [-1, 0, 0, 0], [-1, 7, 7, 7], [-1, 7, 7, 7]])
    fd.fd_pages_reserve(refs, table, _i32([16, 9, 0, 32]), 8)  # pages of 8: one more, two, none, four (too many)
    assert fd.fd_poll_status() == fd.FD_FLAG_POOL_FULL
    assert table[0].tolist() == [3, 1, -1, 7]
    assert table[1, :3].tolist() == [2, 4, -1]
    assert table[2].tolist() == [-1, 7, 7, 7] and table[3, 0] == -1
    assert refs.tolist() == [1, 1, 1, 1, 1, 0, 0, 1]


@pytest.mark.parametrize("seqs", [6, 70])  # a warp a row, and four rows a warp
@pytest.mark.parametrize("behind", [0, 5, 1 << 20])
def test_a_run_over_such_rows(seqs, behind):
    s = Rows(400, 2, 8, 64, seqs, 9, behind=behind)
    g = torch.Generator().manual_seed(seqs)
    lens = [0] * seqs
    first = torch.randint(0, 33, (seqs,), generator=g).tolist()
    first[2:5] = [0, 0, 0]
    first[0], first[1] = 16, 21  # full pages only, and a partly filled one
    assert s.reserve(first)
    s.append([0] * seqs, first)
    s.set_lens(first)
    s.same()
    s.fork([0, 1], [2, 3])
    s.same()
    lens = list(s.host.lens)
    assert s.reserve([n + 9 if n else 0 for n in lens])
    s.same()
    s.compact([n // 2 for n in lens], [[0] if n else None for n in lens])
    s.same()
    s.free([0, 2, 3, 5])
    s.same()
    assert s.reserve([17] * seqs)
    s.same()
    s.free(list(range(seqs)))
    s.same()
    assert not s.refs.any()
