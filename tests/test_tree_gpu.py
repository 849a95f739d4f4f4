"""GPU parity of fd_tree_attention and fd_tree_attention_paged against the 64-bit reference, within
the bounds that serving_ref derives. Cache rows behind a request's last draft hold NaN."""

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _fd():
    import split_kv_decode_flashdecoding_b200 as fd
    return fd


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Requests with prefix[b] cached keys and new[b] drafts, contiguous (page 0) or paged."""

    def __init__(self, prefix, new, hq, hkv, d, page=0, seed=1, words=None, see=None, pad=0, extra=3, fill=0):
        gen, host = torch.Generator(device="cuda").manual_seed(seed), torch.Generator().manual_seed(seed)
        self.prefix, self.new, self.page, self.t = prefix, new, page, sum(new)
        self.see = see or [ref.random_tree(host, n) for n in new]
        words = words or max(1, -(-max(new + [1]) // 32))
        self.mask = torch.cat([ref.mask_words(self.see, words, fill), torch.full((pad, words), -1, dtype=torch.int32)]).cuda()
        self.q = torch.randn((self.t + pad, hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        self.q[self.t:] = NAN
        total = [p + n for p, n in zip(prefix, new)]
        kv = [torch.randn((2, t, hkv, d), generator=gen, device="cuda").to(torch.bfloat16) for t in total]
        self.caches = [(x[0], x[1]) for x in kv]
        self.table = None
        if page:
            counts = [-(-t // page) for t in total]
            pages = sum(counts) + extra
            order = torch.randperm(pages, generator=host)
            self.k = torch.full((pages, hkv, page, d), NAN, dtype=torch.bfloat16, device="cuda")
            self.v = self.k.clone()
            table = torch.full((len(new), max(counts + [1]) + 2), -1, dtype=torch.int32)
            at = 0
            for b, (x, n) in enumerate(zip(kv, counts)):
                ids = order[at:at + n]
                at += n
                table[b, :n] = ids.to(torch.int32)
                for pool, y in ((self.k, x[0]), (self.v, x[1])):
                    full = torch.full((n * page, hkv, d), NAN, dtype=torch.bfloat16, device="cuda")
                    full[:y.shape[0]] = y
                    pool[ids.cuda()] = full.view(n, page, hkv, d).transpose(1, 2)
            self.table = table.cuda()
        else:
            cap = max(total + [1]) + extra
            self.k = torch.full((len(new), hkv, cap, d), NAN, dtype=torch.bfloat16, device="cuda")
            self.v = self.k.clone()
            for b, x in enumerate(kv):
                self.k[b, :, :total[b]], self.v[b, :, :total[b]] = x[0].transpose(0, 1), x[1].transpose(0, 1)

    def run(self, **kw):
        fd = _fd()
        if self.table is None:
            return fd.fd_tree_attention(self.q, self.k, self.v, _i32(self.prefix), _i32(self.new), self.mask, **kw)
        return fd.fd_tree_attention_paged(self.q, self.k, self.v, self.table, _i32(self.prefix), _i32(self.new), self.mask, **kw)

    def want(self):
        return ref.tree(self.q[:self.t], self.caches, self.prefix, self.new, self.see)

    def check(self, flags=0):
        fd = _fd()
        n, hq, d = self.q.shape
        out = torch.full((n + 2, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n + 2, hq), 7.0, device="cuda")
        self.run(out=out[1:-1], lse=lse[1:-1])
        torch.cuda.synchronize()
        assert fd.fd_poll_status() == flags
        for x in (out, lse):
            assert bool((x[0] == 7.0).all()) and bool((x[1 + self.t:] == 7.0).all())
        ref.check_rows(out[1:1 + self.t], lse[1:1 + self.t], self.want(), str((self.prefix, self.new)))
        return out[1:1 + self.t], lse[1:1 + self.t]


@pytest.mark.parametrize("page", [0, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (6, 2, 64)])
def test_prefixes_and_pages(page, hq, hkv, d):
    Case([0, 1, 127, 128, 300, 1000], [3, 1, 2, 5, 17, 9], hq, hkv, d, page, seed=2).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (7, 1), (9, 1), (16, 1), (4, 4), (24, 3), (64, 8)])
def test_groups(hq, hkv):
    Case([70, 333], [20, 9], hq, hkv, 128, 16, seed=3).check()
    Case([70, 333], [20, 9], hq, hkv, 64, 0, seed=3).check()


@pytest.mark.parametrize("new,words", [([1], 1), ([32], 1), ([33], 2), ([64, 1, 40], 2), ([100], 8), ([255, 3], 8), ([256], 8)])
@pytest.mark.parametrize("prefix", [0, 90, 128])
def test_tree_sizes(new, words, prefix):
    Case([prefix] * len(new), new, 8, 2, 128, 16 if prefix else 0, seed=4, words=words).check()
    Case([prefix] * len(new), new, 2, 2, 64, 0, seed=4, words=words).check()


def test_long_prefixes():
    Case([9000, 5, 4097], [8, 8, 8], 16, 2, 128, 16, seed=5).check()
    Case([20000], [4], 8, 1, 128, 0, seed=5).check()
    Case([5000, 2500], [60, 64], 32, 4, 64, 128, seed=5).check()


def test_rows_that_see_nothing():
    none = [torch.zeros(5, 5, dtype=torch.bool), torch.zeros(3, 3, dtype=torch.bool)]
    none[0][2, 1] = True
    Case([0, 10], [5, 3], 8, 2, 128, 0, seed=6, see=none).check()
    Case([0, 10], [5, 3], 8, 2, 64, 16, seed=6, see=none).check()


def test_a_mask_may_show_any_draft():
    gen = torch.Generator().manual_seed(7)
    see = [torch.rand(n, n, generator=gen) < 0.5 for n in (40, 7)]
    Case([200, 0], [40, 7], 8, 2, 128, 32, seed=7, see=see).check()


def test_bits_behind_the_tree_are_ignored():
    Case([30, 5], [6, 33], 4, 2, 128, 16, seed=8, words=3, fill=1).check()


def test_padded_batch_and_empty_requests():
    Case([30, 5, 0, 64], [6, 0, 0, 2], 4, 2, 128, 16, seed=9, pad=5).check()


def test_one_draft_is_a_decode_step():
    fd = _fd()
    c = Case([511, 0, 63], [1, 1, 1], 16, 2, 128, 64, seed=10, see=[torch.ones(1, 1, dtype=torch.bool)] * 3)
    out, lse = c.check()
    o, l = fd.fd_decode_attention_paged(c.q, c.k, c.v, c.table, _i32([512, 1, 64]))
    tol = c.want()
    assert bool(((out.double() - o.double()).abs() <= 2 * tol.out_tol).all())
    assert bool(((lse.double() - l.double()).abs() <= 2 * tol.lse_tol).all())


def test_strided_cache_and_queries():
    c = Case([100, 260], [7, 3], 8, 2, 128, 16, seed=11)
    want = c.run()
    wide = torch.zeros((c.k.shape[0], 5, c.page, 128), dtype=torch.bfloat16, device="cuda")
    wide2 = wide.clone()
    wide[:, 1:5:2], wide2[:, 1:5:2] = c.k, c.v
    c.k, c.v = wide[:, 1:5:2], wide2[:, 1:5:2]
    q = torch.zeros((c.q.shape[0], 9, 136), dtype=torch.bfloat16, device="cuda")
    q[:, :8, 8:] = c.q
    c.q = q[:, :8, 8:]
    assert all(torch.equal(a, b) for a, b in zip(want, c.run()))


def test_lengths_outside_their_range():
    fd = _fd()
    c = Case([50, 20], [6, 5], 4, 2, 128, 0, seed=12, extra=0)  # S_cap 56
    prefix = c.prefix
    c.prefix = [-3, 20]
    got = c.run()
    assert fd.fd_poll_status() == fd.FD_FLAG_LEN_CLAMPED
    caches = [(c.k[b].transpose(0, 1), c.v[b].transpose(0, 1)) for b in range(2)]
    ref.check_rows(*got, ref.tree(c.q, caches, [0, 20], c.new, c.see))
    c.prefix = [53, 20]  # three drafts of the first request stand behind the capacity
    got = c.run()
    assert fd.fd_poll_status() == fd.FD_FLAG_LEN_CLAMPED
    rows = [ref.attend(c.q[:6], caches[0][0], caches[0][1],
                       torch.cat([torch.ones(6, 53, dtype=torch.bool), c.see[0][:, :3]], 1).cuda()),
            ref.attend(c.q[6:], caches[1][0][:25], caches[1][1][:25],
                       torch.cat([torch.ones(5, 20, dtype=torch.bool), c.see[1]], 1).cuda())]
    ref.check_rows(*got, ref.Rows(*(torch.cat(x) for x in zip(*rows))))
    c.prefix = prefix
    for bad in ([6, 6], [-1, 5], [33, 0]):
        c.new = bad
        out, lse = torch.full_like(c.q, 3.0), torch.full(c.q.shape[:2], 3.0, device="cuda")
        c.run(out=out, lse=lse)
        assert fd.fd_poll_status() == fd.FD_FLAG_LEN_CLAMPED
        assert bool((out == 3.0).all()) and bool((lse == 3.0).all())


def test_entries_outside_the_pool_are_not_read():
    fd = _fd()
    c = Case([100, 40], [4, 4], 8, 2, 128, 16, seed=13)
    want = c.run()
    c.table[0, 2] = c.k.shape[0]
    got = c.run()
    assert fd.fd_poll_status() == fd.FD_FLAG_BAD_PAGE
    c.table[0, 2] = -5
    got2 = c.run()
    assert fd.fd_poll_status() == fd.FD_FLAG_BAD_PAGE
    for w, a, b in zip(want, got, got2):
        assert torch.equal(w[4:], a[4:]) and torch.equal(w[4:], b[4:])


def test_same_results_again_and_in_a_graph():
    fd = _fd()
    c = Case([3000, 100, 0], [16, 16, 3], 16, 2, 128, 16, seed=14)
    first, again = c.run(), c.run()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    s = torch.cuda.Stream()
    pre, new = _i32(c.prefix), _i32(c.new)
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cap = c.table.shape[1] * c.page
        fd.fd_reserve_workspace(fd.fd_tree_workspace_bytes(3, c.t, 16, 2, cap, 128), stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fd.fd_tree_attention_paged(c.q, c.k, c.v, c.table, pre, new, c.mask, out=out, lse=lse)
    torch.cuda.synchronize()
    for _ in range(3):
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    new.copy_(_i32([16, 0, 2]))
    out.fill_(9.0)
    g.replay()
    torch.cuda.synchronize()
    assert bool((out[18:] == 9.0).all())
    # other lengths may cut the first request's keys elsewhere: the bounds hold, not every bit
    ref.check_rows(out[:16], lse[:16], ref.tree(c.q[:16], c.caches[:1], c.prefix[:1], [16], c.see[:1]))
    assert fd.fd_poll_status(stream=s) == 0


# enough tokens and heads for items of two row tiles (more tokens than a tile a request, an item a
# multiprocessor), next to requests of one tile and of none, with cuts inside the drafts
@pytest.mark.parametrize("hq,hkv,new", [(64, 8, [64, 33, 1, 0, 64, 48, 64, 17, 64, 50]), (40, 40, [256, 129, 1, 128, 255]),
                                        (96, 48, [65, 128, 200, 0, 64])])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 128), (128, 0), (64, 0)])
def test_two_row_tiles(hq, hkv, new, d, page):
    prefix = [(977 * i + 300) % 2000 for i in range(len(new))]
    Case(prefix, new, hq, hkv, d, page=page, seed=12, pad=3).check()
