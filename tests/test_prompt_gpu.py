"""GPU parity of fd_prompt_attention against the 64-bit reference, within the bounds that
serving_ref derives."""

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _fd():
    import split_kv_decode_flashdecoding_b200 as fd
    return fd


def _inputs(lens, hq, hkv, d, seed, pad=0, fused=False):
    """q, k, v on the GPU; `pad` rows of NaN behind the last request; fused: slices of one tensor."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = sum(lens) + pad
    x = torch.randn((t, hq + 2 * hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
    x[sum(lens):] = NAN
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _check(lens, hq, hkv, d, seed=1, pad=0, fused=False, scale=1.0):
    fd = _fd()
    q, k, v = _inputs(lens, hq, hkv, d, seed, pad, fused)
    q = q * scale if not fused else q
    t = sum(lens)
    out = torch.full((t + pad + 2, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((t + pad + 2, hq), 7.0, device="cuda")
    fd.fd_prompt_attention(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           out=out[1:-1], lse=lse[1:-1])
    torch.cuda.synchronize()
    assert fd.fd_poll_status() == 0
    for x in (out, lse):  # nothing written around the requests' rows
        assert bool((x[0] == 7.0).all()) and bool((x[1 + t:] == 7.0).all())
    if t:
        ref.check_rows(out[1:1 + t], lse[1:1 + t], ref.prompt(q[:t], k[:t], v[:t], lens), str((lens, hq, hkv, d)))
    return out[1:1 + t], lse[1:1 + t]


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255, 1, 256, 257], [0, 0, 3, 0], [31, 32, 33, 0, 1000], [640]])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 4, 64), (64, 8, 128)])
def test_lengths(lens, hq, hkv, d):
    _check(lens, hq, hkv, d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (6, 2), (7, 1), (9, 1), (16, 1), (12, 1), (40, 40), (22, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_groups(hq, hkv, d):
    _check([70, 200, 9], hq, hkv, d, seed=2)


@pytest.mark.parametrize("pad", [1, 300])
def test_padded_batch_leaves_the_rest(pad):
    _check([100, 28, 131], 16, 2, 128, seed=3, pad=pad)


def test_slices_of_a_fused_projection():
    _check([150, 301], 8, 2, 128, seed=4, fused=True)
    _check([150, 301], 8, 2, 64, seed=4, fused=True)


@pytest.mark.parametrize("scale", [0.0, 8.0, 60.0])
def test_flat_and_peaked_scores(scale):
    _check([300, 77], 8, 2, 128, seed=5, scale=scale)


def test_many_requests():
    lens = [(37 * i) % 23 for i in range(600)]
    _check(lens, 4, 2, 64, seed=6)
    _check([1] * 4096, 2, 1, 64, seed=6)


def test_long():
    _check([5000, 3, 2100], 8, 1, 128, seed=7)
    _check([4099], 2, 2, 64, seed=7)


def test_another_requests_non_finite_values_stay_there():
    fd = _fd()
    lens = [100, 50, 200]
    q, k, v = _inputs(lens, 8, 2, 128, 8)
    good = fd.fd_prompt_attention(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for x in (k, v):
        x[100:125], x[125:150] = NAN, float("inf")
    bad = fd.fd_prompt_attention(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for a, b in zip(good, bad):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[150:], b[150:])


def test_a_keys_non_finite_scores_reach_only_the_rows_that_see_it():
    fd = _fd()
    q, k, v = _inputs([300], 8, 2, 128, 9)
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    good = fd.fd_prompt_attention(q, k, v, lens)
    for value in (NAN, float("inf"), float("-inf")):
        k[200] = value
        bad = fd.fd_prompt_attention(q, k, v, lens)
        for a, b in zip(good, bad):
            assert torch.equal(a[:200], b[:200])
            if value != value:
                assert bool(b[200:].isnan().all())
    k[200, :, 1:], k[200, :, 0] = 0.0, float("inf")  # scores of +inf or -inf by the sign of q's first element
    bad = fd.fd_prompt_attention(q, k, v, lens)
    up = q[200:, :, 0] > 0
    assert bool(bad[0][200:][up].isnan().all()) and bool(bad[1][200:][up].isnan().all())
    assert bool(bad[0][200:][~up].isfinite().all()) and bool(bad[1][200:][~up].isfinite().all())


def test_bad_lengths():
    fd = _fd()
    q, k, v = _inputs([64], 4, 2, 64, 10)
    out = torch.full_like(q, 3.0)
    lse = torch.full((64, 4), 3.0, device="cuda")
    fd.fd_prompt_attention(q, k, v, torch.tensor([60, 5], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert fd.fd_poll_status() == fd.FD_FLAG_LEN_CLAMPED
    assert bool((out == 3.0).all()) and bool((lse == 3.0).all())
    fd.fd_prompt_attention(q, k, v, torch.tensor([30, -4, 34], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert fd.fd_poll_status() == fd.FD_FLAG_LEN_CLAMPED
    ref.check_rows(out, lse, ref.prompt(q, k, v, [30, 34]))


def test_same_results_again_and_in_a_graph():
    fd = _fd()
    lens = [700, 0, 45, 1333]
    q, k, v = _inputs(lens, 16, 2, 128, 11)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = fd.fd_prompt_attention(q, k, v, n)
    again = fd.fd_prompt_attention(q, k, v, n)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    s = torch.cuda.Stream()
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fd.fd_reserve_workspace(fd.fd_prompt_workspace_bytes(4, sum(lens), 16, 2, 128), stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fd.fd_prompt_attention(q, k, v, n, out=out, lse=lse)
    torch.cuda.synchronize()
    # a larger call on the same stream outgrows the workspace; the graph keeps its own
    fd.fd_reserve_workspace(64 << 20, stream=s)
    for new in ([700, 0, 45, 1333], [1, 2, 3, 4], [2078, 0, 0, 0], [0, 0, 0, 0]):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(9.0), lse.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        t = sum(new)
        assert bool((out[t:] == 9.0).all()) and bool((lse[t:] == 9.0).all())
        if t:
            ref.check_rows(out[:t], lse[:t], ref.prompt(q[:t], k[:t], v[:t], new))
    assert fd.fd_poll_status(stream=s) == 0


def test_on_another_stream_beside_the_current_one():
    fd = _fd()
    lens = [900, 300]
    q, k, v = _inputs(lens, 8, 8, 64, 12)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = fd.fd_prompt_attention(q, k, v, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [torch.empty_like(x) for x in want]
    for _ in range(5):
        fd.fd_prompt_attention(q, k, v, n, out=got[0], lse=got[1], stream=s)
        here = fd.fd_prompt_attention(q, k, v, n)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, here))


# enough tokens and heads for items of two row tiles, next to requests of one tile, of one token and of none
@pytest.mark.parametrize("hq,hkv,lens", [(40, 40, [1500, 0, 130, 257, 1]), (64, 8, [777, 16, 33, 0, 1025]), (96, 48, [64, 65, 129, 900])])
@pytest.mark.parametrize("d", [64, 128])
def test_two_row_tiles(hq, hkv, lens, d):
    _check(lens, hq, hkv, d, seed=13, pad=5)


@pytest.mark.parametrize("hq,hkv,d", [(40, 40, 128), (40, 40, 64), (64, 8, 128)])
def test_non_finite_values_in_two_row_tiles(hq, hkv, d):
    fd = _fd()
    lens = [500, 130, 300]
    q, k, v = _inputs(lens, hq, hkv, d, 14)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    good = fd.fd_prompt_attention(q, k, v, n)
    k[500:630], v[500:630] = NAN, float("inf")  # another request's
    bad = fd.fd_prompt_attention(q, k, v, n)
    for a, b in zip(good, bad):
        assert torch.equal(a[:500], b[:500]) and torch.equal(a[630:], b[630:])
    for value in (NAN, float("inf"), float("-inf")):
        k[630 + 140] = value
        bad = fd.fd_prompt_attention(q, k, v, n)
        for a, b in zip(good, bad):
            assert torch.equal(a[:500], b[:500]) and torch.equal(a[630:770], b[630:770])
            if value != value:
                assert bool(b[770:].isnan().all())


@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 128), (40, 40, 64)])
def test_two_row_tiles_in_a_graph(hq, hkv, d):
    fd = _fd()
    lens = [700, 0, 45, 1333]
    q, k, v = _inputs(lens, hq, hkv, d, 15)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fd.fd_reserve_workspace(fd.fd_prompt_workspace_bytes(4, sum(lens), hq, hkv, d), stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fd.fd_prompt_attention(q, k, v, n, out=out, lse=lse)
    # the kernel of the padded batch stays that of its rows, whatever the lengths of a replay
    for new in ([700, 0, 45, 1333], [1, 2, 3, 4], [2078, 0, 0, 0], [0, 1, 0, 0]):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(9.0), lse.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        t = sum(new)
        assert bool((out[t:] == 9.0).all()) and bool((lse[t:] == 9.0).all())
        ref.check_rows(out[:t], lse[:t], ref.prompt(q[:t], k[:t], v[:t], new))
    assert fd.fd_poll_status(stream=s) == 0
