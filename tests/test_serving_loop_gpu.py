"""A small serving run through the operators together: prompts are attended and written to pages,
forked, verified with drafted trees, compacted to the accepted drafts, decoded and freed. Every
attention result is compared with the 64-bit reference over keys kept apart on the host."""

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hq,hkv,d,size", [(16, 2, 128, 16), (4, 4, 64, 128), (12, 2, 128, 8)])
def test_serving_run(hq, hkv, d, size):
    import split_kv_decode_flashdecoding_b200 as fd
    gen, host = torch.Generator(device="cuda").manual_seed(3), torch.Generator().manual_seed(3)
    rand = lambda t, h: torch.randn((t, h, d), generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    prompts, seqs = [150, 1, 77], 6
    pages = 120
    k_pages = torch.full((pages, hkv, size, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v_pages = k_pages.clone()
    refs, table = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.full((seqs, 48), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")

    # the prompts: attention over the packed projections, the same rows into the cache
    t = sum(prompts)
    q, k, v = rand(t, hq), rand(t, hkv), rand(t, hkv)
    out, lse = fd.fd_prompt_attention(q, k, v, _i32(prompts))
    ref.check_rows(out, lse, ref.prompt(q, k, v, prompts), "prompts")
    held = prompts + [0] * 3
    fd.fd_pages_reserve(refs, table, _i32(held), size)
    fd.fd_pages_append(k, v, k_pages, v_pages, table, _i32([0] * seqs), _i32(held))
    lens.copy_(_i32(held))
    keys = [list(x) for x in zip(k.split(prompts), v.split(prompts))]

    # two more samples of the first prompt, one of the last
    fd.fd_pages_fork(k_pages, v_pages, refs, table, lens, _i32([0, 0, 2]), _i32([3, 4, 5]))
    keys += [list(keys[0]), list(keys[0]), list(keys[2])]
    held = [150, 1, 77, 150, 150, 77]
    assert lens.tolist() == held

    for step in range(3):
        trees = torch.randint(1, 20, (seqs,), generator=host).tolist()
        see = [ref.random_tree(host, n) for n in trees]
        t = sum(trees)
        q, k, v = rand(t, hq), rand(t, hkv), rand(t, hkv)
        pre = _i32(held)
        fd.fd_pages_reserve(refs, table, _i32([a + n for a, n in zip(held, trees)]), size)
        fd.fd_pages_append(k, v, k_pages, v_pages, table, pre, _i32(trees))
        out, lse = fd.fd_tree_attention_paged(q, k_pages, v_pages, table, pre, _i32(trees), ref.mask_words(see, 1).cuda())
        caches = [(torch.cat([a, x]), torch.cat([b, y])) for (a, b), x, y in zip(keys, k.split(trees), v.split(trees))]
        ref.check_rows(out, lse, ref.tree(q, caches, held, trees, see), f"trees {step}")
        # accept the path to some node of each tree (none of the second sequence's)
        paths = [torch.nonzero(s[int(torch.randint(0, n, (1,), generator=host))])[:, 0].tolist() for s, n in zip(see, trees)]
        paths[1] = []
        kept = [len(x) for x in paths]
        rows = [x + [0] * (max(kept) - len(x)) for x in paths]
        fd.fd_pages_compact(k_pages, v_pages, refs, table, lens, pre, _i32(rows), _i32(kept))
        for b, ((a, c), p, path) in enumerate(zip(caches, held, paths)):
            at = list(range(p)) + [p + i for i in path]
            keys[b] = [a[at], c[at]]
        held = [p + n for p, n in zip(held, kept)]
        assert lens.tolist() == held
        # a plain decode step over what is held now
        q = rand(seqs, hq)
        out, lse = fd.fd_decode_attention_paged(q, k_pages, v_pages, table, lens)
        want = ref.tree(q, [tuple(x) for x in keys], [n - 1 for n in held], [1] * seqs, [torch.ones(1, 1, dtype=torch.bool)] * seqs)
        ref.check_rows(out, lse, want, f"decode {step}")
    used = sum(-(-n // size) for n in held)
    assert int(refs.sum()) == used and int((refs > 1).sum()) > 0 if size <= 64 else True
    fd.fd_pages_free(refs, table, lens, _i32(list(range(seqs))))
    assert not refs.any() and not lens.any() and bool((table < 0).all())
    assert fd.fd_poll_status() == 0


def test_places_behind_2_to_the_31_elements():
    import split_kv_decode_flashdecoding_b200 as fd
    pages, hkv, size, d, hq = 16400, 8, 128, 128, 16
    taken = (1 << 31) // (hkv * size * d)  # the pages from here on lie behind 2^31 elements
    gen = torch.Generator(device="cuda").manual_seed(31)
    k_pages = torch.zeros((pages, hkv, size, d), dtype=torch.bfloat16, device="cuda")
    v_pages, refs, table = torch.zeros_like(k_pages), _i32([1] * taken + [0] * (pages - taken)), _i32([[-1] * 4] * 2)
    prefix, new = 300, 5
    q, k, v = (torch.randn((prefix + new, h, d), generator=gen, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    fd.fd_pages_reserve(refs, table, _i32([prefix + new, 0]), size)
    assert table.tolist() == [[taken, taken + 1, taken + 2, -1], [-1] * 4]
    fd.fd_pages_append(k, v, k_pages, v_pages, table, _i32([0, 0]), _i32([prefix + new, 0]))
    lens = _i32([prefix + new, 0])
    fd.fd_pages_fork(k_pages, v_pages, refs, table, lens, _i32([0]), _i32([1]))
    assert table.tolist() == [[taken, taken + 1, taken + 2, -1], [taken, taken + 1, taken + 3, -1]]
    see = [ref.random_tree(torch.Generator().manual_seed(32), new)] * 2
    drafts = torch.cat([q[prefix:]] * 2)
    out, lse = fd.fd_tree_attention_paged(drafts, k_pages, v_pages, table, _i32([prefix] * 2), _i32([new] * 2),
                                          ref.mask_words(see, 1).cuda())
    ref.check_rows(out, lse, ref.tree(drafts, [(k, v)] * 2, [prefix] * 2, [new] * 2, see), "tree")
    fd.fd_pages_compact(k_pages, v_pages, refs, table, lens, _i32([prefix, 0]), _i32([[1, 4], [0, 0]]), _i32([2, -1]))
    assert lens.tolist() == [prefix + 2, prefix + new]
    for pool, x in ((k_pages, k), (v_pages, v)):
        for page, rows in ((taken + 2, [*range(256, 300), 301, 304]), (taken + 3, [*range(256, 305)])):
            assert torch.equal(pool[page, :, :len(rows)], x[rows].transpose(0, 1))
        assert not bool(pool[:taken].any()) and not bool(pool[taken + 4:].any())
    assert fd.fd_poll_status() == 0
