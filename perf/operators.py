"""Cases of the serving operators around split-KV decoding: attention of whole prompts, attention
of drafted trees over a cache, and the operators of a paged cache's pages.

A pass is one call (or, for the page tables, the few calls of one scheduling step) as a serving loop
makes it. With `own` false every operator is computed from its definition by elementary torch
operations in 32 bits; with `own` true by the package's kernels.
"""

import math

import torch

own = False

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ---------------------------------------------------------------------------- cases -------------

def listed():
    return [
        # a handful of chat turns that arrive together: every length is below one query tile
        {"name": "prompt short", "op": "prompt", "hq": 64, "hkv": 8, "d": 128, "lens": "45,1,96,17"},
        # a batch of mixed requests, multi-head with head_dim 64, ragged lengths, an empty one
        {"name": "prompt ragged mha d64", "op": "prompt", "hq": 32, "hkv": 32, "d": 64,
         "lens": "1024,333,0,2048,7,129,1500,512,61,1999"},
        # two documents: the compute-bound end
        {"name": "prompt long", "op": "prompt", "hq": 64, "hkv": 8, "d": 128, "lens": "16384,9001"},
        # one user, a small tree on a short contiguous cache: latency
        {"name": "tree one user", "op": "tree", "hq": 64, "hkv": 8, "d": 128, "page": 0,
         "prefix": "300", "trees": "5"},
        # 32 users with the 70B-like decode lengths, 16 drafts each, 16-key pages
        {"name": "tree batch paged16", "op": "tree", "hq": 64, "hkv": 8, "d": 128, "page": 16,
         "prefix": "5120,31007,12001,2048,17411,28003,9999,1024,22222,15000,30500,4097,26001,11111,"
                   "19283,7000,32700,13579,24680,3333,16384,20000,8191,29000,6006,18018,10101,27272,"
                   "14141,25252,1500,21212",
         "trees": "16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,16,"
                  "16,16,16,16"},
        # wide trees (up to 64 drafts), groups of 4, 64-key pages, a sequence without a prefix
        {"name": "tree wide paged64", "op": "tree", "hq": 32, "hkv": 8, "d": 128, "page": 64,
         "prefix": "8000,513,0,4099,6144,77,7777,2500", "trees": "64,33,50,64,1,64,47,60"},
        # the new token of each of 64 decoding sequences, 16-key pages: latency
        {"name": "append step bf16", "op": "append", "hkv": 8, "d": 128, "page": 16, "kv": "bf16",
         "starts": ",".join(str(37 * i + 5) for i in range(64)), "news": ",".join(["1"] * 64)},
        # the keys and values of a prefill of ragged prompts into an E4M3 cache of 128-key pages
        {"name": "append prefill e4m3", "op": "append", "hkv": 8, "d": 128, "page": 128, "kv": "e4m3",
         "starts": "0,512,0,1001,0,0,4096,0", "news": "16384,9001,333,4096,1,17000,8191,10000"},
        # one step of a beam search: 8 groups of 4 beams, half of them replaced, 16-key pages
        {"name": "fork beams page16", "op": "fork", "hkv": 8, "d": 128, "page": 16, "groups": 8,
         "beams": 4, "spare": 256, "lens": "100,517,1000,33,16,64,2049,777"},
        # many samples of long prompts, 128-key pages
        {"name": "fork samples page128", "op": "fork", "hkv": 8, "d": 128, "page": 128, "groups": 24,
         "beams": 8, "spare": 2048,
         "lens": ",".join(str(1000 + 613 * i) for i in range(24))},
        # a verification step: 32 sequences write 16 drafts each and keep the accepted ones
        {"name": "compact drafts", "op": "compact", "hkv": 8, "d": 128, "page": 16, "spare": 64,
         "starts": ",".join(str(100 + 211 * i) for i in range(32)),
         "news": ",".join(["16"] * 32), "keeps": ",".join(str(1 + i % 6) for i in range(32))},
        # cache eviction: 2048-odd of 4096 tokens of 16 sequences stay, 64-key pages
        {"name": "compact eviction", "op": "compact", "hkv": 8, "d": 128, "page": 64, "spare": 64,
         "starts": ",".join(str(4 + 13 * i) for i in range(16)),
         "news": ",".join(["4096"] * 16), "keeps": ",".join(str(2048 - 5 * i) for i in range(16))},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in str(text).split(",")]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "append", "fork", "compact"])
    hq, hkv = rng.choice([(64, 8), (32, 32), (40, 40), (32, 8), (8, 2), (12, 2), (6, 2), (16, 1), (7, 1)])
    d = rng.choice([64, 128, 128])
    if op == "prompt":
        longest = _log(rng, 1, 8192)
        n = rng.randint(1, max(1, min(24, (1 << 27) // (longest * longest))))
        lens = [longest] + [min(longest, _log(rng, 1, longest) - (rng.random() < 0.05)) for _ in range(n - 1)]
        rng.shuffle(lens)
        return {"op": op, "hq": hq, "hkv": hkv, "d": d, "lens": _text(lens)}
    if op == "tree":
        n = _log(rng, 1, 32)
        longest = _log(rng, 16, min(32768, 400000 // n))
        most = _log(rng, 1, min(128, max(1, (1 << 30) // (n * hq * longest))))
        return {"op": op, "hq": hq, "hkv": hkv, "d": d, "page": rng.choice([0, 0, 8, 16, 32, 64, 128, 256]),
                "prefix": _text([rng.randint(0, longest) for _ in range(n)]),
                "trees": _text([rng.randint(1, most) for _ in range(n)])}
    hkv = rng.choice([1, 2, 8, 8, 32])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "append":
        n = _log(rng, 1, 128)
        most = _log(rng, 1, max(1, 400000 // (n * hkv)))
        return {"op": op, "hkv": hkv, "d": d, "page": page, "kv": rng.choice(["bf16", "e4m3", "f32"]),
                "starts": _text([rng.randint(0, 2000) for _ in range(n)]),
                "news": _text([rng.randint(0, most) for _ in range(n - 1)] + [most])}
    if op == "fork":
        groups, beams = _log(rng, 1, 24), rng.randint(2, 8)
        longest = _log(rng, 1, max(1, 300000 // (groups * hkv)))
        return {"op": op, "hkv": hkv, "d": d, "page": page, "groups": groups, "beams": beams,
                "spare": groups * beams * 2 + rng.randint(0, 500),
                "lens": _text([rng.randint(1, longest) for _ in range(groups)])}
    n = _log(rng, 1, 64)
    most = _log(rng, 1, max(1, min(8192, 300000 // (n * hkv))))
    news = [rng.randint(1, most) for _ in range(n)]
    return {"op": op, "hkv": hkv, "d": d, "page": page, "spare": rng.randint(0, 100),
            "starts": _text([rng.randint(0, 1000) for _ in range(n)]),
            "news": _text(news), "keeps": _text([rng.randint(0, m) for m in news])}


def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op == "prompt":
        lens, hq = _ints(case["lens"]), case["hq"]
        t = sum(lens)
        return {"bytes": 2 * t * (hq + hkv) * d * 2 + t * hq * 4 + 4 * len(lens),
                "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    if op == "tree":
        pre, new, hq = _ints(case["prefix"]), _ints(case["trees"]), case["hq"]
        t = sum(new)
        keys = sum(p + n for p, n in zip(pre, new))
        table = 0 if case["page"] == 0 else 4 * sum(-(-(p + n) // case["page"]) for p, n in zip(pre, new))
        return {"bytes": 2 * keys * hkv * d * 2 + 2 * t * hq * d * 2 + t * hq * 4 + t * 4 * _words(case) + table,
                "flops": 4 * d * hq * sum(n * (p + 1) for p, n in zip(pre, new))}
    if op == "append":
        t = sum(_ints(case["news"]))
        es, et = {"bf16": (2, 2), "e4m3": (2, 1), "f32": (4, 4)}[case["kv"]]
        return {"bytes": 2 * t * hkv * d * (es + et) + 8 * len(_ints(case["news"])), "flops": 0}
    row = 2 * hkv * d * 2
    if op == "fork":
        copies = sum((n % case["page"]) * (case["beams"] // 2) for n in _beam_lens(case))
        rows, pages = case["groups"] * case["beams"], _fork_pages(case)
        return {"bytes": 2 * copies * row + 8 * rows * _fork_columns(case) + 8 * pages, "flops": 0}
    t, kept = sum(_ints(case["news"])), sum(_ints(case["keeps"]))
    return {"bytes": 2 * t * row + 2 * kept * row + 4 * kept, "flops": 0}


def _words(case):
    return -(-max(_ints(case["trees"])) // 32)


def _beam_lens(case):
    """The length that every beam of a group has."""
    return _ints(case["lens"])


def _fork_columns(case):
    return max(_beam_lens(case)) // case["page"] + 2


def _fork_pages(case):
    per = [n // case["page"] + 2 * case["beams"] for n in _beam_lens(case)]
    return sum(per) + case["spare"]


# ---------------------------------------------------------------------------- inputs ------------

def _i32(values, dev="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _randn(gen, shape, dtype=BF16):
    x = torch.empty(shape, dtype=torch.float32 if dtype == torch.float32 else BF16, device="cuda")
    x.normal_(generator=gen)
    return x if x.dtype == dtype else x.to(dtype)


def _ancestors(gen, n):
    """Visibility of one random tree of n drafts: a draft sees itself and its ancestors."""
    parent = (torch.rand(n, generator=gen) * torch.arange(n + 1)[1:]).long() - 1  # -1: a child of the root
    see = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        if parent[i] >= 0:
            see[i] = see[parent[i]]
        see[i, i] = True
    return see


def _mask_words(see, words):
    n = see.shape[0]
    bits = torch.zeros(n, words * 32, dtype=torch.int64)
    bits[:, :n] = see
    w = (bits.view(n, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    return _PREPARE[case["op"]](case, gen, host)


def _prepare_prompt(case, gen, host):
    lens, hq, hkv, d = _ints(case["lens"]), case["hq"], case["hkv"], case["d"]
    t = sum(lens)
    k = _randn(gen, (t, hkv, d))
    start = 0
    for n in lens:  # the first key of a sequence draws much of the attention
        if n:
            k[start] *= 3
        start += n
    return {"op": "prompt", "q": _randn(gen, (t, hq, d)), "k": k, "v": _randn(gen, (t, hkv, d)),
            "seq_lens": _i32(lens), "longest": max(lens)}


def _shuffled_table(host, counts, columns, pages):
    """A block table whose sequences own counts[b] pages at random places of the pool."""
    order = torch.randperm(pages, generator=host).tolist()
    table = torch.full((len(counts), columns), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    return table.cuda()


def _prepare_tree(case, gen, host):
    pre, new = _ints(case["prefix"]), _ints(case["trees"])
    hq, hkv, d, page, words = case["hq"], case["hkv"], case["d"], case["page"], _words(case)
    total = [p + n for p, n in zip(pre, new)]
    s = {"op": "tree", "q": _randn(gen, (sum(new), hq, d)), "prefix_lens": _i32(pre), "tree_lens": _i32(new),
         "tree_mask": torch.cat([_mask_words(_ancestors(host, n), words) for n in new]).cuda(),
         "table": None, "most": max(new), "keys": max(total)}
    if page:
        counts = [-(-t // page) for t in total]
        s["table"] = _shuffled_table(host, counts, max(counts), sum(counts) + 3)
        shape = (sum(counts) + 3, hkv, page, d)
    else:
        shape = (len(pre), hkv, max(total), d)
    return {**s, "k": _randn(gen, shape), "v": _randn(gen, shape)}


def _prepare_append(case, gen, host):
    starts, news = _ints(case["starts"]), _ints(case["news"])
    hkv, d, page = case["hkv"], case["d"], case["page"]
    counts = [-(-(a + n) // page) for a, n in zip(starts, news)]
    pages = sum(counts) + 1
    dt = {"bf16": BF16, "e4m3": E4M3, "f32": torch.float32}[case["kv"]]
    src = BF16 if dt == E4M3 else dt
    t = sum(news)
    return {"op": "append", "k_new": _randn(gen, (t, hkv, d), src), "v_new": _randn(gen, (t, hkv, d), src),
            "k": _randn(gen, (pages, hkv, page, d), dt), "v": _randn(gen, (pages, hkv, page, d), dt),
            "table": _shuffled_table(host, counts, max(counts), pages), "starts": _i32(starts), "news": _i32(news),
            "k_scale": 0.011, "v_scale": 0.0093}


def _prepare_fork(case, gen, host):
    groups, beams, page = case["groups"], case["beams"], case["page"]
    pages, columns = _fork_pages(case), _fork_columns(case)
    order = torch.randperm(pages, generator=host).tolist()
    table, refs, lens, src, dst = [], [0] * pages, [], [], []
    for g, n in enumerate(_beam_lens(case)):
        shared = [order.pop() for _ in range(n // page)]
        ranks = torch.randperm(beams, generator=host).tolist()
        for i in range(beams):  # the beams of a group share its full pages and own the last one
            mine = shared + ([order.pop()] if n % page else [])
            for p in mine:
                refs[p] += 1
            table.append(mine + [-1] * (columns - len(mine)))
            lens.append(n)
        for i in range(beams // 2):  # the lower half is replaced by copies of the upper half
            src.append(g * beams + ranks[i])
            dst.append(g * beams + ranks[beams - 1 - i])
    shape = (pages, case["hkv"], page, case["d"])
    return {"op": "fork", "k": _randn(gen, shape), "v": _randn(gen, shape), "refs": _i32(refs), "table": _i32(table),
            "lens": _i32(lens), "src": _i32(src), "dst": _i32(dst), "want": _i32([n + 1 for n in lens])}


def _prepare_compact(case, gen, host):
    starts, news, keeps = _ints(case["starts"]), _ints(case["news"]), _ints(case["keeps"])
    hkv, d, page = case["hkv"], case["d"], case["page"]
    full = [-(-(a + n) // page) for a, n in zip(starts, news)]
    now = [-(-a // page) for a in starts]
    pages = sum(full) + case["spare"]
    table = _shuffled_table(host, now, max(full) + 1, pages)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    keep = torch.zeros((len(news), max(max(keeps), 1)), dtype=torch.int32)
    for b, (n, m) in enumerate(zip(news, keeps)):
        keep[b, :m] = torch.randperm(n, generator=host)[:m].sort().values.to(torch.int32)
    t, shape = sum(news), (pages, hkv, page, d)
    return {"op": "compact", "k_new": _randn(gen, (t, hkv, d)), "v_new": _randn(gen, (t, hkv, d)),
            "k": _randn(gen, shape), "v": _randn(gen, shape), "refs": refs, "table": table,
            "lens": _i32(starts), "starts": _i32(starts), "news": _i32(news), "keep": keep.cuda(),
            "keep_lens": _i32(keeps), "want": _i32([a + n for a, n in zip(starts, news)])}


_PREPARE = {"prompt": _prepare_prompt, "tree": _prepare_tree, "append": _prepare_append,
            "fork": _prepare_fork, "compact": _prepare_compact}


# ---------------------------------------------------------------------------- one pass ----------

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import split_kv_decode_flashdecoding_b200 as fd

    op = s["op"]
    if op == "prompt":
        return fd.fd_prompt_attention(s["q"], s["k"], s["v"], s["seq_lens"])
    if op == "tree":
        if s["table"] is None:
            return fd.fd_tree_attention(s["q"], s["k"], s["v"], s["prefix_lens"], s["tree_lens"], s["tree_mask"])
        return fd.fd_tree_attention_paged(s["q"], s["k"], s["v"], s["table"], s["prefix_lens"], s["tree_lens"],
                                          s["tree_mask"])
    if op == "append":
        if s["k"].dtype == E4M3:
            fd.fd_pages_append_fp8(s["k_new"], s["v_new"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"],
                                   s["starts"], s["news"])
        else:
            fd.fd_pages_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["starts"], s["news"])
        return s["k"], s["v"]
    if op == "fork":
        fd.fd_pages_free(s["refs"], s["table"], s["lens"], s["dst"])
        fd.fd_pages_fork(s["k"], s["v"], s["refs"], s["table"], s["lens"], s["src"], s["dst"])
        fd.fd_pages_reserve(s["refs"], s["table"], s["want"], s["k"].shape[2])
    else:
        fd.fd_pages_reserve(s["refs"], s["table"], s["want"], s["k"].shape[2])
        fd.fd_pages_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["starts"], s["news"])
        fd.fd_pages_compact(s["k"], s["v"], s["refs"], s["table"], s["lens"], s["starts"], s["keep"], s["keep_lens"])
    return s["k"], s["v"], s["refs"], s["table"], s["lens"]


def _softmax_sums(scores, v):
    """(sum_j p_j v_j / sum_j p_j, ln sum_j e^s_j) over the last axis of scores; rows of -inf give 0 and -inf."""
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = p @ v
    out = torch.where(total > 0, out / total, 0.0)
    return out, (torch.log(total) + m).squeeze(-1)


def _plain_prompt(s):
    q, k, v, lens, longest = s["q"], s["k"], s["v"], s["seq_lens"].long(), s["longest"]
    t, hq, d = q.shape
    hkv = k.shape[1]
    ends = lens.cumsum(0)
    at = torch.arange(longest, device=q.device)
    rows = (ends - lens)[:, None] + torch.minimum(at, (lens[:, None] - 1).clamp_min(0))  # [B, L], repeated past the end
    rows = rows.clamp_max(t - 1)
    b = rows.shape[0]
    qp = q.float()[rows].view(b, longest, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    kp = k.float()[rows].permute(0, 2, 3, 1)[:, :, None]       # [B, Hkv, 1, D, L]
    vp = v.float()[rows].permute(0, 2, 1, 3)[:, :, None]       # [B, Hkv, 1, L, D]
    out = torch.empty((b, hkv, hq // hkv, longest, d), device=q.device)
    lse = torch.empty((b, hkv, hq // hkv, longest), device=q.device)
    step = max(64, (1 << 29) // (b * hq * longest))
    for i in range(0, longest, step):  # one step where the scores fit 2 GB
        j = min(longest, i + step)
        scores = (qp[:, :, :, i:j] * d ** -0.5) @ kp[..., :j]
        scores = torch.where(at[:j] <= at[i:j, None], scores, -math.inf)
        out[:, :, :, i:j], lse[:, :, :, i:j] = _softmax_sums(scores, vp[:, :, :, :j])
    row = torch.arange(t, device=q.device)
    seq = torch.searchsorted(ends, row, right=True)
    pos = row - (ends - lens)[seq]
    return (out.permute(0, 3, 1, 2, 4)[seq, pos].reshape(t, hq, d).to(q.dtype),
            lse.permute(0, 3, 1, 2)[seq, pos].reshape(t, hq))


def _plain_tree(s):
    q, pre, new, mask, most, keys = s["q"], s["prefix_lens"].long(), s["tree_lens"].long(), s["tree_mask"], s["most"], s["keys"]
    t, hq, d = q.shape
    dev, b = q.device, pre.shape[0]
    if s["table"] is None:
        k, v = s["k"][:, :, :keys].float(), s["v"][:, :, :keys].float()
    else:
        page = s["table"].clamp_min(0).long()
        k, v = (x[page].permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :keys].float() for x in (s["k"], s["v"]))
    hkv = k.shape[1]
    ends = new.cumsum(0)
    rows = ((ends - new)[:, None] + torch.arange(most, device=dev)).clamp_max(t - 1)  # [B, most]
    bits = ((mask[rows][..., None] >> torch.arange(32, device=dev)) & 1).flatten(2).bool()  # [B, most, 32 W]
    key = torch.arange(keys, device=dev)
    draft = (key - pre[:, None])                                # [B, keys]: index of a key among the drafts
    seen = bits.gather(2, draft.clamp(0, bits.shape[2] - 1)[:, None].expand(b, most, keys))
    seen = (draft < 0)[:, None] | (seen & (draft < new[:, None])[:, None])
    qp = (q.float()[rows] * d ** -0.5).view(b, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    scores = (qp.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (hq // hkv, most))
    scores = torch.where(seen[:, None, None], scores, -math.inf).flatten(2, 3)
    out, lse = _softmax_sums(scores, v)
    row = torch.arange(t, device=dev)
    seq = torch.searchsorted(ends, row, right=True)
    pos = row - (ends - new)[seq]
    out = out.unflatten(2, (hq // hkv, most)).permute(0, 3, 1, 2, 4)[seq, pos]
    lse = lse.unflatten(2, (hq // hkv, most)).permute(0, 3, 1, 2)[seq, pos]
    return out.reshape(t, hq, d).to(q.dtype), lse.reshape(t, hq)


def _store(pages, page, slot, rows, scale):
    if pages.dtype == E4M3:
        code = (rows.float() / scale).clamp(-448.0, 448.0).to(E4M3)
        pages.view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
    else:
        pages[page, :, slot] = rows


def _append_rows(s):
    size, news = s["k"].shape[2], s["news"].long()
    ends = news.cumsum(0)
    row = torch.arange(s["k_new"].shape[0], device=news.device)
    seq = torch.searchsorted(ends, row, right=True)
    pos = s["starts"].long()[seq] + row - (ends - news)[seq]
    page, slot = s["table"][seq, pos // size].long(), pos % size
    _store(s["k"], page, slot, s["k_new"], s.get("k_scale"))
    _store(s["v"], page, slot, s["v_new"], s.get("v_scale"))


def _plain_append(s):
    _append_rows(s)
    return s["k"], s["v"]


def _free_pages(refs):
    """The pages without a user, lowest first (then the others)."""
    return torch.argsort((refs > 0).to(torch.int8), stable=True)


def _add_refs(refs, pages, by):
    refs.index_add_(0, pages.clamp_min(0).flatten().long(), (pages >= 0).flatten().to(torch.int32) * by)


def _reserve(s):
    table, size = s["table"], s["k"].shape[2]
    column = torch.arange(table.shape[1], device=table.device)
    missing = (table < 0) & (column < (s["want"][:, None] + size - 1) // size)
    rank = missing.flatten().cumsum(0).view(table.shape) - 1
    table.copy_(torch.where(missing, _free_pages(s["refs"])[rank.clamp_min(0)].to(torch.int32), table))
    _add_refs(s["refs"], torch.where(missing, table, -1), 1)


def _plain_fork(s):
    k, v, refs, table, lens, src, dst = (s[n] for n in ("k", "v", "refs", "table", "lens", "src", "dst"))
    src, dst, size = src.long(), dst.long(), k.shape[2]
    # free the losers
    _add_refs(refs, table[dst], -1)
    table[dst] = -1
    lens[dst] = 0
    # share the winners' full pages, copy the rows of their last ones
    n, column = lens[src], torch.arange(table.shape[1], device=table.device)
    full, tail = n // size, n % size
    row = torch.where(column < full[:, None], table[src], -1)
    # a fork that ends with a full page is given a page too, which it leaves as it is
    rank = torch.where(tail > 0, (tail > 0).cumsum(0) - 1, len(src) + torch.arange(len(src), device=k.device))
    fresh = _free_pages(refs)[rank].to(torch.int32)
    last = full.long().clamp_max(table.shape[1] - 1)[:, None]
    old = table[src].gather(1, last)[:, 0]
    row = torch.where((column == full[:, None]) & (tail > 0)[:, None], fresh[:, None], row)
    table[dst] = row
    lens[dst] = n
    _add_refs(refs, row, 1)
    to, of = fresh.long(), old.clamp_min(0).long()
    live = (torch.arange(size, device=k.device) < tail[:, None])[:, None, :, None]
    k[to] = torch.where(live, k[of], k[to])
    v[to] = torch.where(live, v[of], v[to])
    _reserve(s)
    return k, v, refs, table, lens


def _plain_compact(s):
    k, v, refs, table, lens, keep, kept = (s[n] for n in ("k", "v", "refs", "table", "lens", "keep", "keep_lens"))
    size, starts = k.shape[2], s["starts"]
    _reserve(s)
    _append_rows(s)
    # a place past a sequence's last kept row repeats that row's move (its first one's, in place, if none is kept)
    i = torch.minimum(torch.arange(keep.shape[1], device=keep.device), (kept[:, None] - 1).clamp_min(0))
    to = (starts[:, None] + i).long()
    of = torch.where(kept[:, None] > 0, starts[:, None] + keep.gather(1, i), to)
    seq = torch.arange(keep.shape[0], device=keep.device)[:, None]
    page = table.clamp_min(0).long()
    of, to = (page[seq, of // size], of % size), (page[seq, to // size], to % size)
    k[to[0], :, to[1]] = k[of[0], :, of[1]]
    v[to[0], :, to[1]] = v[of[0], :, of[1]]
    lens.copy_(starts + kept)
    column = torch.arange(table.shape[1], device=table.device)
    unused = column >= ((lens + size - 1) // size)[:, None]
    _add_refs(refs, torch.where(unused, table, -1), -1)
    table.masked_fill_(unused, -1)
    return k, v, refs, table, lens


_PLAIN = {"prompt": _plain_prompt, "tree": _plain_tree, "append": _plain_append, "fork": _plain_fork,
          "compact": _plain_compact}


# ---------------------------------------------------------------------------- in 64 bits --------

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, one sequence after another."""
    s = prepare(case, seed)
    return _EXACT[s["op"]](s)


def _exact_rows(q, k, v, see):
    """One sequence: q [n, Hq, D] against k, v [keys, Hkv, D]; see(rows) -> [rows, keys] truth values."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    step = max(1, (1 << 27) // max(1, k.shape[0]))
    for h in range(hq):
        kk, vv = k[:, h * hkv // hq].double(), v[:, h * hkv // hq].double()
        for i in range(0, n, step):
            x = q[i:i + step, h].double() @ kk.T / math.sqrt(d)
            x.masked_fill_(~see(slice(i, min(n, i + step))), -math.inf)
            lse[i:i + step, h] = torch.logsumexp(x, -1)
            out[i:i + step, h] = torch.softmax(x, -1).nan_to_num(0.0) @ vv
    return out, lse


def _exact_prompt(s):
    at, outs = 0, []
    for n in s["seq_lens"].tolist():
        part = slice(at, at + n)
        at += n
        order = torch.arange(n, device="cuda")
        outs.append(_exact_rows(s["q"][part], s["k"][part], s["v"][part], lambda r: order <= order[r, None]))
    return tuple(torch.cat(x) for x in zip(*outs))


def _exact_tree(s):
    at, outs = 0, []
    for b, (p, n) in enumerate(zip(s["prefix_lens"].tolist(), s["tree_lens"].tolist())):
        if s["table"] is None:
            k, v = (x[b, :, :p + n].transpose(0, 1) for x in (s["k"], s["v"]))
        else:
            size = s["k"].shape[2]
            ids = s["table"][b, :-(-(p + n) // size)].tolist()
            k, v = (torch.cat([x[i].transpose(0, 1) for i in ids])[:p + n] for x in (s["k"], s["v"]))
        words = s["tree_mask"][at:at + n].cpu().tolist()
        see = torch.ones((n, p + n), dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                see[i, p + j] = bool(words[i][j // 32] & (1 << (j % 32)))
        see = see.cuda()
        outs.append(_exact_rows(s["q"][at:at + n], k, v, lambda r: see[r]))
        at += n
    return tuple(torch.cat(x) for x in zip(*outs))


def _exact_write(s, pools, scales):
    at, size = 0, s["k"].shape[2]
    for b, (p, n) in enumerate(zip(s["starts"].tolist(), s["news"].tolist())):
        ids = s["table"][b].tolist()
        i = 0
        while i < n:  # page by page
            slot = (p + i) % size
            m = min(size - slot, n - i)
            for pool, new, scale in zip(pools, ("k_new", "v_new"), scales):
                pool[ids[(p + i) // size], :, slot:slot + m] = (s[new][at + i:at + i + m].double() / scale).transpose(0, 1)
            i += m
        at += n


def _exact_append(s):
    pools = [s["k"].double(), s["v"].double()]
    _exact_write(s, pools, (s["k_scale"], s["v_scale"]) if s["k"].dtype == E4M3 else (1.0, 1.0))
    return [x.clamp(-448, 448) for x in pools] if s["k"].dtype == E4M3 else pools


def _exact_reserve(refs, table, want, size):
    for row, n in zip(table, want):
        for c in range(-(-n // size)):
            if row[c] < 0:
                row[c] = refs.index(0)
                refs[row[c]] = 1


def _exact_fork(s):
    size = s["k"].shape[2]
    refs, table, lens = s["refs"].tolist(), s["table"].tolist(), s["lens"].tolist()
    for b in s["dst"].tolist():
        for p in table[b]:
            if p >= 0:
                refs[p] -= 1
        table[b], lens[b] = [-1] * len(table[b]), 0
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        full, tail = divmod(lens[a], size)
        for c in range(full):
            table[b][c] = table[a][c]
            refs[table[a][c]] += 1
        if tail:
            table[b][full] = refs.index(0)
            refs[table[b][full]] = 1
            for pool in (s["k"], s["v"]):
                pool[table[b][full], :, :tail] = pool[table[a][full], :, :tail]
        lens[b] = lens[a]
    _exact_reserve(refs, table, s["want"].tolist(), size)
    return s["k"].double(), s["v"].double(), _i32(refs), _i32(table), _i32(lens)


def _exact_compact(s):
    size = s["k"].shape[2]
    refs, table, lens = s["refs"].tolist(), s["table"].tolist(), s["lens"].tolist()
    _exact_reserve(refs, table, s["want"].tolist(), size)
    s["table"] = _i32(table)
    pools = [s["k"].double(), s["v"].double()]
    _exact_write(s, pools, (1.0, 1.0))
    for b, (a, m) in enumerate(zip(s["starts"].tolist(), s["keep_lens"].tolist())):
        ids, at = s["table"][b].clamp_min(0).long(), torch.arange(a, a + m, device="cuda")
        of = a + s["keep"][b, :m].long()
        for pool in pools:
            pool[ids[at // size], :, at % size] = pool[ids[of // size], :, of % size].clone()
        lens[b] = a + m
        for c in range(-(-(a + m) // size), len(table[b])):
            if table[b][c] >= 0:
                refs[table[b][c]] -= 1
                table[b][c] = -1
    return pools[0], pools[1], _i32(refs), _i32(table), _i32(lens)


_EXACT = {"prompt": _exact_prompt, "tree": _exact_tree, "append": _exact_append, "fork": _exact_fork,
          "compact": _exact_compact}
