"""Trees of drafted tokens and eviction over the KV cache, as cases that can be timed and checked.

Six operators that a multi-adapter serving step needs next to its cache, its attention and its
verification of drafts:

  build    from the parents of a tree's tokens: which of them each token sees, and its depth
  attend   attention of a tree's tokens over their sequence's paged cache and their own ancestors
  verify   the path of a tree that the target accepts, and the token that follows it
  weigh    the attention that cached tokens get, summed over the new tokens and the query heads of
           a key head, on top of what they had before
  select   the tokens of each sequence and key head that stay in a cache of fewer tokens: the first
           and the latest ones and those with the largest weights
  compact  the tokens that stay (of a tree's path, or of a selection) move together in their pages

A sequence s has q_len new tokens, rows q_start[s] .. q_start[s + 1] of the new tensors, the last
q_len of its kv_len[s] cached ones.  table[s][0 = K, 1 = V][head][b] is the pool page of tokens
b * T .. (b + 1) * T - 1 of one head (T tokens a page).  With E elements in 16 bytes, element d of
token slot t of a K page is at ((d / E) * T + t) * E + d % E, and of a V page at
((t / E) * D + d) * E + t % E.  FP8 tokens have one exponent byte a head.

The new tokens of a tree are numbered 0, 1, .. within their sequence, a parent before its
children.  Bit u % 64 of word u / 64 of a token's row of `seen`: it sees new token u.  A token of
depth d is at position kv_len - q_len + d, whatever its place in the cache.

Sizes are those of this repository's workloads (32 heads of 128 at d = 4096, 40 at d = 5120, and
64 query heads over 8 key heads at d = 8192; a page is one d-row) or generic.
"""
import math
import random

import numpy as np
import torch

own = False

ONE = 1 << 44        # probabilities are summed as whole multiples of 2^-44
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _tree(name, seqs, q, words, lens, window=0):
    """q: (fewest, most) tokens of a tree; lens seeds the lengths."""
    return {"op": "build", "name": name, "seqs": seqs, "q_lo": q[0], "q_hi": q[1], "words": words, "lens": lens,
            "window": window}


def _attend_case(name, dtype, kv, page, heads, kv_heads, dim, seqs, q, kv_len, words, lens, window=0):
    return {"op": "attend", "name": name, "dtype": dtype, "kv": kv, "page": page, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "seqs": seqs, "q_lo": q[0], "q_hi": q[1], "kv_lo": kv_len[0],
            "kv_hi": kv_len[1], "words": words, "lens": lens, "window": window}


def _verify_case(name, dtype, vocab, seqs, q, lens):
    return {"op": "verify", "name": name, "dtype": dtype, "vocab": vocab, "seqs": seqs, "q_lo": q[0], "q_hi": q[1],
            "lens": lens}


def _weigh_case(name, dtype, kv, page, heads, kv_heads, dim, seqs, q, kv_len, lens, window=0, decay=1.0):
    return {"op": "weigh", "name": name, "dtype": dtype, "kv": kv, "page": page, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "seqs": seqs, "q_lo": q[0], "q_hi": q[1], "kv_lo": kv_len[0],
            "kv_hi": kv_len[1], "lens": lens, "window": window, "decay": decay}


def _select_case(name, kv_heads, seqs, kv_len, budget, sinks, recent, lens):
    return {"op": "select", "name": name, "dtype": "bf16", "kv": "bf16", "page": 8192, "kv_heads": kv_heads,
            "dim": 128, "seqs": seqs, "q_lo": 1, "q_hi": 1, "kv_lo": kv_len[0], "kv_hi": kv_len[1],
            "budget": budget, "sinks": sinks, "recent": recent, "lens": lens, "window": 0}


def _compact_case(name, what, dtype, kv, page, kv_heads, dim, seqs, q, kv_len, budget, lens):
    """what: "path" of a tree of q tokens, or "evict" to `budget` tokens."""
    return {"op": "compact", "name": name, "what": what, "dtype": dtype, "kv": kv, "page": page,
            "kv_heads": kv_heads, "dim": dim, "seqs": seqs, "q_lo": q[0], "q_hi": q[1], "kv_lo": kv_len[0],
            "kv_hi": kv_len[1], "budget": budget, "lens": lens, "window": 0}


def listed():
    return [
        # the tree of one request's next tokens: the smallest call, where latency counts
        _tree("build_one", 1, (25, 25), 1, 21),
        # the trees of a batch, wide ones among them, within an attention window
        _tree("build_batch", 128, (1, 250), 4, 22, 5),
        # 9 drafted tokens of one conversation, every query head with its own keys
        _attend_case("attend_one", "f16", "f16", 4096, 32, 32, 128, 1, (9, 9), (777, 777), 1, 23),
        # a verification step: trees of up to 64 tokens of 32 requests, 8 query heads a key head
        _attend_case("attend_batch", "bf16", "bf16", 8192, 64, 8, 128, 32, (17, 64), (900, 4100), 1, 24),
        # the tree of one request
        _verify_case("verify_one", "f32", 32000, 1, (25, 25), 25),
        # 64 requests with up to 63 drafted tokens over an odd vocabulary
        _verify_case("verify_batch", "f32", 131071, 64, (1, 64), 26),
        # a decode step of 64 requests over an FP8 cache, older attention fading
        _weigh_case("weigh_decode_fp8", "bf16", "fp8", 4096, 32, 32, 128, 64, (1, 1), (20, 2048), 27, 0, 0.97),
        # one chunk of a long prompt
        _weigh_case("weigh_chunk", "bf16", "bf16", 8192, 64, 8, 128, 1, (2048, 2048), (16384, 16384), 28),
        # 64 requests of a batch back to 512 tokens a head
        _select_case("select_batch", 32, 64, (20, 2048), 512, 4, 64, 29),
        # two long documents to an eighth
        _select_case("select_long", 8, 2, (100001, 131071), 16384, 4, 1000, 30),
        # after a verification step: the accepted path of 64 trees, FP8 cache
        _compact_case("compact_path_fp8", "path", "bf16", "fp8", 4096, 32, 128, 64, (9, 25), (100, 2000), 0, 31),
        # 16 requests back to 2048 tokens a head, with their weights
        _compact_case("compact_evict", "evict", "bf16", "bf16", 8192, 8, 128, 16, (1, 1), (4001, 16000), 2048, 32),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    op = rng.choice(("build", "attend", "attend", "verify", "weigh", "weigh", "select", "compact"))
    if op == "build":
        words = rng.choice((1, 1, 2, 4))
        hi = _spread(rng, 2, 64 * words)
        return _tree("", _spread(rng, 1, 128 // (words + 3) * 4), (rng.choice((1, hi)), hi), words, lens,
                     rng.choice((0, 0, rng.randint(1, 8))))
    if op == "verify":
        hi = _spread(rng, 2, 64)
        return _verify_case("", rng.choice(("f32", "f32", "f16", "bf16")), _spread(rng, 1000, 131072),
                            _spread(rng, 1, 64), (rng.choice((1, hi)), hi), lens)
    dtype = rng.choice(("f16", "bf16"))
    kv = rng.choice((dtype, dtype, "fp8"))
    page = rng.choice((4096, 5120, 8192))
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 5, 8, 32))
    heads = kv_heads * rng.choice((1, 1, 3, 4, 8) if kv_heads <= 8 else (1,))
    if op == "attend":
        words = rng.choice((1, 1, 2))
        hi = _spread(rng, 2, 64 * words)
        kv_hi = max(_spread(rng, 17, 60000), hi)
        # as many sequences as keep the plain form's scores under 2.2 GB and its keys in 32 bits under 1.1 GB
        most = min(2.2e9 / (4.0 * heads * hi * kv_hi), 1.1e9 / (4.0 * kv_heads * dim * kv_hi))
        seqs = min(_spread(rng, 1, 64), max(1, int(most)))
        kv_lo = max(hi, rng.choice((1, kv_hi // 4, kv_hi)))
        window = rng.choice((0, 0, 0, _spread(rng, 16, 4096)))
        return _attend_case("", dtype, kv, page, heads, kv_heads, dim, seqs, (rng.choice((1, hi)), hi),
                            (min(kv_lo, kv_hi), kv_hi), words, lens, window)
    if op == "weigh":
        kv_hi = _spread(rng, 17, 60000)
        hi = rng.choice((1, 1, rng.randint(2, 8), _spread(rng, 9, 2048)))
        hi = min(hi, kv_hi)
        most = min(8e9 / (4.0 * heads * hi * kv_hi), 1.1e9 / (4.0 * kv_heads * dim * kv_hi))
        seqs = min(_spread(rng, 1, 64), max(1, int(most)))
        kv_lo = max(hi, rng.choice((1, kv_hi // 4, kv_hi)))
        window = rng.choice((0, 0, 0, _spread(rng, 16, 4096)))
        return _weigh_case("", dtype, kv, page, heads, kv_heads, dim, seqs, (rng.choice((1, hi)), hi),
                           (min(kv_lo, kv_hi), kv_hi), lens, window, rng.choice((1.0, 0.9, 0.0)))
    if op == "select":
        kv_hi = _spread(rng, 20, 131072)
        seqs = max(1, min(_spread(rng, 1, 64), 4000000 // (kv_hi * kv_heads)))
        budget = _spread(rng, 8, kv_hi)
        return _select_case("", kv_heads, seqs, (rng.choice((1, max(1, kv_hi // 4), kv_hi)), kv_hi), budget,
                            rng.choice((0, min(4, budget))), rng.randint(0, max(0, budget - 4)), lens)
    if rng.random() < 0.5:
        hi = _spread(rng, 2, 64)
        seqs = max(1, min(_spread(rng, 1, 64), 64 * 32 * 64 // (kv_heads * hi)))
        return _compact_case("", "path", dtype, kv, page, kv_heads, dim, seqs, (rng.choice((1, hi)), hi),
                             (hi, max(hi, 2000)), 0, lens)
    kv_hi = _spread(rng, 100, 30000)
    budget = _spread(rng, 16, max(17, kv_hi // 2))
    seqs = max(1, min(_spread(rng, 1, 64), 2000000 // (kv_hi * kv_heads), 16 * 8 * 2048 // (budget * kv_heads)))
    return _compact_case("", "evict", dtype, kv, page, kv_heads, dim, seqs, (1, 1),
                         (rng.choice((1, max(1, kv_hi // 4), kv_hi)), kv_hi), budget, lens)


def _lengths(case):
    """(q_len, kv_len) of every sequence: lengths follow the case, values the seed."""
    rng = random.Random(case["lens"])
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    q[rng.randrange(len(q))] = case["q_hi"]
    if "kv_hi" not in case:
        return q, q
    kv = [max(n, rng.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    at = rng.randrange(len(q))
    kv[at] = max(q[at], case["kv_hi"])
    return q, kv


def _geometry(case):
    """Bytes of a cached element, elements in 16 bytes, bytes of a page, tokens a page."""
    elt = 1 if case["kv"] == "fp8" else 2
    E, page_bytes = 16 // elt, 2 * case["page"]
    return elt, E, page_bytes, page_bytes // (case["dim"] * elt) // E * E


def work(case):
    q, kv = _lengths(case)
    n, op = sum(q), case["op"]
    if op == "build":
        return {"bytes": n * (8 + 8 * case["words"]), "flops": 0}
    if op == "verify":
        # one row of probabilities a sequence, and one of each drafted token
        size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
        return {"bytes": len(q) * case["vocab"] * size + n * (size + 20), "flops": 2 * len(q) * case["vocab"]}
    if op == "select":
        kept = sum(min(m, case["budget"]) for m in kv)
        return {"bytes": case["kv_heads"] * 4 * (sum(kv) + kept), "flops": case["kv_heads"] * sum(kv)}
    elt, _, _, _ = _geometry(case)
    row = case["kv_heads"] * case["dim"]
    scale = case["kv_heads"] if elt == 1 else 0
    if op == "compact":
        # a path of 4 tokens, of which the first is in its place; most evictions move every token
        kept = sum(min(m, case["budget"]) for m in kv) if case["what"] == "evict" else 3 * len(q)
        return {"bytes": kept * (4 * row * elt + 4 * scale + (12 * case["kv_heads"] if case["what"] == "evict" else 4)),
                "flops": 0}
    w = case["window"] or 1 << 40
    keys = pairs = 0
    for a, m in zip(q, kv):
        if op == "attend":      # a token sees what was there before, itself and about 3 ancestors
            keys += min(m - a, w) + a
            pairs += a * (min(m - a, w) + min(a, 4))
        else:
            keys += m - max(0, m - a + 1 - w)
            pairs += sum(min(p + 1, w) for p in range(m - a, m))
    if op == "attend":
        return {"bytes": keys * (2 * row * elt + 2 * scale) + n * (case["heads"] * (4 * case["dim"] + 4) + 8 * case["words"]),
                "flops": 4 * case["dim"] * case["heads"] * pairs}
    return {"bytes": keys * (row * elt + scale) + n * case["heads"] * (2 * case["dim"] + 4) + 8 * case["kv_heads"] * sum(kv),
            "flops": 2 * case["dim"] * case["heads"] * pairs}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _normal(shape, dtype, gen, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(q):
    return _ints(np.concatenate([[0], np.cumsum(q)]).tolist())


def _numbers(q_start, n):
    """Of every new token: its sequence and its number among the sequence's new ones."""
    i = torch.arange(n, device="cuda")
    s = torch.searchsorted(q_start.long(), i, right=True) - 1
    return s, i - q_start.long()[s]


def _parents(q_start, n, gen):
    """Parents that are as likely as each other: a tree of n tokens is about 2 ln n deep."""
    _, t = _numbers(q_start, n)
    up = torch.rand(n, device="cuda", generator=gen)
    parent = torch.minimum((t * up).long(), t - 1)
    return parent.to(torch.int32)


def _grid(q_start, n, most, values, empty):
    """values [n] of the new tokens as [sequences][most], `empty` where there are none."""
    s, t = _numbers(q_start, n)
    out = torch.full((q_start.shape[0] - 1, most), empty, dtype=values.dtype, device="cuda")
    out[s, t] = values
    return out


def _ancestors(parent):
    """[B][M] parents (a number below the token's own, else none) -> [B][M][M], a token its own too."""
    B, M = parent.shape
    t = torch.arange(M, device="cuda")
    jump = torch.where((parent >= 0) & (parent < t), parent.long(), torch.full_like(parent, M, dtype=torch.int64))
    jump = torch.cat([jump, torch.full((B, 1), M, dtype=torch.int64, device="cuda")], 1)
    sees = torch.eye(M + 1, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    sees[:, M] = False
    for _ in range(max(1, (M - 1).bit_length())):
        sees |= sees.gather(1, jump[:, :, None].expand(-1, -1, M + 1))
        jump = jump.gather(1, jump)
    return sees[:, :M, :M]


def _packed(sees, words):
    """[..][M] truth values -> [..][words] of 64 bits."""
    bits = torch.nn.functional.pad(sees, (0, 64 * words - sees.shape[-1])).to(torch.int64)
    return (bits.view(*sees.shape[:-1], words, 64) << torch.arange(64, device="cuda")).sum(-1)


def _tree_rows(q_start, n, most, parent, words, window=0):
    """(seen [n][words], depth [n]) of the tokens of all trees."""
    sees = _ancestors(_grid(q_start, n, most, parent, -1))
    depth = sees.sum(-1) - 1
    if window:
        sees &= depth[:, None, :] > depth[:, :, None] - window
    s, t = _numbers(q_start, n)
    return _packed(sees[s, t], words), depth[s, t].to(torch.int32)


def _tree_inputs(case, gen):
    q, _ = _lengths(case)
    n = sum(q)
    st = {"case": case, "n": n, "most": max(q), "q_start": _starts(q)}
    st["parent"] = _parents(st["q_start"], n, gen)
    st["seen"] = torch.empty((n, case["words"]), dtype=torch.int64, device="cuda")
    st["depth"] = torch.empty(n, dtype=torch.int32, device="cuda")
    return st


def _older(parent):
    """[B][M][M]: token u is an older child of token t's parent."""
    M = parent.shape[1]
    t = torch.arange(M, device="cuda")
    return (parent[:, :, None] == parent[:, None, :]) & (parent >= 0)[:, :, None] & (t[None] < t[:, None])[None]


def _draft_inputs(case, gen):
    q, _ = _lengths(case)
    n, dt, vocab, most = sum(q), DTYPES[case["dtype"]], case["vocab"], max(q)
    st = {"case": case, "n": n, "most": most, "q_start": _starts(q)}
    st["parent"] = _parents(st["q_start"], n, gen)
    # a few tokens of each row are likely, and the draft proposes these: about every second is accepted
    logits = _normal((n, vocab), torch.float32, gen, 1.0)
    hot = torch.randint(0, vocab, (n, 4), device="cuda", generator=gen)
    base = math.log(vocab) + 0.5
    peaks = torch.tensor([base + 0.7, base - 0.3, base - 0.8, base - 1.8], device="cuda").expand(n, 4)
    logits.scatter_reduce_(1, hot, peaks, "amax")
    st["target"] = torch.softmax(logits, -1).to(dt)
    del logits
    s, t = _numbers(st["q_start"], n)
    rank = _older(_grid(st["q_start"], n, most, st["parent"], -1)).sum(-1)[s, t]
    row = st["q_start"].long()[s] + st["parent"].long().clamp_min(0)
    some = torch.randint(0, vocab, (n,), device="cuda", generator=gen)
    st["drafted"] = torch.where(rank < 4, hot[row, rank.clamp_max(3)], some).to(torch.int32)
    st["u_accept"] = torch.rand(n, device="cuda", generator=gen)
    st["u_sample"] = torch.rand(len(q), device="cuda", generator=gen)
    st["tokens"] = torch.empty((len(q), most), dtype=torch.int32, device="cuda")
    st["path"] = torch.empty((len(q), most), dtype=torch.int32, device="cuda")
    st["n_out"] = torch.empty(len(q), dtype=torch.int32, device="cuda")
    return st


def _weights(shape, gen):
    """Sums of attention: over many powers of ten, some of them zero."""
    w = torch.exp(_normal(shape, torch.float32, gen, 2.0) - 4.0)
    return w.masked_fill_(torch.rand(shape, device="cuda", generator=gen) < 0.01, 0.0)


def _cache_inputs(case, gen):
    q, kv = _lengths(case)
    n, dt, op = sum(q), DTYPES[case["dtype"]], case["op"]
    elt, E, page_bytes, T = _geometry(case)
    H, D, B = case["kv_heads"], case["dim"], len(q)
    blocks = [-(-m // T) for m in kv]
    n_pages = sum(blocks) * 2 * H + 3
    # pages in no order; those that a window has left behind are given back
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(case["lens"] & 0xFFFF)).to(torch.int32)
    table = torch.full((B, 2, H, max(blocks)), -1, dtype=torch.int32)
    at = 0
    for s, b in enumerate(blocks):
        gone = max(0, kv[s] - q[s] + 1 - case["window"]) // T if case["window"] else 0
        table[s, :, :, gone:b] = order[at:at + 2 * H * (b - gone)].view(2, H, b - gone)
        at += 2 * H * b
    st = {"case": case, "table": table.cuda(), "q_start": _starts(q), "kv_len": _ints(kv), "max_q": max(q),
          "n": n, "T": T, "n_pages": n_pages, "most_kv": max(kv)}
    if op == "select":
        # its pages hold nothing that is looked at
        st["pages"] = torch.empty((n_pages, page_bytes), dtype=torch.uint8, device="cuda")
        st["scales"] = None
    elif elt == 1:
        pages = torch.empty((n_pages, page_bytes), dtype=torch.uint8, device="cuda")
        for i in range(0, n_pages, 8192):
            part = _normal((min(8192, n_pages - i), page_bytes), torch.bfloat16, gen, 100.0)
            pages[i:i + 8192] = part.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        st["pages"] = pages
        st["scales"] = torch.randint(118, 122, (n_pages, T), dtype=torch.uint8, device="cuda", generator=gen)
    else:
        st["pages"] = _normal((n_pages, page_bytes // 2), dt, gen).view(torch.uint8)
        st["scales"] = None
    if op in ("attend", "weigh"):
        st["q"] = _normal((n, case["heads"], D), dt, gen)
    if op == "attend":
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((n, case["heads"]), dtype=torch.float32, device="cuda")
        parent = _parents(st["q_start"], n, gen)
        st["seen"], st["depth"] = _tree_rows(st["q_start"], n, max(q), parent, case["words"], case["window"])
    elif op == "weigh":
        # about what attention of such rows gives: ln(tokens) + half the scores' variance
        s, t = _numbers(st["q_start"], n)
        sees = (st["kv_len"].long() - torch.diff(st["q_start"].long()))[s] + t + 1
        sees = sees.clamp_max(case["window"]) if case["window"] else sees
        spread = st["q"].float().square().mean(-1) * (1.1 if elt == 1 else 1.0)
        st["lse"] = torch.log(sees.float())[:, None] + 0.5 * spread
        st["before"] = _weights((B, H, max(kv)), gen)
        st["weights"] = torch.zeros((B, H, max(kv)), dtype=torch.float32, device="cuda")
    elif op == "select":
        st["weights"] = _weights((B, H, max(kv)), gen)
        st["keep"] = torch.full((B, H, case["budget"]), -1, dtype=torch.int32, device="cuda")
        st["n_keep"] = torch.empty(B, dtype=torch.int32, device="cuda")
    elif op == "compact" and case["what"] == "evict":
        st["weights"] = _weights((B, H, max(kv)), gen)
        st["keep"], st["n_keep"] = _chosen(st["weights"], st["kv_len"], case["budget"], 4, 16)
    elif op == "compact":
        # a path of the tree: from the first token to the one that a walk from a late token up finds
        parent = _grid(st["q_start"], n, max(q), _parents(st["q_start"], n, gen), -1)
        q_len = torch.diff(st["q_start"].long())
        at = (torch.rand(B, device="cuda", generator=gen) * q_len).long()
        on = _ancestors(parent)[torch.arange(B, device="cuda"), at]
        st["n_keep"] = on.sum(1).to(torch.int32)
        number = torch.arange(max(q), device="cuda").expand(B, -1)
        keep = torch.where(on, number, torch.full_like(number, 1 << 20)).sort(1)[0]
        st["keep"] = torch.where(keep < 1 << 20, keep, torch.full_like(keep, -1)).to(torch.int32)[:, None].contiguous()
        st["weights"] = None
    return st


def _chosen(weights, kv_len, budget, sinks, recent):
    """(keep [B][H][budget], -1 behind the last; n_keep [B]) of the first, the latest and the largest."""
    B, H, S = weights.shape
    j = torch.arange(S, device="cuda")
    n = kv_len.long()[:, None, None]
    rank = weights.masked_fill((j < sinks) | (j >= n - min(recent, max(0, budget - sinks))), math.inf)
    rank = rank.masked_fill(j >= n, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1]
    k = kv_len.clamp_max(budget)
    take = min(budget, S)
    order = torch.where(j[:take] < k.long()[:, None, None], order[..., :take], torch.full_like(order[..., :take], S))
    keep = order.sort(-1)[0]
    keep = torch.where(keep < S, keep, torch.full_like(keep, -1))
    keep = torch.nn.functional.pad(keep, (0, budget - take), value=-1)
    return keep.to(torch.int32), k


class _Pool:
    """The unified pool over a state's page memory, all of its pages taken for the cache."""

    def __init__(self, lib, st):
        case = st["case"]
        dt = lib.DTYPE_CODE[case["dtype"]]
        self.lib = lib
        self.handle = lib.lora_pool_create(case["page"], dt, st["n_pages"], 1, 8, [(64, 64)], pages_dev=st["pages"])
        lib.lora_pool_alloc_pages(self.handle, st["n_pages"])
        kv = lib.LORA_FP8_E4M3 if case["kv"] == "fp8" else dt
        self.cache = lib.KvCache(self.handle, case["kv_heads"], case["dim"], kv, scales=st["scales"])
        self.batch = lib.KvBatch(st["q_start"], st["kv_len"], st["table"], st["n"], st["max_q"])

    def __del__(self):
        try:
            self.lib.lora_pool_destroy(self.handle)
        except Exception:
            pass


def _space(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _calls(st):
    """What a serving program keeps: its pool, its workspace and its prepared call."""
    import gather_lora_matmul_amd as L
    case = st["case"]
    op = case["op"]
    if op == "build":
        st["call"] = L.prepare_kv_tree_build(st["q_start"], st["parent"], st["seen"], st["depth"], window=case["window"])
        return
    if op == "verify":
        ws = _space(L.lora_spec_verify_tree_workspace_size(case["seqs"], case["vocab"]))
        st["call"] = L.prepare_spec_verify_tree(st["q_start"], st["parent"], st["drafted"], st["target"], st["u_accept"],
                                                st["u_sample"], st["tokens"], st["path"], st["n_out"], ws)
        return
    pool = st["pool"] = _Pool(L, st)
    if op == "attend":
        ws = _space(L.lora_kv_attend_workspace_size(pool.cache, pool.batch, case["heads"]))
        st["call"] = L.prepare_kv_attend_tree(pool.cache, pool.batch, L.KvTree(st["seen"], st["depth"]), st["q"], st["out"],
                                              case["dim"] ** -0.5, window=case["window"], lse=st["lse"], workspace=ws)
    elif op == "weigh":
        ws = _space(L.lora_kv_weigh_workspace_size(pool.cache, pool.batch, case["heads"]))
        st["call"] = L.prepare_kv_weigh(pool.cache, pool.batch, st["q"], st["lse"], st["weights"], case["dim"] ** -0.5,
                                        window=case["window"], decay=case["decay"], before=st["before"], workspace=ws)
    elif op == "select":
        ws = _space(L.lora_kv_select_workspace_size(pool.cache, pool.batch))
        st["call"] = L.prepare_kv_select(pool.cache, pool.batch, st["weights"], case["budget"], st["keep"], st["n_keep"],
                                         sinks=case["sinks"], recent=case["recent"], workspace=ws)
    else:
        st["call"] = L.prepare_kv_compact(pool.cache, pool.batch, st["keep"], st["n_keep"],
                                          from_new=case["what"] == "path", weights=st["weights"])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"build": _tree_inputs, "verify": _draft_inputs}.get(case["op"], _cache_inputs)(case, gen)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        _calls(st)
    return st


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _build(st):
    case = st["case"]
    seen, depth = _tree_rows(st["q_start"], st["n"], st["most"], st["parent"], case["words"], case["window"])
    return {"seen": seen, "depth": depth}


def _power(byte):
    """The fp32 power of two of an exponent byte."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _dense(st, which):
    """K (0) or V (1) of every sequence in 32 bits, [B][H][blocks * T][D]."""
    case = st["case"]
    elt, E, page_bytes, T = _geometry(case)
    D, (B, _, H, nb) = case["dim"], st["table"].shape
    safe = st["table"][:, which].long().clamp_min(0)
    kind = torch.float8_e4m3fn if elt == 1 else DTYPES[case["dtype"]]
    got = st["pages"].view(torch.uint8)[safe, :T * D * elt].view(kind).float()
    if which == 0:
        x = got.view(B, H, nb, D // E, T, E).permute(0, 1, 2, 4, 3, 5).reshape(B, H, nb * T, D)
    else:
        x = got.view(B, H, nb, T // E, D, E).permute(0, 1, 2, 3, 5, 4).reshape(B, H, nb * T, D)
    if elt == 1:
        x = x * _power(st["scales"][safe]).view(B, H, nb * T, 1)
    return x


def _there(st):
    """[B][H][blocks * T]: tokens that have pages."""
    return (st["table"] >= 0).all(1).repeat_interleave(st["T"], dim=2)


def _queries(st):
    """[B][H][G * M][D] in 32 bits, and the rows' numbers."""
    case = st["case"]
    H, D, M = case["kv_heads"], case["dim"], st["max_q"]
    G, B = case["heads"] // H, st["table"].shape[0]
    t = torch.arange(M, device="cuda")
    rows = (st["q_start"].long()[:-1, None] + t).clamp_max(st["n"] - 1)
    q = st["q"].float()[rows].view(B, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * M, D)
    return q, rows, t


def _attend(st):
    case = st["case"]
    dt, D, H, W = DTYPES[case["dtype"]], case["dim"], case["kv_heads"], case["window"]
    G, M = case["heads"] // H, st["max_q"]
    k, v, there = _dense(st, 0), _dense(st, 1), _there(st)
    q, rows, t = _queries(st)
    B, S = k.shape[0], k.shape[2]
    q_len = torch.diff(st["q_start"].long())
    base = st["kv_len"].long() - q_len
    j = torch.arange(S, device="cuda")
    new = j - base[:, None]                                              # [B][S]
    bits = (st["seen"][rows][..., None] >> torch.arange(64, device="cuda")) & 1
    bits = bits.view(B, M, -1).bool()                                    # [B][M][64 words]
    at = new.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, M, -1)
    own_tree = bits.gather(2, at) & ((new >= 0) & (new < q_len[:, None]))[:, None]
    prefix = (new < 0)[:, None].expand(-1, M, -1)
    if W:
        prefix = prefix & (j > (base[:, None] + st["depth"].long()[rows])[:, :, None] - W)
    sees = ((own_tree | prefix)[:, None] & there[:, :, None]).unsqueeze(2)   # [B][H][1][M][S]
    x = (torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5).view(B, H, G, M, S)
    x = x.masked_fill_(~sees, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, H, G * M, S), v).view(B, H, G, M, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = torch.log(total) + top
    s, i = _numbers(st["q_start"], st["n"])
    out = out.permute(0, 3, 1, 2, 4).reshape(B, M, H * G, D)[s, i]
    return {"out": out.to(dt), "lse": lse[..., 0].permute(0, 3, 1, 2).reshape(B, M, H * G)[s, i]}


def _whole(p):
    """Probabilities as whole multiples of 2^-44, so that sums have one value in any order."""
    return (torch.nan_to_num(p, nan=0.0).clamp(0.0, 1.0) * float(ONE)).to(torch.int64)


def _level(total, u):
    part = (u.clamp(0.0, 1.0 - 2.0 ** -24) * 2.0 ** 31).to(torch.int64)
    return (total >> 31) * part + (((total & 0x7FFFFFFF) * part) >> 31)


def _verify(st):
    n, M = st["n"], st["most"]
    q_start = st["q_start"].long()
    B = q_start.shape[0] - 1
    s, t = _numbers(st["q_start"], n)
    parent = _grid(st["q_start"], n, M, st["parent"].long(), -1)
    token = _grid(st["q_start"], n, M, st["drafted"].long(), -1)
    row = (q_start[:-1, None] + parent.clamp_min(0)).clamp_max(n - 1)
    w = _whole(st["target"][row, token.clamp_min(0)].float())             # weight of each drafted token
    older = _older(parent)
    again = (older & (token[:, :, None] == token[:, None, :])).any(-1)    # refused before: no weight left
    w = torch.where(again, torch.zeros_like(w), w)
    left = (ONE - (older * w[:, None, :]).sum(-1)).clamp_min(0)
    good = (_level(left, _grid(st["q_start"], n, M, st["u_accept"], 0.0)) < w) & (parent >= 0)
    best = good & ~(older & good[:, None, :]).any(-1)                     # the first accepted child of its parent
    first = torch.zeros_like(best)
    first[:, 0] = _grid(st["q_start"], n, M, torch.ones_like(t), 0)[:, 0] > 0
    chain = best | first
    on = ~(_ancestors(parent) & ~chain[:, None, :]).any(-1) & chain       # all ancestors too
    count = on.sum(1)
    last = (on * torch.arange(M, device="cuda")).amax(1)
    p = st["target"][(q_start[:-1] + last).clamp_max(n - 1)].float()
    plain = _whole(p)
    refused = (parent == last[:, None]) & (parent >= 0)
    vocab = p.shape[1]
    kept = torch.nn.functional.pad(plain, (0, 1)).scatter(1, torch.where(refused, token, torch.full_like(token, vocab)), 0)
    kept = kept[:, :vocab]
    total = kept.sum(1, keepdim=True)
    kept = torch.where(total > 0, kept, plain)
    total = kept.sum(1)
    new = (kept.cumsum(1) > _level(total, st["u_sample"])[:, None]).to(torch.int32).argmax(1)
    new = torch.where(total > 0, new, torch.full_like(new, -1))
    number = torch.arange(M, device="cuda").expand(B, -1)
    path = torch.where(on, number, torch.full_like(number, M)).sort(1)[0]
    path = torch.where(path < M, path, torch.full_like(path, -1))
    out = token.gather(1, torch.nn.functional.pad(path[:, 1:], (0, 1), value=-1).clamp_min(0))
    out = torch.where(number < (count - 1)[:, None], out, torch.full_like(out, -1))
    out = torch.where(number == (count - 1)[:, None], new[:, None], out)
    return {"tokens": out.to(torch.int32), "path": path.to(torch.int32), "n_out": count.to(torch.int32)}


def _weigh(st):
    case = st["case"]
    D, H, W = case["dim"], case["kv_heads"], case["window"]
    G, M = case["heads"] // H, st["max_q"]
    k, there = _dense(st, 0), _there(st)
    q, rows, t = _queries(st)
    B, S = k.shape[0], k.shape[2]
    q_len = torch.diff(st["q_start"].long())
    base = st["kv_len"].long() - q_len
    j = torch.arange(S, device="cuda")
    pos = base[:, None] + t                                              # [B][M]
    sees = (j <= pos[:, :, None]) & (t < q_len[:, None])[:, :, None]
    if W:
        sees &= j > pos[:, :, None] - W
    x = (torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5).view(B, H, G, M, S)
    lse = st["lse"][rows].view(B, M, H, G).permute(0, 2, 3, 1)
    x = x.sub_(lse[..., None]).exp_().masked_fill_(~sees[:, None, None], 0.0)
    got = x.sum((2, 3)) * there                                          # [B][H][S]
    n = st["most_kv"]
    got = got[..., :n]
    old = torch.where(j[:n] < base[:, None, None], st["before"] * case["decay"], torch.zeros_like(st["before"]))
    return {"weights": torch.where(j[:n] < st["kv_len"][:, None, None], (old + got) * there[..., :n], st["weights"])}


def _select(st):
    case = st["case"]
    keep, n_keep = _chosen(st["weights"], st["kv_len"], case["budget"], case["sinks"], case["recent"])
    return {"keep": keep, "n_keep": n_keep}


def _places(st, s, h, pos):
    """Flat places, in elements of the cache, of K and V [n][D] of tokens (s, h, pos) [n], and of their scales."""
    case = st["case"]
    elt, E, page_bytes, T = _geometry(case)
    D, size = case["dim"], page_bytes // elt
    page = st["table"].long()[s, :, h, pos // T]                          # [n][2]
    slot, d = (pos % T)[:, None], torch.arange(D, device="cuda")[None]
    k = ((d // E) * T + slot) * E + d % E
    v = ((slot // E) * D + d) * E + slot % E
    return page[:, :1] * size + k, page[:, 1:] * size + v, page * T + slot


def _cache_of(st):
    if st["case"]["kv"] == "fp8":
        out = {"pages": st["pages"].view(torch.float8_e4m3fn), "scales": st["scales"]}
    else:
        out = {"pages": st["pages"].view(DTYPES[st["case"]["dtype"]])}
    if st["weights"] is not None:
        out["weights"] = st["weights"]
    return out


def _compact(st):
    case = st["case"]
    B, _, H, _ = st["table"].shape
    i = torch.arange(st["keep"].shape[2], device="cuda")
    there = (i < st["n_keep"][:, None])[:, None].expand(B, H, -1)
    s, h, i = there.nonzero(as_tuple=True)
    first = st["kv_len"].long() - torch.diff(st["q_start"].long()) if case["what"] == "path" else torch.zeros_like(st["kv_len"].long())
    keep = st["keep"].long().expand(B, H, -1)[s, h, i]
    src, dst = first[s] + keep, first[s] + i
    flat = st["pages"].view(torch.uint8 if case["kv"] == "fp8" else torch.int16).view(-1)
    ks, vs, fs = _places(st, s, h, src)
    kd, vd, fd = _places(st, s, h, dst)
    k, v = flat[ks], flat[vs]
    flat[kd] = k
    flat[vd] = v
    if case["kv"] == "fp8":
        scales = st["scales"].view(-1)
        scales[fd] = scales[fs]
    if st["weights"] is not None:
        st["weights"][s, h, dst] = st["weights"][s, h, src]
    return _cache_of(st)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"build": _build, "attend": _attend, "verify": _verify, "weigh": _weigh, "select": _select,
                "compact": _compact}[op](state)
    state["call"]()
    if op == "compact":
        return _cache_of(state)
    names = {"build": ("seen", "depth"), "attend": ("out", "lse"), "verify": ("tokens", "path", "n_out"),
             "weigh": ("weights",), "select": ("keep", "n_keep")}[op]
    return {name: state[name] for name in names}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, one sequence after another
# ---------------------------------------------------------------------------------------------
def _e4m3():
    """The values of the 256 FP8 E4M3 codes."""
    values = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = math.nan if e == 15 and m == 7 else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        values.append(-x if c & 128 else x)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _tokens_of(st, s, which, head, m, values):
    """Cached keys (which 0) or values (1) of the first m tokens of one sequence and head, [m][D]."""
    case = st["case"]
    elt, E, page_bytes, T = _geometry(case)
    D = case["dim"]
    ids = st["table"][s, which, head, :-(-m // T)].long()
    raw = st["pages"].view(torch.uint8)[ids.clamp_min(0), :T * D * elt].contiguous()
    x = values[raw.long()] if elt == 1 else raw.view(DTYPES[case["dtype"]]).double()
    if which == 0:
        x = x.view(-1, D // E, T, E).transpose(1, 2).reshape(-1, D)
    else:
        x = x.view(-1, T // E, D, E).transpose(2, 3).reshape(-1, D)
    if elt == 1:
        x = x * torch.exp2(st["scales"][ids.clamp_min(0)].double() - 127).view(-1, 1)
    return x[:m], (ids >= 0).repeat_interleave(T)[:m]


def _exact_build(st):
    q, _ = _lengths(st["case"])
    parent, words, window = st["parent"].tolist(), st["case"]["words"], st["case"]["window"]
    seen, depth, at = [], [], 0
    for n in q:
        chains = []
        for t in range(n):
            p = parent[at + t]
            chains.append((chains[p] if 0 <= p < t else []) + [t])
            bits = sum(1 << u for u in (chains[t][-window:] if window else chains[t]))
            row = [bits >> 64 * w & (1 << 64) - 1 for w in range(words)]
            seen.append([x - (1 << 64) if x >> 63 else x for x in row])
            depth.append(len(chains[t]) - 1)
        at += n
    return {"seen": torch.tensor(seen, dtype=torch.int64), "depth": torch.tensor(depth, dtype=torch.int32)}


def _exact_attend(st):
    case = st["case"]
    q_len, kv_len = _lengths(case)
    H, D, W, values = case["kv_heads"], case["dim"], case["window"], _e4m3()
    G = case["heads"] // H
    out = torch.zeros((st["n"], case["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((st["n"], case["heads"]), dtype=torch.float64, device="cuda")
    rows, depths = st["seen"].tolist(), st["depth"].tolist()
    at = 0
    for s, (n, m) in enumerate(zip(q_len, kv_len)):
        sees = np.zeros((n, m), bool)
        for t in range(n):
            sees[t, max(0, m - n + depths[at + t] + 1 - W) if W else 0:m - n] = True
            for u in range(n):
                sees[t, m - n + u] = rows[at + t][u // 64] >> (u % 64) & 1
        sees = torch.from_numpy(sees).cuda()
        for h in range(H):
            k, there = _tokens_of(st, s, 0, h, m, values)
            v, _ = _tokens_of(st, s, 1, h, m, values)
            hidden = ~(sees & there)
            v = torch.where(there[:, None], v, torch.zeros_like(v))
            for g in range(h * G, h * G + G):
                x = (st["q"][at:at + n, g].double() @ k.T.contiguous()) / math.sqrt(D)
                x.masked_fill_(hidden, -math.inf)
                lse[at:at + n, g] = torch.logsumexp(x, 1)
                out[at:at + n, g] = torch.nan_to_num(torch.softmax(x, 1), nan=0.0) @ v
        at += n
    return {"out": out, "lse": lse}


def _units(p):
    """Probabilities (an array) as whole numbers of 2^-44."""
    p = np.nan_to_num(np.asarray(p, np.float64), nan=0.0)
    return np.floor(np.clip(p, 0.0, 1.0) * 2.0 ** 44).astype(np.int64)


def _exact_verify(st):
    q_start, parent, drafted = (st[x].tolist() for x in ("q_start", "parent", "drafted"))
    u, us = st["u_accept"].cpu().numpy(), st["u_sample"].cpu().numpy()
    tokens, path = (np.full((len(q_start) - 1, st["most"]), -1, np.int64) for _ in range(2))
    counts = []
    for s in range(len(q_start) - 1):
        a, n = q_start[s], q_start[s + 1] - q_start[s]
        at, taken, walking = 0, [0], True
        while walking:
            walking, gone = False, []
            left = 1 << 44
            w = _units(st["target"][a + at].float().cpu().numpy())
            raw = w.copy()
            for t in range(at + 1, n):
                if parent[a + t] != at:
                    continue
                x = drafted[a + t]
                if left * int(math.floor(float(u[a + t]) * 2 ** 31)) >> 31 < int(w[x]):
                    tokens[s, len(taken) - 1] = x
                    taken.append(t)
                    at, walking = t, True
                    break
                left = max(0, left - int(w[x]))
                w[x] = 0
        w = w if w.sum() else raw
        sums = np.cumsum(w)
        level = int(sums[-1]) * int(math.floor(float(us[s]) * 2 ** 31)) >> 31
        tokens[s, len(taken) - 1] = int(np.searchsorted(sums, level, side="right")) if sums[-1] else -1
        path[s, :len(taken)] = taken
        counts.append(len(taken))
    return {"tokens": torch.from_numpy(tokens).to(torch.int32), "path": torch.from_numpy(path).to(torch.int32),
            "n_out": torch.tensor(counts, dtype=torch.int32)}


def _exact_weigh(st):
    case = st["case"]
    q_len, kv_len = _lengths(case)
    H, D, W, values = case["kv_heads"], case["dim"], case["window"], _e4m3()
    G = case["heads"] // H
    weights = st["weights"].double()
    at = 0
    for s, (n, m) in enumerate(zip(q_len, kv_len)):
        pos = torch.arange(m - n, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None]
        causal = (j <= pos) & (j > pos - W) if W else j <= pos
        for h in range(H):
            k, there = _tokens_of(st, s, 0, h, m, values)
            total = torch.zeros(m, dtype=torch.float64, device="cuda")
            total[:m - n] = st["before"][s, h, :m - n].double() * case["decay"]
            for g in range(h * G, h * G + G):
                x = (st["q"][at:at + n, g].double() @ k.T.contiguous()) / math.sqrt(D)
                x = torch.exp(x - st["lse"][at:at + n, g].double()[:, None])
                total += torch.where(causal, x, torch.zeros_like(x)).sum(0)
            weights[s, h, :m] = torch.where(there, total, torch.zeros_like(total))
        at += n
    return {"weights": weights}


def _exact_select(st):
    case = st["case"]
    _, kv_len = _lengths(case)
    weights = st["weights"].cpu().numpy()
    keep = np.full(tuple(st["keep"].shape), -1, np.int32)
    for s, m in enumerate(kv_len):
        k = min(m, case["budget"])
        for h in range(case["kv_heads"]):
            rank = weights[s, h, :m].copy()
            rank[:case["sinks"]] = np.inf
            rank[max(0, m - case["recent"]):] = np.inf
            keep[s, h, :k] = np.sort(np.lexsort((np.arange(m), -rank))[:k])
    return {"keep": torch.from_numpy(keep), "n_keep": torch.tensor([min(m, case["budget"]) for m in kv_len], dtype=torch.int32)}


def _exact_compact(st):
    """The cache after the moves, sequence by sequence, head by head."""
    case = st["case"]
    elt, E, page_bytes, T = _geometry(case)
    q_len, kv_len = _lengths(case)
    D, values = case["dim"], _e4m3()
    raw = st["pages"].view(torch.uint8)
    pages = values[raw.long()] if elt == 1 else raw.view(DTYPES[case["dtype"]]).double()
    scales = st["scales"].clone() if elt == 1 else None
    weights = st["weights"].double() if st["weights"] is not None else None
    table, keeps, counts = st["table"].cpu().numpy(), st["keep"].cpu().numpy(), st["n_keep"].tolist()
    for s, (n, m) in enumerate(zip(q_len, kv_len)):
        first = m - n if case["what"] == "path" else 0
        for h in range(case["kv_heads"]):
            src = first + keeps[s, h % keeps.shape[1], :counts[s]].astype(np.int64)
            dst = first + np.arange(counts[s])
            for which in (0, 1):
                page = table[s, which, h]
                a, b = (torch.from_numpy(np.stack([page[x // T].astype(np.int64), x % T])).cuda() for x in (src, dst))
                body = pages[:, :T * D].view(-1, D // E, T, E) if which == 0 else pages[:, :T * D].view(-1, T // E, D, E)
                if which == 0:
                    body[b[0], :, b[1]] = body[a[0], :, a[1]]
                else:
                    body[b[0], b[1] // E, :, b[1] % E] = body[a[0], a[1] // E, :, a[1] % E]
                if scales is not None:
                    scales[b[0], b[1]] = scales[a[0], a[1]]
            if weights is not None:
                weights[s, h, torch.from_numpy(dst).cuda()] = weights[s, h, torch.from_numpy(src).cuda()]
    out = {"pages": pages}
    if scales is not None:
        out["scales"] = scales
    if weights is not None:
        out["weights"] = weights
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    return {"build": _exact_build, "attend": _exact_attend, "verify": _exact_verify, "weigh": _exact_weigh,
            "select": _exact_select, "compact": _exact_compact}[case["op"]](st)
