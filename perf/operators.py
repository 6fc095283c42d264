"""The KV-cache operators of the unified page pool, as cases that can be timed and checked.

Four operators that a multi-adapter serving step needs next to its LoRA products:

  write    new keys and values go to their places in the pool's pages, 16-bit as they are or
           quantised to FP8 E4M3 with one power-of-two scale per token and head
  read     the cached keys and values of a run of tokens, back in dense 16-bit rows
  attend   attention of each sequence's new tokens (one, a few drafted ones or a chunk) over its
           paged cache, causal, optionally within a sliding window
  verify   drafted tokens accepted or rejected against the target's probabilities, and the token
           that follows them, from given uniform numbers

A sequence s has q_len new tokens, rows q_start[s] .. q_start[s + 1] of the new tensors, at
positions kv_len[s] - q_len .. kv_len[s] - 1.  table[s][0 = K, 1 = V][head][b] is the pool page of
tokens b * T .. (b + 1) * T - 1 of one head (T tokens a page, -1: no page, its tokens are masked).
With E elements in 16 bytes, element d of token slot t of a K page is at ((d / E) * T + t) * E
+ d % E, and of a V page at ((t / E) * D + d) * E + t % E.

Sizes are those of this repository's workloads (32 heads of 128 at d = 4096, 40 at d = 5120, and
64 query heads over 8 key heads at d = 8192; a page is one d-row) or generic.
"""
import math
import random

import numpy as np
import torch

own = False

FIX = 44             # probabilities are summed as whole multiples of 2^-44
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _cache(op, name, dtype, kv, page, heads, kv_heads, dim, seqs, q, kv_len, lens, window=0):
    """q, kv_len: (shortest, longest) of the sequences; lens seeds their lengths."""
    return {"op": op, "name": name, "dtype": dtype, "kv": kv, "page": page, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "seqs": seqs, "q_lo": q[0], "q_hi": q[1],
            "kv_lo": kv_len[0], "kv_hi": kv_len[1], "lens": lens, "window": window}


def _drafts(name, dtype, vocab, seqs, lo, hi, lens):
    return {"op": "verify", "name": name, "dtype": dtype, "vocab": vocab, "seqs": seqs, "q_lo": lo + 1,
            "q_hi": hi + 1, "lens": lens}


def listed():
    return [
        # a decode step of 64 requests appends one token each (32 heads of 128, page = one 4096-row)
        _cache("write", "write_decode", "f16", "f16", 4096, 32, 32, 128, 64, (1, 1), (1, 2048), 1),
        # a prefill of 32 requests, 40 heads of 128, quantised into FP8 pages of 80 tokens
        _cache("write", "write_prefill_fp8", "bf16", "fp8", 5120, 40, 40, 128, 32, (32, 600), (32, 2000), 2),
        # a shared prefix is taken out of the cache
        _cache("read", "read_prefix", "bf16", "bf16", 8192, 64, 8, 128, 1, (4001, 4001), (4001, 4001), 3),
        # the caches of 16 requests that move to another engine, from FP8
        _cache("read", "read_requests_fp8", "f16", "fp8", 4096, 32, 32, 128, 16, (200, 3000), (200, 3000), 4),
        # the first tokens of one conversation: the smallest call, where latency counts
        _cache("attend", "attend_one", "f16", "f16", 4096, 32, 32, 128, 1, (1, 1), (517, 517), 5),
        # a decode step of 64 requests, every query head with its own keys
        _cache("attend", "attend_decode", "bf16", "bf16", 4096, 32, 32, 128, 64, (1, 1), (20, 2048), 6),
        # decode of long documents with shared heads and an FP8 cache
        _cache("attend", "attend_long_fp8", "bf16", "fp8", 8192, 64, 8, 128, 3, (1, 1), (40001, 131071), 7),
        # a verification step: 4 drafted tokens and the last accepted one of 32 requests
        _cache("attend", "attend_drafts", "bf16", "bf16", 8192, 64, 8, 128, 32, (5, 5), (900, 4100), 8),
        # one chunk of a long prompt
        _cache("attend", "attend_chunk", "bf16", "bf16", 8192, 64, 8, 128, 1, (2048, 2048), (16384, 16384), 9),
        # chunks and single tokens in one batch, window of 1000 tokens, pages of 80 tokens, 3 queries a head
        _cache("attend", "attend_mixed_window", "f16", "f16", 5120, 15, 5, 64, 32, (1, 255), (300, 4093), 10, 1000),
        # 4 drafted tokens of one request
        _drafts("verify_one", "f32", 32000, 1, 4, 4, 11),
        # 128 requests with none to 7 drafted tokens over an odd vocabulary
        _drafts("verify_batch", "f32", 131071, 128, 0, 7, 12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    op = rng.choice(("write", "read", "attend", "attend", "attend", "verify"))
    if op == "verify":
        lo = rng.choice((0, 0, 1, 3))
        return _drafts("", rng.choice(("f32", "f32", "f16", "bf16")), _spread(rng, 1000, 131072), _spread(rng, 1, 128),
                       lo, rng.randint(max(lo, 1), 7), lens)
    dtype = rng.choice(("f16", "bf16"))
    kv = rng.choice((dtype, dtype, "fp8"))
    page = rng.choice((4096, 5120, 8192))
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 5, 8, 32))
    heads = kv_heads * rng.choice((1, 1, 3, 4, 8) if kv_heads <= 8 else (1,))
    if op != "attend":
        # at most about 8192 tokens of 40 heads
        hi = _spread(rng, 1, 2000)
        seqs = min(_spread(rng, 1, 64), max(1, 8192 * 40 // (hi * kv_heads)))
        lo = rng.choice((1, max(1, hi // 4), hi))
        return _cache(op, "", dtype, kv, page, heads, kv_heads, dim, seqs, (lo, hi), (lo, max(hi, 2000)), lens)
    form = rng.choice(("token", "drafts", "chunk"))
    kv_hi = _spread(rng, 17, 60000)
    if form == "token":
        q = (1, 1)
    elif form == "drafts":
        q = (rng.choice((1, 3)), rng.randint(3, 8))
    else:
        hi = min(_spread(rng, 9, 2048), kv_hi)
        q = (rng.choice((1, hi)), hi)
    kv_hi = max(kv_hi, q[1])
    # as many sequences as keep the plain form's scores under 8 GB and its keys in 32 bits under 1.1 GB
    most = min(8e9 / (4.0 * heads * q[1] * kv_hi), 1.1e9 / (4.0 * kv_heads * dim * kv_hi))
    seqs = min(_spread(rng, 1, 64), max(1, int(most)))
    kv_lo = max(q[1], rng.choice((1, kv_hi // 4, kv_hi)))
    window = rng.choice((0, 0, 0, _spread(rng, 16, 4096)))
    return _cache("attend", "", dtype, kv, page, heads, kv_heads, dim, seqs, q, (min(kv_lo, kv_hi), kv_hi), lens, window)


def _lengths(case):
    """(q_len, kv_len) of every sequence: lengths follow the case, values the seed."""
    rng = random.Random(case["lens"])
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    q[rng.randrange(len(q))] = case["q_hi"]
    if case["op"] == "verify":
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
    if case["op"] == "verify":
        size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
        # one row of the target's probabilities a sequence, and one of the draft's where a token is
        # refused (of drafts that are accepted about 7 times in 10)
        rows = sum(2 - 0.7 ** (n - 1) for n in q)
        return {"bytes": rows * case["vocab"] * size + 24 * sum(q), "flops": 3 * rows * case["vocab"]}
    elt, _, _, _ = _geometry(case)
    row = case["kv_heads"] * case["dim"]
    if case["op"] in ("write", "read"):
        scales = 2 * case["kv_heads"] if elt == 1 else 0
        return {"bytes": sum(q) * (2 * row * (2 + elt) + scales), "flops": sum(q) * 2 * row * (2 if elt == 1 else 0)}
    pairs = keys = 0
    w = case["window"] or 1 << 40
    for n, m in zip(q, kv):
        keys += m - max(0, m - n + 1 - w)
        pairs += sum(min(p + 1, w) for p in range(m - n, m))
    cached = keys * (2 * row * elt + (2 * case["kv_heads"] if elt == 1 else 0))
    return {"bytes": cached + sum(q) * case["heads"] * (4 * case["dim"] + 4), "flops": 4 * case["dim"] * case["heads"] * pairs}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _normal(shape, dtype, gen, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(q):
    return _ints(np.concatenate([[0], np.cumsum(q)]).tolist())


def _draft_inputs(case, gen):
    q, _ = _lengths(case)
    n, dt, vocab = sum(q), DTYPES[case["dtype"]], case["vocab"]
    logits = _normal((n, vocab), torch.float32, gen, 2.0)
    drafts = [i for s, k in enumerate(q) for i in range(sum(q[:s]), sum(q[:s]) + k - 1)]
    rows = torch.tensor(drafts, dtype=torch.int64, device="cuda")
    near = logits[rows] + _normal((len(drafts), vocab), torch.float32, gen, 0.7)
    st = {"case": case, "q_start": _starts(q), "target": torch.softmax(logits, -1).to(dt)}
    del logits
    st["draft"] = torch.softmax(near, -1).to(dt)
    st["drafted"] = torch.zeros(0, dtype=torch.int32, device="cuda")
    if drafts:
        st["drafted"] = torch.multinomial(st["draft"].float(), 1, generator=gen)[:, 0].to(torch.int32)
    st["u_accept"] = torch.rand(len(drafts), device="cuda", generator=gen)
    st["u_sample"] = torch.rand(len(q), device="cuda", generator=gen)
    st["tokens"] = torch.empty(n, dtype=torch.int32, device="cuda")
    st["n_out"] = torch.empty(len(q), dtype=torch.int32, device="cuda")
    return st


def _cache_inputs(case, gen):
    q, kv = _lengths(case)
    n, dt = sum(q), DTYPES[case["dtype"]]
    elt, E, page_bytes, T = _geometry(case)
    H, D = case["kv_heads"], case["dim"]
    blocks = [-(-m // T) for m in kv]
    n_pages = sum(blocks) * 2 * H + 3
    # pages in no order; those that a window has left behind are given back
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(case["lens"] & 0xFFFF)).to(torch.int32)
    table = torch.full((len(q), 2, H, max(blocks)), -1, dtype=torch.int32)
    at = 0
    for s, b in enumerate(blocks):
        gone = max(0, kv[s] - q[s] + 1 - case["window"]) // T if case["window"] else 0
        table[s, :, :, gone:b] = order[at:at + 2 * H * (b - gone)].view(2, H, b - gone)
        at += 2 * H * b
    st = {"case": case, "table": table.cuda(), "q_start": _starts(q), "kv_len": _ints(kv), "max_q": max(q),
          "n": n, "T": T, "n_pages": n_pages}
    if elt == 1:
        pages = torch.empty((n_pages, page_bytes), dtype=torch.uint8, device="cuda")
        for i in range(0, n_pages, 8192):
            part = _normal((min(8192, n_pages - i), page_bytes), torch.bfloat16, gen, 100.0)
            pages[i:i + 8192] = part.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        st["pages"] = pages
        st["scales"] = torch.randint(118, 122, (n_pages, T), dtype=torch.uint8, device="cuda", generator=gen)
    else:
        st["pages"] = _normal((n_pages, page_bytes // 2), dt, gen).view(torch.uint8)
        st["scales"] = None
    if case["op"] == "attend":
        st["q"] = _normal((n, case["heads"], D), dt, gen)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((n, case["heads"]), dtype=torch.float32, device="cuda")
    elif case["op"] == "write":
        # rows of unequal size, as projections give them
        size = torch.exp(_normal((n, H, 1), torch.float32, gen, 1.0))
        st["k"] = (_normal((n, H, D), torch.float32, gen) * size).to(dt)
        st["v"] = (_normal((n, H, D), torch.float32, gen) * size).to(dt)
    else:
        st["k"] = torch.empty((n, H, D), dtype=dt, device="cuda")
        st["v"] = torch.empty_like(st["k"])
    return st


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


def _calls(st):
    """What a serving program keeps: its pool, its workspace and its prepared call."""
    import gather_lora_matmul_amd as L
    case = st["case"]
    if case["op"] == "verify":
        ws = torch.empty(L.lora_spec_verify_workspace_size(case["seqs"], case["vocab"]), dtype=torch.uint8, device="cuda")
        st["call"] = L.prepare_spec_verify(st["q_start"], st["drafted"], st["target"], st["draft"], st["u_accept"],
                                           st["u_sample"], st["tokens"], st["n_out"], ws)
        return
    pool = st["pool"] = _Pool(L, st)
    if case["op"] == "write":
        st["call"] = L.prepare_kv_write(pool.cache, pool.batch, st["k"], st["v"])
    elif case["op"] == "read":
        st["call"] = L.prepare_kv_read(pool.cache, pool.batch, st["k"], st["v"])
    else:
        need = L.lora_kv_attend_workspace_size(pool.cache, pool.batch, case["heads"])
        st["call"] = L.prepare_kv_attend(pool.cache, pool.batch, st["q"], st["out"], case["dim"] ** -0.5,
                                         window=case["window"], lse=st["lse"],
                                         workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return (_draft_inputs if case["op"] == "verify" else _cache_inputs)(case, gen)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        _calls(st)
    return st


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _rows(st):
    """Of every new token: its sequence, its number among the sequence's new ones, its position."""
    q_start = st["q_start"].long()
    i = torch.arange(st["n"], device="cuda")
    s = torch.searchsorted(q_start, i, right=True) - 1
    t = i - q_start[s]
    return s, t, st["kv_len"].long()[s] - (q_start[s + 1] - q_start[s]) + t


def _places(st):
    """Flat places, in elements of the cache, of K and V [n][H][D], and of their scales [n][H]."""
    case = st["case"]
    elt, E, page_bytes, T = _geometry(case)
    D, size = case["dim"], page_bytes // elt
    s, _, pos = _rows(st)
    page = st["table"].long()[s, :, :, pos // T]                       # [n][2][H]
    slot, d = (pos % T)[:, None], torch.arange(D, device="cuda")[None]
    k = ((d // E) * T + slot) * E + d % E
    v = ((slot // E) * D + d) * E + slot % E
    scale = page * T + slot[:, :, None]
    return page[:, 0, :, None] * size + k[:, None], page[:, 1, :, None] * size + v[:, None], scale[:, 0], scale[:, 1]


def _power(byte):
    """The fp32 power of two of an exponent byte."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _quantised(x):
    """(codes, exponent bytes): the smallest power of two with the row's largest value <= 448 of it."""
    x = x.float()
    frac, ex = torch.frexp(x.abs().amax(-1))
    e = (ex - 9 + (frac > 0.875).to(ex.dtype)).clamp(-126, 127)
    e = torch.where(frac == 0, torch.full_like(e, -126), e)
    return (x * _power(127 - e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _write(st):
    fp8 = st["case"]["kv"] == "fp8"
    kind = torch.uint8 if fp8 else DTYPES[st["case"]["dtype"]]
    flat = st["pages"].view(kind).view(-1)
    at_k, at_v, at_ks, at_vs = _places(st)
    k, v = st["k"], st["v"]
    if fp8:
        (k, ks), (v, vs) = _quantised(k), _quantised(v)
        st["scales"].view(-1)[at_ks] = ks
        st["scales"].view(-1)[at_vs] = vs
    flat[at_k] = k
    flat[at_v] = v
    return _cache_of(st)


def _cache_of(st):
    if st["case"]["kv"] == "fp8":
        return {"pages": st["pages"].view(torch.float8_e4m3fn), "scales": st["scales"]}
    return {"pages": st["pages"].view(DTYPES[st["case"]["dtype"]])}


def _read(st):
    dt = DTYPES[st["case"]["dtype"]]
    at_k, at_v, at_ks, at_vs = _places(st)
    if st["case"]["kv"] != "fp8":
        flat = st["pages"].view(dt).view(-1)
        return {"k": flat[at_k], "v": flat[at_v]}
    flat, scales = st["pages"].view(-1), st["scales"].view(-1)
    k = flat[at_k].view(torch.float8_e4m3fn).float() * _power(scales[at_ks])[..., None]
    v = flat[at_v].view(torch.float8_e4m3fn).float() * _power(scales[at_vs])[..., None]
    return {"k": k.to(dt), "v": v.to(dt)}


def _dense(st):
    """K and V of every sequence in 32 bits, [B][H][blocks * T][D], and which tokens have pages."""
    case = st["case"]
    elt, E, page_bytes, T = _geometry(case)
    D, (B, _, H, nb) = case["dim"], st["table"].shape
    table = st["table"].long()
    safe = table.clamp_min(0)
    kind = torch.float8_e4m3fn if elt == 1 else DTYPES[case["dtype"]]
    got = st["pages"].view(torch.uint8)[safe, :T * D * elt].view(kind).float()
    k = got[:, 0].view(B, H, nb, D // E, T, E).permute(0, 1, 2, 4, 3, 5).reshape(B, H, nb * T, D)
    v = got[:, 1].view(B, H, nb, T // E, D, E).permute(0, 1, 2, 3, 5, 4).reshape(B, H, nb * T, D)
    if elt == 1:
        scale = _power(st["scales"][safe]).view(B, 2, H, nb * T, 1)
        k, v = k * scale[:, 0], v * scale[:, 1]
    return k, v, (table >= 0).all(1).repeat_interleave(T, dim=2)


def _attend(st):
    case = st["case"]
    dt, D, H, W = DTYPES[case["dtype"]], case["dim"], case["kv_heads"], case["window"]
    G = case["heads"] // H
    k, v, there = _dense(st)
    B, M, S = k.shape[0], st["max_q"], k.shape[2]
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    t = torch.arange(M, device="cuda")
    q_len = q_start[1:] - q_start[:-1]
    rows = (q_start[:-1, None] + t).clamp_max(st["n"] - 1)
    q = st["q"].float()[rows].view(B, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * M, D)
    pos = (kv_len - q_len)[:, None] + t                                 # [B][M]
    j = torch.arange(S, device="cuda")
    seen = j <= pos[:, :, None]
    if W:
        seen &= j > pos[:, :, None] - W
    seen = (seen[:, None] & there[:, :, None]).unsqueeze(2)              # [B][H][1][M][S]
    x = (torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5).view(B, H, G, M, S)
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, H, G * M, S), v).view(B, H, G, M, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = torch.log(total) + top
    s, i, _ = _rows(st)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, M, H * G, D)[s, i]
    return {"out": out.to(dt), "lse": lse[..., 0].permute(0, 3, 1, 2).reshape(B, M, H * G)[s, i]}


def _fixed(p):
    """Probabilities as whole multiples of 2^-44, so that sums have one value in any order."""
    return (torch.nan_to_num(p, nan=0.0).clamp(0.0, 1.0) * 2.0 ** FIX).to(torch.int64)


def _verify(st):
    B = st["u_sample"].shape[0]
    M = st["case"]["q_hi"]
    q_start = st["q_start"].long()
    k = q_start[1:] - q_start[:-1] - 1                                   # drafted tokens of each sequence
    t = torch.arange(M, device="cuda")
    n, nd = st["target"].shape[0], st["draft"].shape[0]
    target, draft, drafted, u = st["target"], st["draft"], st["drafted"], st["u_accept"]
    row = (q_start[:-1, None] + t).clamp_max(n - 1)
    first = torch.zeros(B, dtype=torch.int64, device="cuda")
    seq = torch.arange(B, device="cuda")
    if nd:
        at = (q_start[:-1, None] - seq[:, None] + t).clamp_max(nd - 1)   # rows of the draft's tensors
        token = drafted.long()[at]
        good = u[at] * draft[at, token].float() < target[row, token].float()
        good &= t < k[:, None]
        first = good.to(torch.int64).cumprod(1).sum(1)
    p = target[row[seq, first]].float()
    rest = p
    if nd:
        against = draft[at[seq, first]].float()
        rest = torch.where((first < k)[:, None], p - against, p)
    rest = _fixed(rest)
    total = rest.sum(1, keepdim=True)
    rest = torch.where(total > 0, rest, _fixed(p))
    total = rest.sum(1)
    part = (st["u_sample"].clamp(0.0, 1.0 - 2.0 ** -24) * 2.0 ** 31).to(torch.int64)
    level = (total >> 31) * part + (((total & 0x7FFFFFFF) * part) >> 31)
    token = (rest.cumsum(1) > level[:, None]).to(torch.int32).argmax(1)
    token = torch.where(total > 0, token, torch.full_like(token, -1))
    i = torch.arange(n, device="cuda")
    s = torch.searchsorted(q_start, i, right=True) - 1
    t = i - q_start[s]
    out = token[s]
    if nd:
        out = torch.where(t < first[s], drafted.long()[(i - s).clamp_max(nd - 1)], out)
    out = torch.where(t > first[s], torch.full_like(out, -1), out)
    return {"tokens": out.to(torch.int32), "n_out": (first + 1).to(torch.int32)}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"write": _write, "read": _read, "attend": _attend, "verify": _verify}[op](state)
    state["call"]()
    if op == "write":
        return _cache_of(state)
    names = {"read": ("k", "v"), "attend": ("out", "lse"), "verify": ("tokens", "n_out")}[op]
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


def _exact_attend(st):
    case = st["case"]
    q_len, kv_len = _lengths(case)
    H, D, W, values = case["kv_heads"], case["dim"], case["window"], _e4m3()
    G = case["heads"] // H
    out = torch.zeros((st["n"], case["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((st["n"], case["heads"]), dtype=torch.float64, device="cuda")
    at = 0
    for s, (n, m) in enumerate(zip(q_len, kv_len)):
        pos = torch.arange(m - n, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None]
        causal = (j <= pos) & (j > pos - W) if W else j <= pos
        for h in range(H):
            k, there = _tokens_of(st, s, 0, h, m, values)
            v, _ = _tokens_of(st, s, 1, h, m, values)
            hidden = ~(causal & there)
            v = torch.where(there[:, None], v, torch.zeros_like(v))
            for g in range(h * G, h * G + G):
                x = (st["q"][at:at + n, g].double() @ k.T.contiguous()) / math.sqrt(D)
                x.masked_fill_(hidden, -math.inf)
                lse[at:at + n, g] = torch.logsumexp(x, 1)
                out[at:at + n, g] = torch.nan_to_num(torch.softmax(x, 1), nan=0.0) @ v
        at += n
    return {"out": out, "lse": lse}


def _exact_cache(st):
    """The cache after the write, or the rows that a read gives, token by token of one sequence."""
    case = st["case"]
    elt, E, page_bytes, T = _geometry(case)
    q_len, kv_len = _lengths(case)
    H, D, values = case["kv_heads"], case["dim"], _e4m3()
    if case["op"] == "read":
        k = torch.zeros((st["n"], H, D), dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        at = 0
        for s, (n, m) in enumerate(zip(q_len, kv_len)):
            for h in range(H):
                k[at:at + n, h] = _tokens_of(st, s, 0, h, m, values)[0][m - n:]
                v[at:at + n, h] = _tokens_of(st, s, 1, h, m, values)[0][m - n:]
            at += n
        return {"k": k, "v": v}
    raw = st["pages"].view(torch.uint8)
    pages = values[raw.long()] if elt == 1 else raw.view(DTYPES[case["dtype"]]).double()
    levels = torch.sort(values[:127])[0]
    at = 0
    for s, (n, m) in enumerate(zip(q_len, kv_len)):
        for which, x in ((0, st["k"]), (1, st["v"])):
            x = x[at:at + n].double()
            if elt == 1:
                top = x.abs().amax(-1, keepdim=True)
                e = torch.ceil(torch.log2(top / 448)).clamp(-126, 127)
                e = torch.where(torch.exp2(e) * 448 < top, e + 1, torch.where(torch.exp2(e - 1) * 448 >= top, e - 1, e))
                x = x / torch.exp2(e)
                # the nearer of the two neighbouring levels, the even one of two that are as near
                up = torch.searchsorted(levels, x.abs().contiguous()).clamp_max(126)
                low = (up - 1).clamp_min(0)
                a, b = x.abs() - levels[low], levels[up] - x.abs()
                x = torch.where((a < b) | ((a == b) & (low % 2 == 0)), levels[low], levels[up]) * torch.sign(x)
            for b0 in range((m - n) // T, -(-m // T)):
                lo, hi = max(m - n, b0 * T), min(m, b0 * T + T)
                page = st["table"][s, which, :, b0].long()
                part = pages[page, :T * D]                               # [H][T * D]
                part = part.view(H, D // E, T, E).transpose(1, 2) if which == 0 else part.view(H, T // E, D, E).transpose(2, 3)
                part = part.reshape(H, T, D).clone()
                part[:, lo - b0 * T:hi - b0 * T] = x[lo - (m - n):hi - (m - n)].transpose(0, 1)
                part = part.view(H, T, D // E, E).transpose(1, 2) if which == 0 else part.view(H, T // E, E, D).transpose(2, 3)
                pages[page, :T * D] = part.reshape(H, T * D)
        at += n
    return {"pages": pages, "scales": None} if elt == 1 else {"pages": pages}


def _exact_verify(st):
    q_start = st["q_start"].cpu().numpy()
    drafted, u, us = (st[x].cpu().numpy() for x in ("drafted", "u_accept", "u_sample"))
    tokens, counts = np.full(st["target"].shape[0], -1, np.int64), []
    for s in range(len(q_start) - 1):
        a, k = int(q_start[s]), int(q_start[s + 1] - q_start[s]) - 1
        done = 0
        while done < k:
            r, c = a - s + done, int(drafted[a - s + done])
            if not np.float32(u[r]) * np.float32(st["draft"][r, c].item()) < np.float32(st["target"][a + done, c].item()):
                break
            tokens[a + done] = c
            done += 1
        p = st["target"][a + done].float().cpu().numpy()
        rest = p - st["draft"][a - s + done].float().cpu().numpy() if done < k else p
        sums = np.cumsum(np.floor(np.clip(rest, 0, 1).astype(np.float64) * 2.0 ** FIX).astype(np.int64))
        if sums[-1] == 0:
            sums = np.cumsum(np.floor(np.clip(p, 0, 1).astype(np.float64) * 2.0 ** FIX).astype(np.int64))
        level = int(sums[-1]) * int(math.floor(float(us[s]) * 2 ** 31)) >> 31
        tokens[a + done] = int(np.searchsorted(sums, level, side="right")) if sums[-1] else -1
        counts.append(done + 1)
    return {"tokens": torch.from_numpy(tokens).to(torch.int32), "n_out": torch.tensor(counts, dtype=torch.int32)}


def exact(case, seed):
    st = _inputs(case, seed)
    return {"attend": _exact_attend, "verify": _exact_verify}.get(case["op"], _exact_cache)(st)
