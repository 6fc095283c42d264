"""KV cache in the unified pool: write, read and attention against plain
implementations in 64 bits, at the sizes and masks where they can go wrong.

Tolerances, derived from the operators' roundings:
  * write and read move bits or round to the nearest code: compared exactly;
  * attention: p is rounded to 16 bits (unit roundoff u = 2^-8 for bf16's 8-bit significand,
    2^-11 for f16's 11 bits; bf16 for FP8 caches) and the output once to its type, so an element is off by at most
    u_p * sum_j p_j |v_j| + u_out * |o|, plus fp32 arithmetic, for which a tenth of
    the first term is allowed;
  * lse: fp32 scores of dot products of D terms, within D * 2^-24 * scale * sum |q||k|
    (at most) of the value, plus 2^-21 of its size for exp, log and the sums.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gather_lora_matmul_amd as L
from gpu_helpers import log

TD = {"f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # unit roundoff of the format


class Case:
    """A pool with a cache, the tables of a few sequences and dense fp64 copies
    of what the cache holds."""

    def __init__(self, act, kv, page, Hkv, D, q_len, kv_len, seed=0, drop=(), extra_blocks=1, fp8_pool=False):
        self.act, self.fp8, self.H, self.D = act, kv == "fp8", Hkv, D
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt = L.DTYPE_CODE["e4m3" if fp8_pool else act]
        elt_pool = 1 if fp8_pool else 2
        self.page_bytes = page * elt_pool
        elt = 1 if self.fp8 else 2
        self.E = 16 // elt
        T = self.page_bytes // (D * elt) // self.E * self.E
        nb = max(1, max([-(-n // T) for n in kv_len] or [1]) + extra_blocks)
        need = len(q_len) * 2 * Hkv * nb
        self.n_pages = need + 7
        self.pages = torch.full((self.n_pages, self.page_bytes), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs
        self.pool = L.lora_pool_create(page, dt, self.n_pages, 1, 8, [(64, 64)], shuffle_seed=seed + 1,
                                       pages_dev=self.pages, act_dtype=L.DTYPE_CODE[act])
        code = L.LORA_FP8_E4M3 if self.fp8 else L.DTYPE_CODE[act]
        self.T, per, sb = L.lora_kv_layout(self.pool, Hkv, D, code)
        assert (self.T, per) == (T, 2 * Hkv)
        self.scales = torch.full((self.n_pages, T), 255, dtype=torch.uint8, device="cuda") if self.fp8 else None
        assert sb == (self.n_pages * T if self.fp8 else 0)
        self.cache = L.KvCache(self.pool, Hkv, D, code, scales=self.scales)
        ids = L.lora_pool_alloc_pages(self.pool, need)
        table = np.full((len(q_len), 2, Hkv, nb), -1, np.int32)
        at = 0
        for s, n in enumerate(kv_len):
            b = -(-n // T)
            table[s, :, :, :b] = ids[at:at + 2 * Hkv * b].reshape(2, Hkv, b)
            at += 2 * Hkv * b
        self.full_table = table.copy()
        for s, b in drop:
            table[s, :, :, b] = -1
        self.table_host = table
        self.table = torch.from_numpy(table).cuda()
        self.q_len, self.kv_len = list(q_len), list(kv_len)
        self.n = int(sum(q_len))
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)).cuda()
        self.kvl = torch.tensor(np.array(kv_len, np.int32)).cuda()
        self.rng = rng

    def batch(self, full=False, n=None, max_q=None):
        t = torch.from_numpy(self.full_table).cuda() if full else self.table
        return L.KvBatch(self.q_start, self.kvl, t, self.n if n is None else n,
                         max(self.q_len + [0]) if max_q is None else max_q)

    def fill(self, spread=1.0):
        """Write every sequence's whole cache; returns dense fp64 (k, v) lists as stored."""
        dt = TD[self.act]
        n = sum(self.kv_len)
        k = torch.empty((max(n, 1), self.H, self.D), dtype=dt, device="cuda").normal_(generator=self.gen)
        v = torch.empty_like(k).normal_(generator=self.gen)
        if spread != 1.0:
            k *= spread
        starts = torch.tensor(np.concatenate([[0], np.cumsum(self.kv_len)]).astype(np.int32)).cuda()
        b = L.KvBatch(starts, self.kvl, torch.from_numpy(self.full_table).cuda(), n, max(self.kv_len + [0]))
        L.lora_kv_write(self.cache, b, k, v)
        self.k, self.v = k, v
        kd, vd, at = [], [], 0
        for m in self.kv_len:
            x, y = k[at:at + m].double().cpu().numpy(), v[at:at + m].double().cpu().numpy()
            if self.fp8:
                x, y = dequant(*quant(x)), dequant(*quant(y))
            kd.append(x)
            vd.append(y)
            at += m
        self.kd, self.vd = kd, vd
        return kd, vd

    def close(self):
        L.lora_pool_destroy(self.pool)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        self.close()


def quant(x):
    """(codes, exponent) of rows x[..., D] by the rule, in 64 bits."""
    import workloads as W
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    top = fin.max(-1)
    with np.errstate(divide="ignore"):
        f, ex = np.frexp(top / 448.0)
    e = np.where(top > 0, ex - (f == 0.5), -126)  # smallest e with top <= 448 2^e
    e = np.clip(e, -126, 127).astype(np.int64)
    y = x * np.exp2(-e.astype(np.float64))[..., None]
    codes = W.quantize_e4m3(np.where(np.isfinite(y), y, 0.0))
    codes = np.where(np.isfinite(x), codes, 0x7F).astype(np.uint8)
    return codes, e


def dequant(codes, e):
    import workloads as W
    return W.dequantize(codes, "e4m3") * np.exp2(e.astype(np.float64))[..., None]


def slot_bytes(case, which, s, h, pos):
    """The stored bytes of one token's row, element by element in the documented order."""
    T, E, D = case.T, case.E, case.D
    pg = int(case.full_table[s, which, h, pos // T])
    t = pos % T
    d = np.arange(D)
    at = ((d // E) * T + t) * E + d % E if which == 0 else ((t // E) * D + d) * E + t % E
    row = case.host_pages[pg]
    return row[at] if case.fp8 else row.view(np.uint16)[at]


LAYOUTS = [
    # act, kv, page elements, kv heads, head dim: T of 32, 40, 64, 80 tokens, one group, a page with a tail
    ("f16", "f16", 4096, 3, 128), ("bf16", "bf16", 5120, 2, 128), ("bf16", "fp8", 5120, 2, 128),
    ("f16", "fp8", 4096, 1, 64), ("bf16", "bf16", 520, 2, 64), ("f16", "fp8", 1100 * 8, 3, 128),
]


@pytest.mark.parametrize("act,kv,page,H,D", LAYOUTS)
def test_write_places_and_read_back(act, kv, page, H, D):
    # lengths zero, one, page ends inside a group, several pages; appended in pieces of odd sizes
    kv_len = [0, 1, 7, 8, 41, 130, 97, 64]
    with Case(act, kv, page, H, D, [0] * 8, kv_len, seed=5) as c:
        log("[case] write/read %s %s page %d T %d" % (act, kv, page, c.T))
        n = sum(kv_len)
        dt = TD[act]
        # rows of a wider tensor (fused projection), unequal magnitudes, zeros
        wide = torch.empty((n, 3 * H, D), dtype=dt, device="cuda").normal_(generator=c.gen)
        wide *= torch.exp(2 * torch.randn((n, 3 * H, 1), device="cuda", generator=c.gen)).to(dt)
        k, v = wide[:, H:2 * H], wide[:, 2 * H:]
        k[n // 2] = 0
        v[3, 0, 1] = 0
        off = np.concatenate([[0], np.cumsum(kv_len)])
        done = [0] * 8
        step = 0
        before = c.pages.clone()
        while any(d < m for d, m in zip(done, kv_len)):
            take = [min(m - d, [1, 13, 50][(step + i) % 3]) for i, (d, m) in enumerate(zip(done, kv_len))]
            rows = np.concatenate([np.arange(off[i] + d, off[i] + d + t) for i, (d, t) in enumerate(zip(done, take))])
            done = [d + t for d, t in zip(done, take)]
            qs = torch.tensor(np.concatenate([[0], np.cumsum(take)]).astype(np.int32)).cuda()
            b = L.KvBatch(qs, torch.tensor(np.array(done, np.int32)).cuda(), torch.from_numpy(c.full_table).cuda(),
                          len(rows), max(take))
            buf = torch.empty((len(rows), 3 * H, D), dtype=dt, device="cuda")
            buf[:, H:] = wide[torch.from_numpy(rows).cuda()][:, H:]
            L.lora_kv_write(c.cache, b, buf[:, H:2 * H], buf[:, 2 * H:])
            step += 1
        torch.cuda.synchronize()
        c.host_pages = c.pages.cpu().numpy()
        scales = c.scales.cpu().numpy() if c.fp8 else None
        touched = np.zeros_like(c.host_pages, bool)
        for which, x in ((0, k), (1, v)):
            x = x.double().cpu().numpy()
            bits = (k if which == 0 else v).contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
            for s, m in enumerate(kv_len):
                for pos in range(m):
                    for h in range(H):
                        got = slot_bytes(c, which, s, h, pos)
                        if c.fp8:
                            codes, e = quant(x[off[s] + pos, h])
                            assert np.array_equal(got & 0x7F, codes & 0x7F) and np.array_equal(got, codes), (which, s, pos)
                            assert scales[c.full_table[s, which, h, pos // c.T], pos % c.T] == e + 127
                        else:
                            assert np.array_equal(got, bits[off[s] + pos, h]), (which, s, pos)
        # nothing else was written: the poison of free slots, tails and pages is whole
        used = {}
        for s, m in enumerate(kv_len):
            for which in (0, 1):
                for h in range(H):
                    for pos in range(m):
                        used.setdefault(int(c.full_table[s, which, h, pos // c.T]), set()).add((which, pos % c.T))
        elt = 1 if c.fp8 else 2
        for pg in range(c.n_pages):
            mark = np.zeros(c.page_bytes // elt, bool)
            for which, t in used.get(pg, ()):
                d = np.arange(D)
                at = ((d // c.E) * c.T + t) * c.E + d % c.E if which == 0 else ((t // c.E) * D + d) * c.E + t % c.E
                mark[at] = True
            free = ~np.repeat(mark, elt)
            free = np.concatenate([free, np.ones(c.page_bytes - free.size, bool)])
            assert np.all(c.host_pages[pg][free] == 0xFF), "page %d: bytes outside the tokens" % pg
        # read back the last tokens of every sequence, into rows of a wider tensor
        take = [min(m, 45 + i) for i, m in enumerate(kv_len)]
        qs = torch.tensor(np.concatenate([[0], np.cumsum(take)]).astype(np.int32)).cuda()
        b = L.KvBatch(qs, c.kvl, torch.from_numpy(c.full_table).cuda(), sum(take), max(take))
        out = torch.full((sum(take), 2 * H, D), 7.0, dtype=dt, device="cuda")
        L.lora_kv_read(c.cache, b, out[:, :H], out[:, H:])
        torch.cuda.synchronize()
        at = 0
        for s, (m, t) in enumerate(zip(kv_len, take)):
            for src, dst in ((k, out[:, :H]), (v, out[:, H:])):
                want = src[off[s] + m - t:off[s] + m]
                if c.fp8:
                    w = dequant(*quant(want.double().cpu().numpy()))
                    want = torch.from_numpy(w).to(torch.float32).to(dt).cuda()
                assert torch.equal(dst[at:at + t], want)
            at += t


def test_write_fp8_of_extreme_rows():
    # zeros, subnormals, the largest values, infinities and NaN
    with Case("bf16", "fp8", 4096, 1, 64, [0], [8], seed=2) as c:
        x = torch.zeros((8, 1, 64), dtype=torch.float32)
        x[1, 0, :] = 1e-39
        x[2, 0, 3] = 3.0e38
        x[3, 0, :] = torch.linspace(-448, 448, 64)
        x[4, 0, 5] = float("inf")
        x[4, 0, 6] = 2.0
        x[5, 0, 7] = float("nan")
        x[5, 0, 8] = -1.0
        x[6, 0, :] = float("-inf")
        x[7, 0, :] = 449.0
        xb = x.to(torch.bfloat16).cuda()
        qs = torch.tensor([0, 8], dtype=torch.int32).cuda()
        b = L.KvBatch(qs, c.kvl, torch.from_numpy(c.full_table).cuda(), 8, 8)
        L.lora_kv_write(c.cache, b, xb, xb)
        torch.cuda.synchronize()
        c.host_pages = c.pages.cpu().numpy()
        sc = c.scales.cpu().numpy()
        codes, e = quant(xb.double().cpu().numpy())
        for which in (0, 1):
            for t in range(8):
                got = slot_bytes(c, which, 0, 0, t)
                nan = (codes[t, 0] & 0x7F) == 0x7F
                assert np.array_equal(got[~nan], codes[t, 0][~nan]), (which, t)
                assert np.all((got[nan] & 0x7F) == 0x7F)
                assert sc[c.full_table[0, which, 0, 0], t] == e[t, 0] + 127


def test_write_and_read_skip_what_has_no_place():
    # a table with a missing page, a length shorter than the new tokens, ids past the pool
    with Case("bf16", "bf16", 4096, 2, 128, [5, 40, 3], [2, 70, 3], seed=3) as c:
        table = c.full_table.copy()
        table[1, :, :, 1] = -1
        table[2, :, :, 0] = c.n_pages
        dt = TD["bf16"]
        k = torch.randn((48, 2, 128), device="cuda", generator=c.gen).to(dt)
        v = torch.randn((48, 2, 128), device="cuda", generator=c.gen).to(dt)
        b = L.KvBatch(c.q_start, c.kvl, torch.from_numpy(table).cuda(), 48, 40)
        L.lora_kv_write(c.cache, b, k, v)
        ko, vo = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
        L.lora_kv_read(c.cache, b, ko, vo)
        torch.cuda.synchronize()
        for src, got in ((k, ko), (v, vo)):
            assert torch.all(got[:3] == 9.0)                       # positions -3 .. -1
            assert torch.equal(got[3:5], src[3:5])
            # sequence 1: tokens at positions 30 .. 69, block 1 (32 .. 63) missing
            assert torch.equal(got[5:7], src[5:7]) and torch.equal(got[39:45], src[39:45])
            assert torch.all(got[7:39] == 0)
            assert torch.all(got[45:] == 0)


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def reference(c, q, scale, window, there=None):
    """(out, lse, sum p|v|) in 64 bits; there[s]: bool [kv_len] of tokens with pages."""
    n, Hq, D = q.shape
    G = Hq // c.H
    out, lse, size = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D))
    slack = np.zeros((n, Hq))
    at = 0
    for s, (m, kl) in enumerate(zip(c.q_len, c.kv_len)):
        ok = np.ones(kl, bool) if there is None else there[s]
        for t in range(m):
            pos = kl - m + t
            j = np.arange(kl)
            see = (j <= pos) & ok
            if window:
                see &= j > pos - window
            if not see.any():
                continue
            for h in range(Hq):
                k, v = c.kd[s][see, h // G], c.vd[s][see, h // G]
                with np.errstate(invalid="ignore", over="ignore"):
                    x = scale * (k @ q[at + t, h])
                    mx = x.max()
                    p = np.exp(x - mx)
                    tot = p.sum()
                    out[at + t, h] = p @ v / tot
                    size[at + t, h] = p @ np.abs(v) / tot
                    lse[at + t, h] = mx + np.log(tot)
                    slack[at + t, h] = scale * (np.abs(k) @ np.abs(q[at + t, h])).max()
        at += m
    return out, lse, size, slack


def attend(c, q, scale, window=0, batch=None, lse=True, out=None, stream=None):
    b = batch or c.batch()
    n = L.lora_kv_attend_workspace_size(c.cache, b, q.shape[1])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 5.0) if out is None else out
    ls = torch.full((q.shape[0], q.shape[1]), 5.0, dtype=torch.float32, device="cuda") if lse else None
    L.lora_kv_attend(c.cache, b, q, out, scale, window=window, lse=ls, workspace=ws, stream=stream)
    return out, ls


def check(c, q, scale, window=0, there=None, got=None, what=""):
    out, lse = got or attend(c, q, scale, window)
    torch.cuda.synchronize()
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ro, rl, size, slack = reference(c, q.double().cpu().numpy(), scale, window, there)
    up = ROUND["bf16" if c.fp8 else c.act]
    tol = 1.1 * up * size + 1.01 * ROUND[c.act] * np.abs(ro) + 1e-7 * size + (2.0 ** -25 if c.act == "f16" else 0)
    fine = np.isfinite(ro)
    assert np.array_equal(np.isnan(o), np.isnan(ro)), what
    assert np.array_equal(o[~fine & ~np.isnan(ro)], ro[~fine & ~np.isnan(ro)]), what
    # scores off by d change p by a factor of e^d, d at most D * 2^-24 * slack
    d = np.expm1(2 * c.D * 2.0 ** -24 * slack)[..., None]
    bad = np.abs(o - ro)[fine] > (tol + d * size)[fine]
    assert not bad.any(), "%s: %d of %d off, worst %.3e" % (what, bad.sum(), bad.size,
                                                           np.max((np.abs(o - ro) / (tol + d * size + 1e-300))[fine]))
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), empty), what
    f = np.isfinite(rl)
    assert np.all(np.abs(l - rl)[f] <= (c.D * 2.0 ** -24 * slack + 2.0 ** -21 * np.maximum(1, np.abs(rl)))[f]), what
    return out, lse


KINDS = [("f16", "f16", 4096, 128), ("bf16", "bf16", 5120, 128), ("bf16", "fp8", 5120, 128), ("f16", "fp8", 4096, 128),
         ("f16", "f16", 5120, 64), ("bf16", "fp8", 8192, 64), ("bf16", "bf16", 520, 64)]


@pytest.mark.parametrize("act,kv,page,D", KINDS)
@pytest.mark.parametrize("H,G", [(1, 1), (2, 3), (1, 8), (1, 16)])
def test_attend_single_tokens(act, kv, page, D, H, G):
    # lengths around the tiles' and pages' ends; an idle sequence; q shorter than the cache
    kv_len = [1, 2, 31, 32, 33, 65, 128, 129, 257, 500, 3]
    q_len = [1] * 10 + [0]
    with Case(act, kv, page, H, D, q_len, kv_len, seed=11) as c:
        log("[case] single %s %s D %d H %d G %d T %d" % (act, kv, D, H, G, c.T))
        c.fill()
        q = torch.randn((c.n, H * G, D), device="cuda", generator=c.gen).to(TD[act])
        check(c, q, D ** -0.5)
        check(c, q, 0.3, window=40)


@pytest.mark.parametrize("act,kv,page,D", KINDS)
@pytest.mark.parametrize("H,G,q_len,kv_len,window", [
    (2, 1, [17, 1, 64, 65], [17, 90, 64, 300], 0),          # a prompt's beginning, a token, tiles and one more
    (1, 8, [5, 3, 4, 1], [5, 77, 200, 131], 0),              # drafted tokens: below and above 16 rows
    (1, 3, [130, 2, 43], [190, 2, 600], 0),                  # 390 rows: tiles of 128 that end inside a token
    (2, 4, [33, 70, 1], [100, 70, 280], 24),                 # windows shorter than a tile
    (1, 2, [100], [413], 150),
])
def test_attend_chunks(act, kv, page, D, H, G, q_len, kv_len, window):
    with Case(act, kv, page, H, D, q_len, kv_len, seed=12) as c:
        log("[case] chunk %s %s D %d H %d G %d" % (act, kv, D, H, G))
        c.fill()
        q = torch.randn((c.n, H * G, D), device="cuda", generator=c.gen).to(TD[act])
        check(c, q, D ** -0.5, window)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attend_long_split(kv):
    # one sequence over many blocks, and many short ones beside it
    q_len, kv_len = [1, 40] + [1] * 30, [20011, 9000] + [37] * 30
    with Case("bf16", kv, 8192, 1, 128, q_len, kv_len, seed=13) as c:
        log("[case] long %s" % kv)
        c.fill()
        q = torch.randn((c.n, 2, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        a = check(c, q, 128 ** -0.5)
        b = attend(c, q, 128 ** -0.5)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])   # the same bits again


def test_attend_many_sequences():
    rng = np.random.default_rng(3)
    q_len = [int(x) for x in rng.integers(0, 4, 700)]
    kv_len = [max(q, int(x)) for q, x in zip(q_len, rng.integers(0, 60, 700))]
    with Case("f16", "f16", 4096, 1, 128, q_len, kv_len, seed=14, extra_blocks=0) as c:
        log("[case] 700 sequences")
        c.fill()
        q = torch.randn((c.n, 2, 128), device="cuda", generator=c.gen).to(TD["f16"])
        check(c, q, 0.1)


@pytest.mark.parametrize("q_len", [[1, 1], [20, 30]])
@pytest.mark.parametrize("kv", ["f16", "fp8"])
def test_attend_rows_without_keys(q_len, kv):
    # more new tokens than the cache holds: those before position 0 see nothing; a cache of none;
    # a window whose pages were given back
    kv_len = [0, max(1, q_len[1] // 2)]
    with Case("f16", kv, 4096, 1, 128, q_len, kv_len, seed=15) as c:
        c.fill()
        q = torch.randn((c.n, 2, 128), device="cuda", generator=c.gen).to(TD["f16"])
        out, lse = check(c, q, 0.1)
        assert torch.all(out[:q_len[0]] == 0) and torch.all(torch.isneginf(lse[:q_len[0]]))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("q_len", [[1, 2], [50, 40]])
def test_attend_absent_pages(kv, q_len):
    kv_len = [400, 300]
    with Case("bf16", kv, 4096, 2, 128, q_len, kv_len, seed=16, drop=[(0, 0), (0, 3), (1, 1)]) as c:
        c.fill()
        there = []
        for s, m in enumerate(kv_len):
            ok = (c.table_host[s] >= 0).all((0, 1))
            there.append(np.repeat(ok, c.T)[:m])
        # a K page alone is missing, and one past the pool's end
        q = torch.randn((c.n, 4, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        check(c, q, 0.1, there=there)
        last = (m - 1) // c.T
        c.table[1, 0, :, last] = -1
        c.table[0, 1, :, 1] = c.n_pages + 5
        there[1][last * c.T:] = False
        there[0][c.T:2 * c.T] = False
        check(c, q, 0.1, there=there)


@pytest.mark.parametrize("kv", ["f16", "bf16", "fp8"])
@pytest.mark.parametrize("G,q_len", [(1, [1]), (2, [4]), (4, [40])])
def test_what_is_not_seen_has_no_influence(kv, G, q_len):
    # infinities and NaN behind the causal line, before the window and in free slots: rows that
    # see them get what the formula says, the others nothing
    act = "f16" if kv != "bf16" else "bf16"
    with Case(act, kv, 4096, 1, 128, q_len, [150], seed=17) as c:
        c.fill()
        q = torch.randn((c.n, G, 128), device="cuda", generator=c.gen).to(TD[act])
        new = c.v.clone()
        knew = c.k.clone()
        n = c.n
        new[149, 0, 3] = float("inf")
        new[150 - (n + 1) // 2, 0, 64] = float("nan")
        new[150 - (n + 1) // 2, 0, 100] = -float("inf")
        new[20, 0, 5] = float("nan")
        knew[149, 0, 7] = float("nan")
        starts = torch.tensor([0, 150], dtype=torch.int32).cuda()
        b = L.KvBatch(starts, c.kvl, torch.from_numpy(c.full_table).cuda(), 150, 150)
        if kv == "fp8":   # codes have no infinities
            new = torch.where(torch.isinf(new), torch.full_like(new, float("nan")), new)
        L.lora_kv_write(c.cache, b, knew, new)
        x, y = knew.double().cpu().numpy(), new.double().cpu().numpy()
        if c.fp8:
            x, y = dequant(*quant(x)), dequant(*quant(y))
        c.kd, c.vd = [x], [y]
        w = 100   # of 4 new tokens' windows token 20 is before all, of 40 only before the last ones'
        out, lse = attend(c, q, 0.05, w)
        torch.cuda.synchronize()
        o = out.double().cpu().numpy()
        ro, rl, size, slack = reference(c, q.double().cpu().numpy(), 0.05, w)
        # the last token's key is NaN: its own row is NaN
        assert np.isnan(o[-1]).all() and np.isnan(ro[-1]).all()
        assert np.array_equal(np.isnan(o), np.isnan(ro)) and np.array_equal(np.isinf(o), np.isinf(ro))
        inf = np.isinf(ro)
        assert np.array_equal(o[inf], ro[inf])
        if n > 1:
            if 150 - n - w >= 20:   # the first row sees none of them
                assert np.isfinite(o[0]).all()
            f = np.isfinite(ro)
            up = ROUND["bf16" if c.fp8 else act]
            tol = 1.1 * up * size + 1.01 * ROUND[act] * np.abs(ro) + 1e-6 * size + 2.0 ** -25
            assert np.all(np.abs(o - ro)[f] <= tol[f])


@pytest.mark.parametrize("q_len", [[1], [30]])
def test_attend_scores_of_all_sizes(q_len):
    # scores far apart, falling and rising along the keys (the running maximum moves late and often)
    with Case("bf16", "bf16", 4096, 1, 128, q_len, [600], seed=18) as c:
        c.fill()
        for slope in (-0.3, 0.3):
            k = c.k.clone()
            k[:, :, :] = 0
            k[:, 0, 0] = (torch.arange(600, device="cuda") * slope).to(k.dtype)
            k[:, 0, 1] = 1.0
            starts = torch.tensor([0, 600], dtype=torch.int32).cuda()
            b = L.KvBatch(starts, c.kvl, torch.from_numpy(c.full_table).cuda(), 600, 600)
            L.lora_kv_write(c.cache, b, k, c.v)
            c.kd = [k.double().cpu().numpy()]
            q = torch.zeros((c.n, 2, 128), device="cuda", dtype=TD["bf16"])
            q[:, :, 0] = 4.0
            q[:, 1, 1] = -3.0e4
            check(c, q, 1.0)


def test_attend_strides_streams_and_bounds():
    # q and out inside wider rows, another stream, a max_q_len below the truth, rows past the sequences
    with Case("bf16", "bf16", 8192, 2, 128, [3, 20], [50, 333], seed=19) as c:
        c.fill()
        wide = torch.randn((c.n + 2, 14, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        q = wide[:, 2:10]
        holder = torch.full((c.n + 2, 11, 128), 5.0, device="cuda", dtype=TD["bf16"])
        want, lse = check(c, q[:c.n].contiguous(), 0.09)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        b = c.batch(n=c.n + 2)
        with torch.cuda.stream(side):
            out, ls = attend(c, q, 0.09, batch=b, out=holder[:, 1:9], stream=side)
        side.synchronize()
        assert torch.equal(holder[:c.n, 1:9], want) and torch.equal(ls[:c.n], lse)
        assert torch.all(holder[:, 0] == 5) and torch.all(holder[:, 9:] == 5) and torch.all(holder[c.n:] == 5)
        # a bound that is too small changes the kernels, not the result's rows
        out, ls = attend(c, q[:c.n].contiguous(), 0.09, batch=c.batch(max_q=1))
        check(c, q[:c.n].contiguous(), 0.09, got=(out, ls))


def test_attend_past_32_bits():
    # pages whose byte offsets pass 2^32: a pool of 4.5 GiB, the sequence in its last pages
    with Case("bf16", "bf16", 8192, 1, 128, [1, 30], [200, 500], seed=20) as c:
        c.fill()
        q = torch.randn((c.n, 4, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        want, lse = check(c, q, 0.1)
        far = 300000
        big = torch.empty((far, c.page_bytes), dtype=torch.uint8, device="cuda")
        big[far - c.n_pages:] = c.pages
        pool = L.lora_pool_create(8192, L.LORA_BF16, far, 1, 8, [(64, 64)], pages_dev=big)
        try:
            cache = L.KvCache(pool, 1, 128, L.LORA_BF16)
            t = torch.where(c.table >= 0, c.table + (far - c.n_pages), c.table)
            b = L.KvBatch(c.q_start, c.kvl, t, c.n, 30)
            ws = torch.empty(L.lora_kv_attend_workspace_size(cache, b, 4), dtype=torch.uint8, device="cuda")
            out, ls = torch.empty_like(q), torch.empty((c.n, 4), dtype=torch.float32, device="cuda")
            L.lora_kv_attend(cache, b, q, out, 0.1, lse=ls, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(ls, lse)
        finally:
            L.lora_pool_destroy(pool)


def test_attend_in_a_graph_with_changing_lengths():
    with Case("f16", "f16", 4096, 2, 128, [1, 1, 1], [100, 200, 300], seed=21) as c:
        c.fill()
        q = torch.randn((3, 4, 128), device="cuda", generator=c.gen).to(TD["f16"])
        b = c.batch()
        ws = torch.empty(L.lora_kv_attend_workspace_size(c.cache, b, 4), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((3, 4), dtype=torch.float32, device="cuda")
        call = L.prepare_kv_attend(c.cache, b, q, out, 0.1, lse=lse, workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(torch.cuda.current_stream())
        for lens in ([100, 200, 300], [3, 199, 64], [1, 1, 300], [0, 7, 33]):
            c.kvl.copy_(torch.tensor(lens, dtype=torch.int32))
            out.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            got, gl = out.clone(), lse.clone()
            out.fill_(4.0)
            call()
            torch.cuda.synchronize()
            assert torch.equal(got, out) and torch.equal(gl, lse)
            c2 = Case.__new__(Case)
            c2.__dict__.update(c.__dict__)
            c2.kv_len = lens
            c2.kd = [k[:n] for k, n in zip(c.kd, lens)]
            c2.vd = [v[:n] for v, n in zip(c.vd, lens)]
            check(c2, q, 0.1, got=(got, gl))


def test_fp8_pool_holds_a_cache():
    # a pool whose pages hold FP8 adapters: caches of its activations' type and of FP8
    for kv in ("f16", "fp8"):
        with Case("f16", kv, 4096, 1, 128, [1, 9], [77, 130], seed=22, fp8_pool=True) as c:
            c.fill()
            q = torch.randn((c.n, 2, 128), device="cuda", generator=c.gen).to(TD["f16"])
            check(c, q, 0.1)


@pytest.mark.parametrize("q_len", [[1, 4], [20, 90]])
def test_attend_widest_window(q_len):
    # a window of 2^31 - 1 reaches as far back as none, also from positions before 0
    with Case("bf16", "bf16", 8192, 1, 128, q_len, [3, 50], seed=23) as c:
        c.fill()
        q = torch.randn((c.n, 2, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        want, lse = check(c, q, 0.1)
        for w in (2 ** 31 - 1, 2 ** 28, 2 ** 28 + 1):
            out, ls = attend(c, q, 0.1, window=w)
            assert torch.equal(out, want) and torch.equal(ls, lse)


@pytest.mark.parametrize("n_seqs,n,length", [(1024, 32768, 1 << 18), (60, 1 << 19, 1 << 18), (60, 1 << 18, 1 << 20)])
def test_attend_of_overlapping_rows_does_nothing_when_they_are_too_many(n_seqs, n, length):
    # every other sequence claims all the rows: more units (a tile of 128 rows with 64
    # keys) than 2^31, which no ascending q_start of a call that is not refused can
    # have; if they are fewer (the second case), the rows see absent pages
    last = length - n + np.minimum(np.arange(128 // 8 - 1, n, 128 // 8), n - 1)   # position of each tile's last row
    units = (n_seqs // 2) * int(np.maximum(1, -(-(last + 1) // 64)).sum())
    with Case("f16", "f16", 4096, 1, 128, [1], [1], seed=24) as c:
        nb = length // c.T
        i32 = dict(dtype=torch.int32, device="cuda")
        b = L.KvBatch(torch.tensor([0, n], **i32).repeat(n_seqs // 2 + 1)[:n_seqs + 1],
                      torch.full((n_seqs,), length, **i32), torch.full((n_seqs, 2, 1, nb), -1, **i32), n, n)
        q = torch.zeros((n, 8, 128), dtype=torch.float16, device="cuda")
        out, lse = attend(c, q, 0.1, batch=b)
        torch.cuda.synchronize()
        if units >= 1 << 31:
            assert torch.all(out == 5) and torch.all(lse == 5)
        else:
            assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("act,kv,page,D", [("f16", "f16", 4096, 128), ("bf16", "fp8", 5120, 128), ("f16", "fp8", 4096, 64)])
@pytest.mark.parametrize("H,G,q_len,window", [(1, 1, [17, 32, 5], 0), (2, 8, [2, 4, 3], 0), (1, 16, [2, 1, 0], 40),
                                              (3, 3, [10, 1, 7], 1), (1, 1, [31, 33, 2], 0), (1, 17, [1, 1, 1], 0)])
def test_attend_between_the_kernels(act, kv, page, D, H, G, q_len, window):
    # 16 and 32 rows of a head and their neighbours: one and two tiles of 16 rows, and tiles of 128
    with Case(act, kv, page, H, D, q_len, [300, 33, 129], seed=30) as c:
        c.fill()
        q = torch.randn((c.n, H * G, D), device="cuda", generator=c.gen).to(TD[act])
        check(c, q, 0.09, window)


# Batches whose rows and tables make them calls of the tiles of 256 rows (8 waves), which
# the host chooses by the tables' capacity: short caches in long tables
WIDE = [("f16", "f16", 4096, 128), ("bf16", "bf16", 5120, 128), ("bf16", "fp8", 5120, 128), ("f16", "fp8", 4096, 128),
        ("f16", "f16", 5120, 64), ("bf16", "bf16", 2056, 64)]


def wide_case(act, kv, page, D, H, G, q_len, kv_len, **kw):
    keys = 64 * (24 * 512 * 256 // (sum(q_len) * G * H) + 64)     # capacity, with room for any number of CUs
    T = page * 2 // (D * (1 if kv == "fp8" else 2))
    return Case(act, kv, page, H, D, q_len, kv_len, extra_blocks=keys // (T // 16 * 16 or 8), **kw)


@pytest.mark.parametrize("act,kv,page,D", WIDE)
@pytest.mark.parametrize("H,G,q_len,kv_len,window", [
    (1, 8, [130], [130], 0),                 # from the first position on
    (2, 3, [256, 200], [256, 463], 0),       # tiles with one row left over, odd positions
    (1, 16, [5, 70], [700, 71], 0),          # few and many rows, one key before them
    (1, 8, [100, 64], [350, 1000], 0),
])
def test_attend_wide_chunks(act, kv, page, D, H, G, q_len, kv_len, window):
    log("[case] attend wide %s/%s page %d D %d H %d G %d %s %s window %d" % (act, kv, page, D, H, G, q_len, kv_len, window))
    with wide_case(act, kv, page, D, H, G, q_len, kv_len, seed=25) as c:
        c.fill()
        q = torch.randn((c.n, H * G, D), device="cuda", generator=c.gen).to(TD[act])
        check(c, q, 0.09, window)


@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "fp8")])
def test_attend_wide_absent_pages_and_rows_without_keys(act, kv):
    # pages that are gone at the start, in the middle and at the end; rows before position 0
    q_len, kv_len = [90, 60], [400, 33]
    with wide_case(act, kv, 4096, 128, 1, 8, q_len, kv_len, seed=26, drop=[(0, 0), (0, 3)]) as c:
        c.fill()
        there = [np.repeat((c.table_host[s] >= 0).all((0, 1)), c.T)[:m] for s, m in enumerate(kv_len)]
        q = torch.randn((c.n, 8, 128), device="cuda", generator=c.gen).to(TD[act])
        check(c, q, 0.1, there=there)
        c.table[0, 1, :, 5] = c.n_pages + 3
        there[0][5 * c.T:6 * c.T] = False
        check(c, q, 0.1, there=there)


@pytest.mark.parametrize("kv", ["f16", "bf16", "fp8"])
def test_attend_wide_what_is_not_seen_has_no_influence(kv):
    # infinities and NaN in K and V: rows that see them get them, others not
    act = "bf16" if kv == "fp8" else kv
    with wide_case(act, kv, 4096, 128, 1, 8, [90, 70], [300, 200], seed=27) as c:
        c.fill()
        q = torch.randn((c.n, 8, 128), device="cuda", generator=c.gen).to(TD[act])
        want, _ = check(c, q, 0.1)
        # tokens 250 and 299 of the first sequence, 140 of the second: seen by later rows only
        for s, j, d, val in ((0, 250, 5, float("nan")), (0, 299, 7, float("inf")), (1, 140, 100, -float("inf"))):
            at = j + (300 if s else 0)
            c.v[at, 0, d] = val
            x = c.v[at:at + 1].double().cpu().numpy()
            c.vd[s][j:j + 1] = dequant(*quant(x)) if c.fp8 else x
        starts = torch.tensor([0, 300, 500], dtype=torch.int32, device="cuda")
        L.lora_kv_write(c.cache, L.KvBatch(starts, c.kvl, torch.from_numpy(c.full_table).cuda(), 500, 300), c.k, c.v)
        out, _ = check(c, q, 0.1)
        assert torch.equal(out[:40], want[:40]) and torch.equal(out[90:100], want[90:100])


def check_rows(c, q, scale, window, tokens, got):
    """Some tokens of a batch of one sequence (tolerances as in check, bf16)."""
    o, l = got[0][tokens].double().cpu().numpy(), got[1][tokens].double().cpu().numpy()
    x, H, base = q[tokens].double().cpu().numpy(), q.shape[1], c.kv_len[0] - c.n
    for i, t in enumerate(tokens):
        pos = base + t
        lo = max(0, pos - window + 1) if window else 0
        for h in range(H):
            k, v = c.kd[0][lo:pos + 1, h * c.H // H], c.vd[0][lo:pos + 1, h * c.H // H]
            s = scale * (k @ x[i, h])
            p = np.exp(s - s.max())
            want, size = p @ v / p.sum(), p @ np.abs(v) / p.sum()
            d = c.D * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(x[i, h])).max()
            assert np.all(np.abs(o[i, h] - want) <= 1.1 * 2.0 ** -8 * size + 1.01 * 2.0 ** -8 * np.abs(want)
                          + (np.expm1(2 * d) + 1e-7) * size), (t, h)
            ls = s.max() + np.log(p.sum())
            assert abs(l[i, h] - ls) <= d + 2.0 ** -21 * max(1, abs(ls)), (t, h)


def test_attend_wide_repeats_and_spans_many_tiles():
    # several tiles of 256 rows a head, whole rounds of them and a cut rest, twice the same bits
    with wide_case("bf16", "bf16", 4096, 64, 8, 8, [1100], [1100], seed=28) as c:
        c.fill()
        q = torch.randn((c.n, 64, 64), device="cuda", generator=c.gen).to(TD["bf16"])
        a, b = attend(c, q, 0.1), attend(c, q, 0.1)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        check_rows(c, q, 0.1, 0, [0, 1, 31, 32, 255, 256, 700, 1023, 1024, 1098, 1099], a)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attend_wide_in_a_window(kv):
    # 64 heads on one and a window of 2000: tiles enough for the wide form
    with Case("bf16", kv, 8192, 1, 128, [900], [3100], seed=29) as c:
        c.fill()
        q = torch.randn((c.n, 64, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        check_rows(c, q, 0.1, 2000, [0, 1, 3, 4, 63, 64, 500, 898, 899], attend(c, q, 0.1, window=2000))
