"""Eviction from the KV cache: weights against the formula in 64 bits, selection and moves against the definitions,
where everything must be equal.

Tolerance of a weight w_j = decay before_j + sum_i exp(x_ij - lse_i), x = scale q . k:
  * a score is a sum of D products in fp32 times a rounded scale, within (D + 4) 2^-24 scale sum |q| |k| =: e of
    its value; lse times log2(e), the difference and the exponential's argument round three times more, each by at
    most 2^-24 (|x| + |lse| + 1), and the exponential itself by 2^-22 of its value: a factor of
    exp(2 e + 4 * 2^-24 (|x| + |lse| + 1)) and 2^-22;
  * the sum of N terms in fp32, at worst N 2^-24 of it; the faded weight rounds once, the last addition once.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gather_lora_matmul_amd as L
from gpu_helpers import log
from kv_formula import agree, formula, visible
from test_gpu_kv import TD, Case
from test_gpu_kv_limits import host, i32


# ---------------------------------------------------------------------------------------------
# weights
# ---------------------------------------------------------------------------------------------
def weighed(c, q, lse, scale, window, decay, before, n, there=None):
    """(weights [S][H][n], tolerance) in 64 bits; NaN where a call leaves the entry."""
    S, G = len(c.q_len), q.shape[1] // c.H
    w, tol = np.full((S, c.H, n), np.nan), np.zeros((S, c.H, n))
    at = 0
    for s, (a, m) in enumerate(zip(c.q_len, c.kv_len)):
        see = visible(np.arange(m - a, m), m, window)
        for h in range(c.H):
            k = c.kd[s][:, h]
            have = np.zeros(m)
            if before is not None and decay:
                old = min(max(m - a, 0), n)
                have[:old] = decay * before[s, h, :old]
            total, err = have.copy(), 2.0 ** -23 * np.abs(have)
            if a:
                x = scale * np.einsum("igd,jd->igj", q[at:at + a, h * G:h * G + G], k)
                size = scale * np.einsum("igd,jd->igj", np.abs(q[at:at + a, h * G:h * G + G]), np.abs(k))
                ls = lse[at:at + a, h * G:h * G + G, None]
                with np.errstate(over="ignore", invalid="ignore"):
                    p = np.where(see[:, None], np.exp(x - ls), 0.0)
                    e = (c.D + 4) * 2.0 ** -24 * size
                    off = np.expm1(2 * e + 2.0 ** -22 * (np.abs(x) + np.abs(ls) + 1)) + 2.0 ** -22
                    total = total + p.sum((0, 1))
                    err = err + np.where(see[:, None], p * off, 0.0).sum((0, 1)) + a * G * 2.0 ** -24 * total
            if there is not None:
                total, err = np.where(there[s][h], total, 0.0), np.where(there[s][h], err, 0.0)
            keep = min(m, n)
            w[s, h, :keep], tol[s, h, :keep] = total[:keep], err[:keep] + 2.0 ** -24 * np.abs(total[:keep]) + 2.0 ** -126
        at += a
    return w, tol


def true_lse(c, q, scale, window):
    """fp32 log-sum-exps of the rows, as the attention leaves them (to within its rounding)."""
    out, at = np.zeros(q.shape[:2], np.float32), 0
    for s, (a, m) in enumerate(zip(c.q_len, c.kv_len)):
        see = visible(np.arange(m - a, m), m, window)
        if a:
            out[at:at + a] = formula(q[at:at + a], c.kd[s], np.zeros_like(c.kd[s]), see, scale)[1]
        at += a
    return out


def weigh(c, q, lse, weights, scale, window=0, decay=1.0, before=None, batch=None, stream=None):
    b = batch or c.batch()
    n = L.lora_kv_weigh_workspace_size(c.cache, b, q.shape[1])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    L.lora_kv_weigh(c.cache, b, q, lse, weights, scale, window=window, decay=decay, before=before, workspace=ws, stream=stream)


def check_weights(c, q, scale, window=0, decay=1.0, with_before=True, n=None, there=None, same=False, lse=None):
    qh = host(q)
    lse = true_lse(c, qh, scale, window) if lse is None else lse
    n = max(c.kv_len + [1]) + 5 if n is None else n
    before = torch.rand((len(c.q_len), c.H, n), device="cuda", generator=c.gen) * 3 if with_before else None
    old = None if before is None else host(before)
    weights = before if same else torch.full((len(c.q_len), c.H, n), 7.0, device="cuda")
    mark = host(weights)
    weigh(c, q, torch.from_numpy(lse).cuda(), weights, scale, window, decay, before)
    torch.cuda.synchronize()
    want, tol = weighed(c, qh, lse.astype(np.float64), scale, window, decay, old, n, there)
    got = host(weights)
    left = np.isnan(want)
    assert np.array_equal(got[left], mark[left]), "entries behind the last token"
    bad = ~(np.abs(got - want)[~left] <= tol[~left])
    assert not bad.any(), "%d of %d, worst %g" % (bad.sum(), bad.size, (np.abs(got - want)[~left] / tol[~left]).max())
    return weights


TYPES = [("f16", "f16", 4096, 128), ("bf16", "bf16", 5120, 64), ("bf16", "fp8", 4096, 128), ("f16", "fp8", 2048, 64),
         ("bf16", "bf16", 8192, 128)]


def queries(c, heads):
    return torch.randn((c.n, heads, c.D), device="cuda", generator=c.gen).to(TD[c.act])


@pytest.mark.parametrize("act,kv,page,D", TYPES)
@pytest.mark.parametrize("H,G,q_len,kv_len", [
    (2, 1, [1, 1, 0, 1], [1, 333, 50, 64]), (1, 8, [2, 1], [2, 700]), (3, 3, [5, 1, 4], [31, 32, 1025]),   # few rows
    (1, 8, [9, 1, 40], [9, 2000, 300]), (2, 1, [130, 17], [500, 17]), (2, 3, [100, 0, 65], [101, 7, 64 + 65])])
@pytest.mark.parametrize("window", [0, 20])
def test_weights(act, kv, page, D, H, G, q_len, kv_len, window):
    log("[case] weights %s/%s D %d H %d G %d %s %s window %d" % (act, kv, D, H, G, q_len, kv_len, window))
    with Case(act, kv, page, H, D, q_len, kv_len, seed=81) as c:
        c.fill()
        q = queries(c, H * G)
        check_weights(c, q, 0.09, window, 0.9)


@pytest.mark.parametrize("G,q_len", [(1, [1, 3]), (4, [40, 70])])
def test_what_was_before(G, q_len):
    # nothing; not looked at for decay 0 (NaN there); in place; faded and whole
    with Case("bf16", "bf16", 4096, 2, 128, q_len, [200, 90], seed=82) as c:
        c.fill()
        q = queries(c, 2 * G)
        check_weights(c, q, 0.1, with_before=False)
        check_weights(c, q, 0.1, decay=1.0, same=True)
        check_weights(c, q, 0.1, decay=0.5)
        check_weights(c, q, 0.1, decay=0.25, n=61)          # fewer entries than tokens
        lse = torch.from_numpy(true_lse(c, host(q), 0.1, 0)).cuda()
        a, b = (torch.zeros((2, 2, 200), device="cuda") for _ in range(2))
        weigh(c, q, lse, a, 0.1)
        weigh(c, q, lse, b, 0.1, decay=0.0, before=torch.full_like(a, float("nan")))
        assert torch.equal(a, b)
        # new tokens have nothing from before, whatever lies there
        nan = torch.zeros((2, 2, 200), device="cuda")
        for s, (n, m) in enumerate(zip(q_len, [200, 90])):
            nan[s, :, m - n:] = float("nan")
        weigh(c, q, lse, nan, 0.1, before=nan)
        assert torch.equal(nan[0], a[0]) and torch.equal(nan[1, :, :90], a[1, :, :90])


@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "fp8")])
@pytest.mark.parametrize("G,q_len", [(1, [2, 1]), (4, [50, 20])])
def test_weights_of_absent_tokens_are_none(act, kv, G, q_len):
    kv_len = [300, 33]
    with Case(act, kv, 2048, 2, 64, q_len, kv_len, seed=83, drop=[(0, 0), (0, 2)]) as c:
        c.fill()
        # of one head, one of the two pages
        t = c.table_host.copy()
        t[0, 1, 1, 1] = -1
        t[1, 0, 0, 0] = 2 ** 30
        c.table = torch.from_numpy(t).cuda()
        ok = ((t >= 0) & (t < c.n_pages)).all(1)
        there = [[np.repeat(ok[s, h], c.T)[:m] for h in range(2)] for s, m in enumerate(kv_len)]
        q = queries(c, 2 * G)
        check_weights(c, q, 0.1, decay=0.7, there=there)


@pytest.mark.parametrize("kv", ["f16", "fp8"])
@pytest.mark.parametrize("G,n", [(1, 3), (8, 40)])
def test_keys_and_rows_that_are_not_finite_stay_where_they_are(kv, G, n):
    # a NaN key is its own weight's, and of the rows that see it; rows without keys (lse -inf, +inf) add nothing
    m = 150
    with Case("f16", kv, 4096, 1, 128, [n, n], [m, n - 2], seed=84) as c:
        c.fill()
        q = queries(c, G)
        lse = true_lse(c, host(q), 0.1, 0)
        weights = check_weights(c, q, 0.1, lse=lse)
        # (the second sequence's first two rows see nothing: their lse is -inf already)
        assert np.isneginf(lse[n:n + 2]).all()
        bad, base = m - 2, m - n
        pg = int(c.full_table[0, 0, 0, bad // c.T])
        t, d = bad % c.T, torch.arange(128, device="cuda")
        at = ((d // c.E) * c.T + t) * c.E + d % c.E
        if kv == "fp8":
            c.pages[pg, at] = 0x7F
        else:
            c.pages[pg].view(torch.int16)[at] = 0x7E00
        w = torch.zeros_like(weights)
        weigh(c, q, torch.from_numpy(lse).cuda(), w, 0.1)
        v = torch.zeros_like(weights)
        torch.cuda.synchronize()
        got = host(w)[0, 0, :m]
        assert np.isnan(got[bad]) and np.isfinite(np.delete(got, bad)).all()
        inf = lse.copy()
        inf[0] = np.inf
        weigh(c, q, torch.from_numpy(inf).cuda(), v, 0.1)
        c2 = host(v)[0, 0, :m]
        assert np.isfinite(np.delete(c2, bad)).all()


def test_many_rows_and_long_sums():
    # sums of thousands of terms
    with Case("bf16", "bf16", 8192, 1, 128, [700], [900], seed=85) as c:
        c.fill()
        q = queries(c, 8)
        check_weights(c, q, 128 ** -0.5)
    with Case("f16", "f16", 4096, 2, 64, [1, 1, 300], [9000, 1, 400], seed=86) as c:
        c.fill()
        check_weights(c, queries(c, 2), 0.125, 250, 0.5)


@pytest.mark.parametrize("act,kv,G", [("bf16", "bf16", 8), ("f16", "fp8", 5)])
@pytest.mark.parametrize("window", [0, 150])
def test_long_rows_among_many_short_ones(act, kv, G, window):
    # tiles cut into several parts, into two, and not at all; sequences of nothing; more of them than a wave has lanes
    rng = np.random.default_rng(G)
    q_len, kv_len = [1] * 150, [int(x) for x in rng.integers(1, 60, 150)]
    for s, (a, m) in {0: (0, 0), 3: (300, 700), 63: (0, 300), 64: (90, 500), 70: (2, 5), 100: (130, 130), 149: (250, 251)}.items():
        q_len[s], kv_len[s] = a, m
    with Case(act, kv, 2048, 1, 64, q_len, kv_len, seed=88) as c:
        c.fill()
        check_weights(c, queries(c, G), 0.11, window, 0.9)


def test_one_long_sequence_in_parts_on_few_tiles():
    # 32 parts of one tile, and a batch whose blocks all get whole tiles
    for H, G, q_len, kv_len in ((1, 8, [600], [200 + 600]), (1, 16, [520, 1], [520, 9]), (8, 6, [90] * 9, [90] * 9)):
        with Case("bf16", "bf16", 4096, H, 128, q_len, kv_len, seed=91) as c:
            c.fill()
            check_weights(c, queries(c, H * G), 0.08, 0, 1.0)


@pytest.mark.parametrize("max_q", [0, 1, 60])
def test_a_wrong_longest_length_changes_the_rounding_only(max_q):
    with Case("bf16", "bf16", 4096, 1, 128, [60, 3], [200, 90], seed=87) as c:
        c.fill()
        q = queries(c, 8)
        lse = torch.from_numpy(true_lse(c, host(q), 0.1, 0)).cuda()
        a, b = (torch.zeros((2, 1, 200), device="cuda") for _ in range(2))
        weigh(c, q, lse, a, 0.1)
        weigh(c, q, lse, b, 0.1, batch=c.batch(max_q=max_q))
        torch.cuda.synchronize()
        assert torch.allclose(a, b, rtol=480 * 2.0 ** -23 + 2.0 ** -18, atol=0)


@pytest.mark.parametrize("kv,G", [("bf16", 6), ("fp8", 6), ("bf16", 64), ("bf16", 1)])
def test_weights_of_lengths_and_rows_far_from_each_other(kv, G):
    # positions past the table and rows before the first token: rows that see nothing leave what was before
    with Case("bf16", kv, 4096, 2, 128, [70, 9], [300, 130], seed=89, extra_blocks=0) as c:
        c.fill()
        q = queries(c, 2 * G)
        lse = torch.zeros((c.n, 2 * G), device="cuda")
        cap = c.table_host.shape[3] * c.T
        for lens, starts, window, had in ((2 ** 31 - 1, None, 20, True), (2 ** 30, None, 2 ** 28, True),
                                          (100, [0, 2 ** 31 - 1, 2 ** 31 - 1], 0, False),
                                          (100, [0, 2 ** 31 - 1, 2 ** 31 - 1], 5, False), (-5, None, 7, None)):
            log("[case] weigh far %s G %d kv_len %d starts %s window %d" % (kv, G, lens, starts, window))
            c.kvl.fill_(lens)
            c.q_start.copy_(torch.tensor([0, 70, 79] if starts is None else starts, dtype=torch.int32))
            before = torch.rand((2, 2, cap + 4), device="cuda", generator=c.gen)
            weights = torch.full_like(before, 7.0)
            weigh(c, q, lse, weights, 0.1, window, 0.5, before)
            torch.cuda.synchronize()
            end = min(max(lens, 0), cap)
            first = (weights[0], before[0])
            assert (weights[:, :, end:] == 7.0).all()
            if had is not None:
                assert torch.equal(first[0][:, :end], first[1][:, :end] * 0.5 if had else torch.zeros_like(first[1][:, :end]))


# ---------------------------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------------------------
def selected(w, m, there, budget, sinks, recent, end):
    """Positions that stay of one head, by sorting."""
    j = np.flatnonzero(there[:m])
    key = w[j].astype(np.float64)
    key = np.where(np.isnan(key), -np.inf, key)
    cls = np.where((j < sinks) | (j >= end - recent), 2, np.where(np.isnan(w[j]), 0, 1))
    order = np.lexsort((j, -key, -cls))
    # (among the first and the latest ones the first come first)
    top = cls == 2
    order = np.concatenate([np.flatnonzero(top), [i for i in order if not top[i]]]).astype(int)
    return np.sort(j[order[:budget]])


def select(c, weights, budget, sinks=0, recent=0, ld=None, stream=None, batch=None):
    b = batch or c.batch()
    S = b.desc.n_seqs
    keep = torch.full((S, c.H, budget + 3 if ld is None else ld), -9, dtype=torch.int32, device="cuda")
    n_keep = torch.full((S,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((L.lora_kv_select_workspace_size(c.cache, b),), 0xFF, dtype=torch.uint8, device="cuda")
    L.lora_kv_select(c.cache, b, weights, budget, keep, n_keep, sinks=sinks, recent=recent, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), n_keep.cpu().numpy()


def check_selection(c, weights, budget, sinks=0, recent=0, lens=None):
    keep, n_keep = select(c, weights, budget, sinks, recent)
    lens = c.kv_len if lens is None else lens
    w, n, T = weights.cpu().numpy(), weights.shape[2], c.T
    cap = c.table_host.shape[3] * T
    ok = ((c.table_host >= 0) & (c.table_host < c.n_pages)).all(1)
    for s, m in enumerate(lens):
        end = min(max(m, 0), cap)
        m = min(end, n)
        there = [np.repeat(ok[s, h], T)[:m] for h in range(c.H)]
        k = min([budget] + [int(t.sum()) for t in there])
        assert n_keep[s] == k, (s, n_keep[s], k)
        for h in range(c.H):
            want = selected(w[s, h, :m], m, there[h], k, sinks, recent, end)
            assert np.array_equal(keep[s, h, :k], want), (s, h)
            assert (keep[s, h, k:] == -9).all()


def empty_case(H, kv_len, page=4096, drop=(), **kw):
    return Case("bf16", "bf16", page, H, 128, [0] * len(kv_len), kv_len, drop=drop, **kw)


def some_weights(c, n, seed, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (len(c.kv_len), c.H, n)
    w = torch.randn(shape, device="cuda", generator=g).exp()
    if kind == "ties":
        w = torch.randint(0, 4, shape, device="cuda", generator=g).float()
    elif kind == "equal":
        w.fill_(0.25)
    elif kind == "near":        # that differ in their last bits only
        w = (torch.randint(0, 3000, shape, device="cuda", generator=g, dtype=torch.int32) + 0x3F800000).view(torch.float32)
    elif kind == "odd":
        x = torch.tensor([0.0, -0.0, float("nan"), float("inf"), float("-inf"), -1.5, 1e-45, 3e38, -3e38, 2.0], device="cuda")
        w = x[torch.randint(0, 10, shape, device="cuda", generator=g)]
        w.view(torch.int32)[..., ::7] |= torch.where(torch.isnan(w[..., ::7]), -2 ** 31, 0).to(torch.int32)   # NaN of both signs
    return w


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "near", "odd"])
def test_selection(kind):
    lens = [0, 1, 31, 64, 65, 500, 300]
    with empty_case(3, lens, seed=91) as c:
        w = some_weights(c, 517, 5, kind)
        for budget, sinks, recent in ((0, 0, 0), (1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 4, 10), (64, 64, 0), (64, 0, 64),
                                      (64, 30, 34), (300, 2, 3), (499, 0, 0), (500, 1, 1), (700, 100, 200)):
            log("[case] select %s budget %d sinks %d recent %d" % (kind, budget, sinks, recent))
            check_selection(c, w, budget, sinks, recent)


@pytest.mark.parametrize("kind", ["random", "ties", "near"])
@pytest.mark.parametrize("lens,budget", [([8191, 8192, 20], 1000), ([8193, 9, 16384], 4096), ([70001, 33000], 20000),
                                         ([140000], 3)])
def test_selection_of_long_caches(kind, lens, budget):
    with empty_case(2, lens, seed=92) as c:
        log("[case] select long %s %s" % (kind, lens))
        sinks, recent = (4, budget // 3) if budget > 4 else (0, 0)
        check_selection(c, some_weights(c, max(lens), 6, kind), budget, sinks, recent)


def test_selection_of_absent_and_unweighed_tokens():
    lens = [300, 200, 90, 64]
    with empty_case(2, lens, seed=93, page=2048, drop=[(0, 0), (0, 5), (2, 0), (3, 0), (3, 1), (3, 2), (3, 3)]) as c:
        t = c.table_host
        t[1, 0, 1, 2] = -1                   # one page of one head: every head keeps as many as that one can
        t[1, 1, 1, 3] = c.n_pages
        c.table = torch.from_numpy(t).cuda()
        for n in (300, 120, 17, 1):          # entries of a head
            w = some_weights(c, n, 7, "random")
            for budget, sinks, recent in ((50, 4, 10), (160, 0, 0), (1000, 40, 60), (8, 8, 0)):
                check_selection(c, w, budget, sinks, recent)
        # lengths past the table, and below 0
        for bad in ([100000, 2 ** 31 - 1, -1, -2 ** 31],):
            c.kvl.copy_(torch.tensor(bad, dtype=torch.int32))
            check_selection(c, some_weights(c, 500, 8, "random"), 60, 3, 9, lens=bad)


@pytest.mark.parametrize("lens", [(4097, 8192, 5000), (8193, 16384, 3)])
def test_selection_of_many_heads_of_long_caches(lens):
    # more heads than the device has compute units
    lens = [lens[i % 3] if i % 9 < 3 else 30 for i in range(36)]
    with empty_case(8, lens, seed=103, page=16384) as c:
        check_selection(c, some_weights(c, max(lens), 7, "ties"), 700, 4, 100)
        check_selection(c, some_weights(c, max(lens), 8, "random"), 2500)


def test_counts_past_32_bits_are_refused():
    with empty_case(1, [20], seed=90) as c:
        w = torch.rand((1, 1, 20), device="cuda")
        for kw in (dict(budget=2 ** 32 + 5), dict(budget=8, sinks=2 ** 32), dict(budget=8, recent=2 ** 32 + 1),
                   dict(budget=8, sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(budget=-2 ** 32 + 8)):
            with pytest.raises(Exception, match="budget|keep_ld"):
                select(c, w, ld=11, **kw)


def test_many_heads_and_sequences():
    lens = np.random.default_rng(4).integers(0, 90, 300).tolist()
    with empty_case(9, lens, seed=94, page=1024, extra_blocks=0) as c:
        check_selection(c, some_weights(c, 90, 9, "ties"), 33, 2, 8)


# ---------------------------------------------------------------------------------------------
# moves
# ---------------------------------------------------------------------------------------------
def moved(c, keep, n_keep, from_new, weights):
    """(pages, scales, weights) after the moves, one token after another."""
    pages = c.pages.cpu().numpy().copy()
    flat = pages if c.fp8 else pages.view(np.uint16)
    scales = None if c.scales is None else c.scales.cpu().numpy().copy()
    w = None if weights is None else weights.cpu().numpy().copy()
    lens, starts = c.kvl.cpu().numpy(), c.q_start.cpu().numpy()
    T, E, D = c.T, c.E, c.D
    cap = c.table_host.shape[3] * T
    d = np.arange(D)
    for s in range(len(lens)):
        end = min(max(int(lens[s]), 0), cap)
        first = max(int(lens[s]), 0) - int(starts[s + 1] - starts[s]) if from_new else 0
        for h in range(c.H):
            for i in range(min(max(int(n_keep[s]), 0), keep.shape[2])):
                k = int(keep[s, h if keep.shape[1] > 1 else 0, i])
                src, dst = first + k, first + i
                if k < 0 or src >= end or src < 0 or dst < 0 or dst >= end:
                    continue
                for which in (0, 1):
                    a, b = (int(c.table_host[s, which, h, x // T]) for x in (src, dst))
                    if not (0 <= a < c.n_pages and 0 <= b < c.n_pages):
                        continue
                    place = lambda t: ((d // E) * T + t) * E + d % E if which == 0 else ((t // E) * D + d) * E + t % E
                    flat[b, place(dst % T)] = flat[a, place(src % T)]
                    if scales is not None:
                        scales[b, dst % T] = scales[a, src % T]
                if w is not None and src < w.shape[2]:
                    w[s, h, dst] = w[s, h, src]
    return pages, scales, w


def check_moves(c, keep, n_keep, from_new=False, weights=None, stream=None, flat=False):
    want = moved(c, keep, n_keep, from_new, weights)
    k = i32(keep)
    L.lora_kv_compact(c.cache, c.batch(), k[:, 0].contiguous() if flat else k, i32(n_keep), from_new=from_new,
                      weights=weights, stream=stream)
    torch.cuda.synchronize()
    assert np.array_equal(c.pages.cpu().numpy(), want[0]), "pages"
    if c.scales is not None:
        assert np.array_equal(c.scales.cpu().numpy(), want[1]), "scales"
    if weights is not None:
        assert np.array_equal(weights.cpu().numpy(), want[2], equal_nan=True), "weights"


def lists(rng, lens, heads, most):
    """Ascending lists of min(len, most) of each sequence's tokens."""
    keep = np.full((len(lens), heads, max(most, 1)), 77, np.int64)
    for s, m in enumerate(lens):
        for h in range(heads):
            k = min(m, most)
            keep[s, h, :k] = np.sort(rng.choice(m, k, replace=False)) if k else []
    return keep, np.array([min(m, most) for m in lens])


LAYOUTS = [("f16", "f16", 4096, 3, 128), ("bf16", "bf16", 5120, 2, 64), ("bf16", "fp8", 5120, 2, 128), ("f16", "fp8", 4096, 1, 64),
           ("bf16", "bf16", 520, 2, 64), ("f16", "fp8", 1100 * 8, 3, 128)]


@pytest.mark.parametrize("act,kv,page,H,D", LAYOUTS)
def test_moves_of_selections(act, kv, page, H, D):
    lens = [0, 1, 7, 8, 130, 300, 64]
    rng = np.random.default_rng(3)
    for most, heads in ((100, H), (33, 1), (300, H), (1, H)):
        log("[case] compact %s/%s page %d heads %d most %d" % (act, kv, page, heads, most))
        with Case(act, kv, page, H, D, [0] * 7, lens, seed=95) as c:
            c.fill()
            keep, n_keep = lists(rng, lens, heads, most)
            w = torch.rand((7, H, 310), device="cuda", generator=c.gen)
            check_moves(c, keep, n_keep, weights=w)


@pytest.mark.parametrize("act,kv,page,H,D", LAYOUTS)
def test_moves_of_paths(act, kv, page, H, D):
    q_len, kv_len = [1, 9, 25, 0, 60, 14], [1, 9, 200, 30, 61, 95]
    rng = np.random.default_rng(4)
    log("[case] compact paths %s/%s page %d" % (act, kv, page))
    with Case(act, kv, page, H, D, q_len, kv_len, seed=96) as c:
        c.fill()
        keep = np.full((6, 1, 20), -1, np.int64)
        n_keep = np.zeros(6, np.int64)
        for s, n in enumerate(q_len):
            if n:
                path = np.concatenate([[0], 1 + np.sort(rng.choice(n - 1, min(n - 1, 1 + s), replace=False))])
                keep[s, 0, :len(path)], n_keep[s] = path, len(path)
        check_moves(c, keep, n_keep, from_new=True, flat=True)


def test_moves_over_many_steps_and_back_to_front():
    # long lists, every second token, all but the first, nothing moved, and what lies behind stays
    for kv in ("bf16", "fp8"):
        for pick in (lambda m: np.arange(0, m, 2), lambda m: np.arange(1, m), lambda m: np.arange(m),
                     lambda m: np.concatenate([np.arange(5), np.arange(m - 400, m)])):
            with Case("bf16", kv, 4096, 1, 128, [0, 0], [3000, 1111], seed=97) as c:
                c.fill()
                a, b = pick(3000), pick(1111)
                keep = np.zeros((2, 1, max(len(a), len(b))), np.int64)
                keep[0, 0, :len(a)], keep[1, 0, :len(b)] = a, b
                check_moves(c, keep, [len(a), len(b)], weights=torch.rand((2, 1, 2000), device="cuda", generator=c.gen))


def test_numbers_and_pages_that_are_not_there():
    q_len, kv_len = [20, 9, 9, 9], [100, 90, 60, 64]
    for from_new in (False, True):
        for kv in ("bf16", "fp8"):
            with Case("bf16", kv, 2048, 2, 64, q_len, kv_len, seed=98, extra_blocks=0, drop=[(0, 1), (1, 0), (3, 0)]) as c:
                c.fill()
                t = c.table_host
                t[2, 1, 0, 0] = c.n_pages + 5
                c.table = torch.from_numpy(t).cuda()
                keep = np.zeros((4, 1, 12), np.int64)
                keep[:, 0] = [-1, 1, 2, -2 ** 31, 5, 7, 9, 30, 99, 100, 2 ** 30, 2 ** 31 - 1]
                check_moves(c, keep, [12, 7, 2 ** 31 - 1, -4], from_new=from_new)
                c.kvl.copy_(torch.tensor([4, 2 ** 31 - 1, 0, 5], dtype=torch.int32))   # fewer tokens than rows; past the table
                check_moves(c, keep, [12, 12, 12, 12], from_new=from_new)


def test_lists_that_do_not_ascend_stay_within_the_weights():
    # which tokens the places get is open; nothing behind the rows of weights or in pages of others is touched
    for most in (12, 200):
        with Case("bf16", "bf16", 4096, 2, 128, [0, 0], [260, 90], seed=99) as c:
            c.fill()
            n = 7
            flat = torch.rand((2 * 2 * n + 500,), device="cuda", generator=c.gen)
            mark = flat.clone()
            weights = flat[:2 * 2 * n].view(2, 2, n)
            keep = np.zeros((2, 2, most), np.int64)
            keep[:, :, ::2] = 5
            keep[:, 1] = np.arange(most)[::-1]
            pages = c.pages.clone()
            used = set(int(x) for x in c.table_host.ravel())
            L.lora_kv_compact(c.cache, c.batch(), i32(keep), i32([most, most]), weights=weights)
            torch.cuda.synchronize()
            assert torch.equal(flat[2 * 2 * n:], mark[2 * 2 * n:])
            assert all(torch.isin(weights[s, h], mark[:2 * 2 * n].view(2, 2, n)[s, h]).all() for s in (0, 1) for h in (0, 1))
            others = [p for p in range(c.n_pages) if p not in used]
            assert torch.equal(c.pages[others], pages[others])


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "fp8")])
@pytest.mark.parametrize("G,q_len", [(2, [1, 1, 1]), (4, [30, 1, 17])])
def test_a_step_of_eviction(act, kv, G, q_len):
    """Attention, weights, selection and moves as a serving step makes them; what the next step attends to is what
    was selected."""
    kv_len, H, D, budget = [400, 77, 50], 2, 128, 64
    with Case(act, kv, 4096, H, D, q_len, kv_len, seed=99) as c:
        c.fill()
        q = queries(c, H * G)
        b = c.batch()
        space = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((c.n, H * G), device="cuda")
        w = torch.zeros((3, H, 400), device="cuda")
        keep = torch.zeros((3, H, budget), dtype=torch.int32, device="cuda")
        n_keep = torch.zeros(3, dtype=torch.int32, device="cuda")
        steps = [L.prepare_kv_attend(c.cache, b, q, out, 0.1, lse=lse, workspace=space(L.lora_kv_attend_workspace_size(c.cache, b, H * G))),
                 L.prepare_kv_weigh(c.cache, b, q, lse, w, 0.1, decay=0.5, before=w, workspace=space(L.lora_kv_weigh_workspace_size(c.cache, b, H * G))),
                 L.prepare_kv_select(c.cache, b, w, budget, keep, n_keep, sinks=2, recent=8, workspace=space(L.lora_kv_select_workspace_size(c.cache, b))),
                 L.prepare_kv_compact(c.cache, b, keep, n_keep, weights=w)]
        for st in steps:
            st()
        torch.cuda.synchronize()
        assert n_keep.tolist() == [64, 64, 50]
        kept = keep.cpu().numpy()
        kd = [np.stack([c.kd[s][kept[s, h, :n], h] for h in range(H)], 1) for s, n in enumerate(n_keep.tolist())]
        vd = [np.stack([c.vd[s][kept[s, h, :n], h] for h in range(H)], 1) for s, n in enumerate(n_keep.tolist())]
        one = torch.randn((3, H * G, D), device="cuda", generator=c.gen).to(TD[act])
        b2 = L.KvBatch(i32([0, 1, 2, 3]), n_keep, c.table, 3, 1)
        o2, l2 = torch.empty_like(one), torch.empty((3, H * G), device="cuda")
        L.lora_kv_attend(c.cache, b2, one, o2, 0.1, lse=l2, workspace=space(L.lora_kv_attend_workspace_size(c.cache, b2, H * G)))
        torch.cuda.synchronize()
        for s, n in enumerate(n_keep.tolist()):
            want = formula(host(one)[s:s + 1], kd[s], vd[s], np.ones((1, n), bool), 0.1)
            agree(host(o2)[s:s + 1], host(l2)[s:s + 1], want, "bf16" if kv == "fp8" else act, 2, act, n, "sequence %d" % s)


def test_graphs_with_changing_lengths_and_another_stream():
    with Case("bf16", "bf16", 4096, 2, 128, [1, 1, 1], [500, 200, 90], seed=100) as c:
        c.fill()
        q, b = queries(c, 4), c.batch()
        lse = torch.full((3, 4), 5.0, device="cuda")
        space = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        w = torch.zeros((3, 2, 500), device="cuda")
        old = torch.rand((3, 2, 500), device="cuda", generator=c.gen)
        keep = torch.zeros((3, 2, 100), dtype=torch.int32, device="cuda")
        n_keep = torch.zeros(3, dtype=torch.int32, device="cuda")
        steps = [L.prepare_kv_weigh(c.cache, b, q, lse, w, 0.1, decay=0.9, before=old, workspace=space(L.lora_kv_weigh_workspace_size(c.cache, b, 4))),
                 L.prepare_kv_select(c.cache, b, w, 100, keep, n_keep, sinks=1, recent=5, workspace=space(L.lora_kv_select_workspace_size(c.cache, b))),
                 L.prepare_kv_compact(c.cache, b, keep, n_keep, weights=w)]
        pages = c.pages.clone()

        def eager(stream):
            c.pages.copy_(pages)
            w.fill_(3.0)
            keep.fill_(-1)
            stream.wait_stream(torch.cuda.current_stream())
            for st in steps:
                st(stream)
            torch.cuda.synchronize()
            return [x.clone() for x in (c.pages, w, keep, n_keep)]

        eager(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        c.pages.copy_(pages)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for st in steps:
                st(torch.cuda.current_stream())
        side = torch.cuda.Stream()
        for lens in ([500, 200, 90], [3, 500, 101], [0, 1, 499], [100, 100, 100]):
            c.kvl.copy_(torch.tensor(lens, dtype=torch.int32))
            want = eager(side)
            c.pages.copy_(pages)
            w.fill_(3.0)
            keep.fill_(-1)
            n_keep.fill_(-1)
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip((c.pages, w.view(torch.int32), keep, n_keep), (want[0], want[1].view(torch.int32), *want[2:])):
                assert torch.equal(x, y)   # (by bits: places past what was filled hold NaN)


def test_a_step_with_a_tree():
    """Build, write, attend, verify, compact; then the cache is that of the accepted path."""
    rng = np.random.default_rng(7)
    S, H, D, V, n = 3, 2, 64, 500, 12
    base = [40, 7, 129]
    for kv in ("f16", "fp8"):
        with Case("f16", kv, 2048, H, D, [n] * S, [b + n for b in base], seed=101) as c:
            c.fill()
            parents = np.stack([np.minimum((np.arange(n) * rng.random(n)).astype(int), np.arange(n) - 1) for _ in range(S)])
            parent = i32(parents.reshape(-1))
            seen = torch.zeros((S * n, 1), dtype=torch.int64, device="cuda")
            depth = torch.zeros(S * n, dtype=torch.int32, device="cuda")
            L.lora_kv_tree_build(c.q_start, parent, seen, depth)
            b, q = c.batch(), queries(c, H * 2)
            out = torch.empty_like(q)
            space = lambda k: torch.empty(max(k, 1), dtype=torch.uint8, device="cuda")
            L.lora_kv_attend_tree(c.cache, b, L.KvTree(seen, depth), q, out, 0.1, workspace=space(L.lora_kv_attend_workspace_size(c.cache, b, H * 2)))
            # a target that accepts about every second draft
            target = torch.full((S * n, V), 0.3 / V, device="cuda")
            drafted = torch.randint(0, V, (S * n,), device="cuda", generator=c.gen).to(torch.int32)
            for s in range(S):
                for t in range(1, n):
                    target[s * n + parents[s, t], int(drafted[s * n + t])] = 0.4
            target /= target.sum(1, keepdim=True)
            tokens, path = (torch.zeros((S, n), dtype=torch.int32, device="cuda") for _ in range(2))
            n_out = torch.zeros(S, dtype=torch.int32, device="cuda")
            L.lora_spec_verify_tree(c.q_start, parent, drafted, target, torch.rand(S * n, device="cuda", generator=c.gen),
                                    torch.rand(S, device="cuda", generator=c.gen), tokens, path, n_out,
                                    space(L.lora_spec_verify_tree_workspace_size(S, V)))
            L.lora_kv_compact(c.cache, b, path, n_out, from_new=True)
            lens = i32(base) + n_out
            one = torch.randn((S, H * 2, D), device="cuda", generator=c.gen).half()
            b2 = L.KvBatch(i32([0, 1, 2, 3]), lens, c.table, S, 1)
            o2, l2 = torch.empty_like(one), torch.empty((S, H * 2), device="cuda")
            L.lora_kv_attend(c.cache, b2, one, o2, 0.1, lse=l2, workspace=space(L.lora_kv_attend_workspace_size(c.cache, b2, H * 2)))
            torch.cuda.synchronize()
            assert max(n_out.tolist()) > 1
            for s in range(S):
                at = np.concatenate([np.arange(base[s]), base[s] + path[s, :int(n_out[s])].cpu().numpy()])
                want = formula(host(one)[s:s + 1], c.kd[s][at], c.vd[s][at], np.ones((1, len(at)), bool), 0.1)
                agree(host(o2)[s:s + 1], host(l2)[s:s + 1], want, "bf16" if kv == "fp8" else "f16", 2, "f16", len(at), str(s))


def test_selection_in_tables_wider_than_the_caches():
    # the launches follow the tables' width, the work the lengths
    lens = [0, 5, 300, 9000, 8192, 20]
    with empty_case(2, lens, seed=102, extra_blocks=300, drop=[(3, 4), (3, 270)]) as c:
        for kind in ("random", "equal", "near"):
            w = some_weights(c, 18000, 10, kind)
            for budget, sinks, recent in ((0, 0, 0), (4, 4, 0), (250, 3, 40), (8999, 0, 0), (9000, 0, 9000)):
                check_selection(c, w, budget, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "near", "zeros"])
@pytest.mark.parametrize("lens", [(2048, 300), (4096, 2049), (8192, 5000), (16384, 8193), (30000, 16385)])
def test_selection_whose_border_has_more_ranks_than_a_block_has_threads(lens, kind):
    with empty_case(2, list(lens), seed=104, page=16384) as c:
        w = some_weights(c, max(lens), 11, "random" if kind == "zeros" else kind)
        if kind == "zeros":
            w[torch.rand(w.shape, device="cuda", generator=c.gen) < 0.98] = 0.0
        for budget, sinks, recent in ((max(lens) // 3, 4, 100), (max(lens) // 2, 0, 0)):
            log("[case] select crowded %s %s budget %d" % (kind, lens, budget))
            check_selection(c, w, budget, sinks, recent)
