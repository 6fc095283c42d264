"""Trees of drafted tokens: their visibility and verification against whole-number arithmetic on the host, where
everything must be equal, and their attention against the formula in 64 bits, within the bound that kv_formula
derives from the kernels' roundings."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gather_lora_matmul_amd as L
from gpu_helpers import log
from kv_formula import agree, formula
from test_gpu_kv import TD, Case, wide_case
from test_gpu_kv_limits import host, i32


# ---------------------------------------------------------------------------------------------
# visibility
# ---------------------------------------------------------------------------------------------
def chains(parent, most=1 << 30):
    """Of every token: itself and its ancestors, root first.  Parents that are not below are none."""
    out = []
    for t, p in enumerate(parent):
        out.append((out[p] if 0 <= p < t and t < most else []) + [t])
    return out


def rows_of(parent, words, window=0):
    """(seen [n][words] uint64, depth [n], sees [n][n]) of one tree by definition."""
    n = len(parent)
    seen, depth, sees = np.zeros((n, words), np.uint64), np.zeros(n, np.int32), np.zeros((n, n), bool)
    for t, c in enumerate(chains(parent)):
        if t >= 64 * words:
            continue
        depth[t] = len(c) - 1
        for u in c[-window:] if window else c:
            seen[t, u // 64] |= np.uint64(1 << u % 64)
            sees[t, u] = True
    return seen, depth, sees


def random_parents(rng, n, kind):
    t = np.arange(n)
    if kind == "chain":
        return t - 1
    if kind == "star":
        return np.where(t, 0, -1)
    if kind == "forest":     # several roots, and parents that are none: negative, the token itself, later ones
        return np.where(rng.random(n) < 0.3, rng.choice([-1, -7, n + 3, 2 ** 30, -2 ** 31], n),
                        np.where(rng.random(n) < 0.1, t + rng.integers(0, 3, n), (t * rng.random(n)).astype(int)))
    return np.minimum((t * rng.random(n)).astype(int), t - 1)


def build(q_start, parent, words, window=0, stream=None):
    n = len(parent)
    seen = torch.full((n, words), 77, dtype=torch.int64, device="cuda")
    depth = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    L.lora_kv_tree_build(i32(q_start), i32(parent), seen, depth, window=window, stream=stream)
    return seen, depth


@pytest.mark.parametrize("words,sizes", [(1, [1]), (1, [0, 64, 1, 7, 0]), (2, [100, 128, 3]), (3, [70, 65, 192, 64]),
                                         (16, [1024, 5, 600]), (1, [66, 2]), (2, [300, 129])])
@pytest.mark.parametrize("window", [0, 1, 3, 2 ** 31 - 1])
def test_build(words, sizes, window):
    rng = np.random.default_rng(words + len(sizes) + window % 100)
    for kind in ("tree", "chain", "star", "forest"):
        log("[case] build words %d sizes %s window %d %s" % (words, sizes, window, kind))
        parents = [random_parents(rng, n, kind) for n in sizes]
        starts = np.concatenate([[0], np.cumsum(sizes)])
        rest = 3   # rows of no sequence
        flat = np.concatenate(parents + [np.zeros(rest, int)])
        seen, depth = build(starts, flat, words, window)
        torch.cuda.synchronize()
        got, gd = seen.cpu().numpy().view(np.uint64), depth.cpu().numpy()
        for s, p in enumerate(parents):
            want, wd, _ = rows_of(p, words, window)
            a, b = starts[s], starts[s + 1]
            assert np.array_equal(got[a:b], want) and np.array_equal(gd[a:b], wd), (kind, s)
        assert (got[starts[-1]:] == 77).all() and (gd[starts[-1]:] == 77).all()


def test_build_holds_rows_inside_the_tensors():
    # starts that do not ascend, lie below 0 or past the tokens
    for starts in ([-5, 3, 2, 9, 40], [7, 7, 100, 100, -3], [2 ** 31 - 1, -2 ** 31, 5, 10, 10]):
        seen, depth = build(starts, np.arange(10) - 1, 1)
        torch.cuda.synchronize()
        got = seen.cpu().numpy()
        covered = np.zeros(10, bool)
        for a, b in zip(starts, starts[1:]):
            a = min(max(a, 0), 10)
            covered[a:min(max(b, a), 10)] = True
        assert (got[~covered] == 77).all() and (got[covered] != 77).all()


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def sees_of(c, s, sees, depth, window, there=None):
    """[n][kv_len] what the new tokens of sequence s see."""
    n, m = c.q_len[s], c.kv_len[s]
    base = m - n
    out = np.zeros((n, max(m, 0)), bool)
    for t in range(n):
        lo = base + int(depth[t]) + 1 - window if window else 0
        out[t, max(lo, 0):max(base, 0)] = True
        for u in range(n):
            if base + u >= 0:
                out[t, base + u] = sees[t, u]
    return out if there is None else out & there[None]


def attend(c, q, seen, depth, scale, window=0, batch=None, stream=None, out=None):
    b = batch or c.batch()
    ws = torch.full((L.lora_kv_attend_workspace_size(c.cache, b, q.shape[1]),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 5.0) if out is None else out
    lse = torch.full((q.shape[0], q.shape[1]), 5.0, dtype=torch.float32, device="cuda")
    L.lora_kv_attend_tree(c.cache, b, L.KvTree(seen, depth), q, out, scale, window=window, lse=lse, workspace=ws,
                          stream=stream)
    return out, lse


def check(c, q, trees, scale, window=0, wide=False, kd=None, vd=None, there=None, rows=None):
    """trees: of each sequence (seen, depth, sees); runs and compares, rows of each sequence if given."""
    seen = torch.from_numpy(np.concatenate([t[0] for t in trees]).view(np.int64)).cuda()
    depth = i32(np.concatenate([t[1] for t in trees]))
    out, lse = attend(c, q, seen, depth, scale, window)
    torch.cuda.synchronize()
    few = max(c.q_len) * q.shape[1] // c.H <= (32 if c.fp8 else 16)
    p_type, terms = ("bf16" if c.fp8 and few else c.act), 1 if wide else 2
    qh, oh, lh = host(q), host(out), host(lse)
    at = 0
    for s, (n, m) in enumerate(zip(c.q_len, c.kv_len)):
        r = np.arange(n) if rows is None else np.array([x for x in rows if x < n], int)
        if n:
            see = sees_of(c, s, trees[s][2], trees[s][1], window, None if there is None else there[s])[r]
            want = formula(qh[at:at + n][r], (kd or c.kd)[s][:m], (vd or c.vd)[s][:m], see, scale)
            agree(oh[at:at + n][r], lh[at:at + n][r], want, p_type, terms, c.act, max(m, 1), "sequence %d" % s)
        at += n
    return out, lse


def trees_for(c, seed, words, window=0, kinds=("tree", "chain", "star", "forest")):
    rng = np.random.default_rng(seed)
    return [rows_of(random_parents(rng, n, kinds[s % len(kinds)]), words, window) for s, n in enumerate(c.q_len)]


def queries(c, heads):
    return torch.randn((c.n, heads, c.D), device="cuda", generator=c.gen).to(TD[c.act])


TYPES = [("f16", "f16", 4096, 128), ("bf16", "bf16", 5120, 64), ("bf16", "fp8", 4096, 128), ("f16", "fp8", 2048, 64)]
FEW = [(2, 1, [9, 1, 16, 0, 3], [40, 1, 300, 7, 3]), (1, 4, [4, 2], [1000, 2]), (3, 5, [3, 1, 2], [130, 64, 67])]
MANY = [(2, 8, [64, 5, 33], [200, 5, 700]), (1, 3, [100, 1, 128], [100, 900, 333]), (2, 1, [70, 130], [71, 1999])]


@pytest.mark.parametrize("act,kv,page,D", TYPES)
@pytest.mark.parametrize("H,G,q_len,kv_len", FEW + MANY)
@pytest.mark.parametrize("window", [0, 5, 100])
def test_attention(act, kv, page, D, H, G, q_len, kv_len, window):
    words = (max(q_len) + 63) // 64
    log("[case] tree attention %s/%s D %d H %d G %d %s %s window %d" % (act, kv, D, H, G, q_len, kv_len, window))
    with Case(act, kv, page, H, D, q_len, kv_len, seed=61) as c:
        c.fill()
        check(c, queries(c, H * G), trees_for(c, 3, words, window), 0.09, window)


@pytest.mark.parametrize("act,kv,page,D", TYPES)
def test_attention_by_waves_for_themselves(act, kv, page, D):
    # two (sequence, head) pairs a block and more
    S, H = 40, 32
    rng = np.random.default_rng(5)
    q_len, kv_len = rng.integers(0, 10, S).tolist(), None
    kv_len = [n + int(x) for n, x in zip(q_len, rng.integers(0, 150, S))]
    log("[case] tree attention, waves, %s/%s D %d" % (act, kv, D))
    with Case(act, kv, page, H, D, q_len, kv_len, seed=62, extra_blocks=0) as c:
        c.fill()
        check(c, queries(c, H), trees_for(c, 4, 1, 7), 0.09, 7)


@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")])
@pytest.mark.parametrize("H,G,q_len,kv_len,window", [(1, 8, [100, 64], [350, 1000], 0), (2, 6, [128, 90], [128, 463], 40)])
def test_attention_of_wide_tiles(act, kv, H, G, q_len, kv_len, window):
    log("[case] tree attention, wide, %s/%s %s window %d" % (act, kv, q_len, window))
    with wide_case(act, kv, 4096, 128, H, G, q_len, kv_len, seed=63) as c:
        c.fill()
        check(c, queries(c, H * G), trees_for(c, 5, 2, window), 0.09, window, wide=True)


@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")])
@pytest.mark.parametrize("H,G,q_len,kv_len", [(1, 8, [9, 14, 10, 30, 2], [20, 300, 10, 64, 700]), (2, 5, [20, 17, 16], [400, 17, 90])])
def test_attention_of_wide_tiles_with_few_rows(act, kv, H, G, q_len, kv_len):
    log("[case] tree attention, wide, few rows, %s/%s %s" % (act, kv, q_len))
    with wide_case(act, kv, 4096, 128, H, G, q_len, kv_len, seed=74) as c:
        c.fill()
        check(c, queries(c, H * G), trees_for(c, 15, 1), 0.09, wide=True)


@pytest.mark.parametrize("act,kv", [("bf16", "bf16"), ("f16", "fp8")])
def test_attention_of_wide_tiles_in_a_window(act, kv):
    S, rng = 100, np.random.default_rng(16)
    kv_len = [int(x) for x in rng.integers(12, 500, S)]
    log("[case] tree attention, wide, window, %s/%s" % (act, kv))
    with Case(act, kv, 4096, 8, 128, [12] * S, kv_len, seed=75, extra_blocks=0) as c:
        c.fill()
        check(c, queries(c, 64), trees_for(c, 17, 1, 192), 0.09, 192, wide=True, rows=[0, 5, 11])


@pytest.mark.parametrize("G,n", [(1, 7), (8, 30)])
def test_rows_of_any_bits(G, n):
    # not trees: rows that see nothing, not themselves, later tokens, tokens that the sequence has not
    with Case("bf16", "bf16", 4096, 1, 128, [n, n], [n, 90], seed=64) as c:
        c.fill()
        rng = np.random.default_rng(6)
        trees = []
        for s in range(2):
            sees = rng.random((n, n)) < 0.4
            sees[1] = False
            seen = np.zeros((n, 2), np.uint64)
            for t in range(n):
                for u in np.flatnonzero(sees[t]):
                    seen[t, u // 64] |= np.uint64(1 << int(u) % 64)
            seen[:, 0] |= np.uint64(1 << 40)      # new token 40 is not there
            seen[:, 1] = np.uint64(2 ** 64 - 1)
            trees.append((seen, rng.integers(-3, 5, n).astype(np.int32), sees))
        out, lse = check(c, queries(c, G), trees, 0.1)
        assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
        # depths: below 0 they count as 0, and far ones leave nothing of the window
        far = [(t[0], np.where(np.arange(n) % 3 == 0, 2 ** 31 - 1, t[1]).astype(np.int32), t[2]) for t in trees]
        clipped = [(t[0], np.maximum(t[1], 0), t[2]) for t in far]
        seen = torch.from_numpy(np.concatenate([t[0] for t in far]).view(np.int64)).cuda()
        q = queries(c, G)
        got = attend(c, q, seen, i32(np.concatenate([t[1] for t in far])), 0.1, 20)
        want, wl = check(c, q, clipped, 0.1, 20)
        assert torch.equal(got[0], want) and torch.equal(got[1], wl)


@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "fp8")])
@pytest.mark.parametrize("G,q_len", [(1, [9, 6]), (4, [40, 20])])
def test_absent_pages(act, kv, G, q_len):
    kv_len = [300, 33]
    with Case(act, kv, 2048, 2, 64, q_len, kv_len, seed=65, drop=[(0, 0), (0, 2), (1, 0)]) as c:
        c.fill()
        there = [np.repeat((c.table_host[s] >= 0).all((0, 1)), c.T)[:m] for s, m in enumerate(kv_len)]
        check(c, queries(c, 2 * G), trees_for(c, 7, 1), 0.1, there=there)


def rewrite(c, k=None, v=None):
    starts = np.concatenate([[0], np.cumsum(c.kv_len)])
    L.lora_kv_write(c.cache, L.KvBatch(i32(starts), c.kvl, torch.from_numpy(c.full_table).cuda(), int(starts[-1]),
                                       max(c.kv_len)), c.k, c.v)
    return [host(x) for x in c.k.split(c.kv_len)], [host(x) for x in c.v.split(c.kv_len)]


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("G,n,window,wide", [(1, 9, 0, False), (1, 9, 12, False), (8, 40, 0, False), (8, 40, 30, False),
                                             (8, 80, 0, True)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(act, G, n, window, wide):
    m = 500
    make = wide_case if wide else Case
    args = (act, act, 4096, 128, 1, G, [n], [m]) if wide else (act, act, 4096, 1, 128, [n], [m])
    with make(*args, seed=66) as c:
        log("[case] tree attention, infinities, %s G %d n %d window %d" % (act, G, n, window))
        c.fill()
        base = m - n
        c.v[base + 2, 0, 5] = float("inf")       # a new token that some rows see
        c.v[base + 3, 0, 5] = float("-inf")
        c.v[base + 3, 0, 9] = float("nan")
        c.v[base + n - 1, 0, 11] = float("-inf")
        c.v[base - 3, 0, 5] = float("-inf")      # and tokens before them
        c.v[base - 3, 0, 20] = float("inf")
        c.v[base - 11, 0, 21] = float("nan")
        c.v[10, 0, 22] = float("inf")
        kd, vd = rewrite(c)
        rng = np.random.default_rng(8)
        trees = [rows_of(random_parents(rng, n, "tree"), 2, window)]
        check(c, queries(c, G), trees, 0.1, window, wide=wide, kd=kd, vd=vd)


@pytest.mark.parametrize("kv", ["f16", "fp8"])
@pytest.mark.parametrize("G,n", [(1, 9), (8, 40)])
def test_what_is_not_seen_has_no_influence(kv, G, n):
    # new tokens that no row sees hold NaN and infinities in K and V, and scale bytes out of range; so does what
    # lies behind the last token
    m = 200
    with Case("f16", kv, 4096, 1, 128, [n], [m], seed=67) as c:
        c.fill()
        rng = np.random.default_rng(9)
        seen, depth, sees = rows_of(random_parents(rng, n, "tree"), 1)
        gone = [4, 5, n - 1]
        for u in gone:
            sees[:, u] = False
            seen[:, 0] &= ~np.uint64(1 << u)
        q = queries(c, G)
        want, lse = check(c, q, [(seen, depth, sees)], 0.1)
        for u in gone:
            b, t = (m - n + u) // c.T, (m - n + u) % c.T
            for which in (0, 1):
                pg = int(c.full_table[0, which, 0, b])
                d = torch.arange(128, device="cuda")
                at = ((d // c.E) * c.T + t) * c.E + d % c.E if which == 0 else ((t // c.E) * 128 + d) * c.E + t % c.E
                if kv == "fp8":
                    c.pages[pg, at] = 0x7F
                    c.scales[pg, t] = 255
                else:
                    c.pages[pg].view(torch.int16)[at] = 0x7E00 if which else 0x7C00
        st = torch.from_numpy(seen.view(np.int64)).cuda()
        out, ls = attend(c, q, st, i32(depth), 0.1)
        assert torch.equal(out, want) and torch.equal(ls, lse)


@pytest.mark.parametrize("G,n", [(2, 5), (8, 30)])
def test_lengths_past_the_table_and_below_the_tokens(G, n):
    # fewer cached tokens than new ones (the first ones have no place), none, and more than the table holds
    q_len = [n, n, n]
    with Case("bf16", "bf16", 2048, 1, 64, q_len, [n, n, 400], seed=68, extra_blocks=0) as c:
        c.fill()
        trees = trees_for(c, 10, 1, kinds=("tree", "chain"))
        q = queries(c, G)
        cap = c.table_host.shape[3] * c.T
        c.full_table[:2, :, :, (n + c.T - 1) // c.T:] = -1
        for lens in ([n - 3, 0, 400], [2, -5, 400], [n, 1, cap + 7]):
            c.kvl.copy_(torch.tensor(lens, dtype=torch.int32))
            seen = torch.from_numpy(np.concatenate([t[0] for t in trees]).view(np.int64)).cuda()
            out, lse = attend(c, q, seen, i32(np.concatenate([t[1] for t in trees])), 0.1)
            torch.cuda.synchronize()
            for s in range(3):
                base = max(lens[s], 0) - n
                m = min(max(lens[s], 0), cap)
                see = np.zeros((n, max(m, 1)), bool)
                for t in range(n):
                    see[t, :max(min(base, m), 0)] = True
                    for u in np.flatnonzero(trees[s][2][t]):
                        if 0 <= base + u < m:
                            see[t, base + u] = True
                kd, vd = np.zeros((max(m, 1), 1, 64)), np.zeros((max(m, 1), 1, 64))
                have = min(m, len(c.kd[s]))
                kd[:have], vd[:have] = c.kd[s][:have], c.vd[s][:have]
                see[:, have:] = False
                r = slice(s * n, s * n + n)
                if lens[s] <= len(c.kd[s]):   # past what was filled lies anything
                    agree(host(out)[r], host(lse)[r], formula(host(q)[r], kd, vd, see, 0.1), "bf16", 2, "bf16", m + 1, str((lens, s)))


def test_rows_streams_strides_and_graphs():
    # rows behind the last sequence are left, rows have strides, another stream, two calls at once, a graph replayed
    q_len, kv_len = [20, 33], [150, 90]
    with Case("f16", "f16", 4096, 2, 128, q_len, kv_len, seed=69) as c:
        c.fill()
        rng = np.random.default_rng(11)
        parents = [random_parents(rng, n, "tree") for n in q_len]
        starts = np.concatenate([[0], np.cumsum(q_len)])
        big = torch.randn((c.n + 4, 3, 8, 128), device="cuda", generator=c.gen).half()
        q = big[:, 1]
        room = torch.full((c.n + 4, 16, 128), 9.0, dtype=torch.float16, device="cuda")
        out, lse = room[:, :8], torch.full((c.n + 4, 8), 9.0, device="cuda")
        b = L.KvBatch(c.q_start, c.kvl, c.table, c.n + 4, 33)
        seen = torch.zeros((c.n + 4, 1), dtype=torch.int64, device="cuda")
        depth = torch.zeros(c.n + 4, dtype=torch.int32, device="cuda")
        parent = i32(np.concatenate(parents + [np.zeros(4, int)]))
        make = L.prepare_kv_tree_build(c.q_start, parent, seen, depth)
        size = L.lora_kv_attend_workspace_size(c.cache, b, 8)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        call = L.prepare_kv_attend_tree(c.cache, b, L.KvTree(seen, depth), q, out, 0.1, lse=lse, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        make(side)
        call(side)
        torch.cuda.synchronize()
        assert bool((room[c.n:] == 9).all()) and bool((lse[c.n:] == 9).all()) and bool((room[:, 8:] == 9).all())
        trees = [rows_of(p, 1) for p in parents]
        want, wl = check(c, q[:c.n].contiguous(), trees, 0.1)
        assert torch.equal(out[:c.n], want) and torch.equal(lse[:c.n], wl)
        # two calls at once, each with its own workspace
        out2, ws2 = torch.zeros_like(room)[:, :8], torch.empty_like(ws)
        other = L.prepare_kv_attend_tree(c.cache, b, L.KvTree(seen, depth), q, out2, 0.1, workspace=ws2)
        torch.cuda.synchronize()
        for _ in range(5):
            call(side)
            other(torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(out2[:c.n], want) and torch.equal(out[:c.n], want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            make(torch.cuda.current_stream())
            call(torch.cuda.current_stream())
        for k in range(4):
            parents = [random_parents(rng, n, ("tree", "forest", "star", "chain")[k]) for n in q_len]
            parent.copy_(i32(np.concatenate(parents + [np.zeros(4, int)])))
            room.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            want, wl = check(c, q[:c.n].contiguous(), [rows_of(p, 1) for p in parents], 0.1)
            assert torch.equal(out[:c.n], want) and torch.equal(lse[:c.n], wl) and bool((room[c.n:] == 9).all())


def test_tokens_past_the_words_are_seen_by_none():
    n, m = 70, 100
    with Case("bf16", "bf16", 4096, 1, 128, [n], [m], seed=70) as c:
        c.fill()
        seen, depth, sees = rows_of(np.arange(n) - 1, 1)
        sees[:, 64:] = False
        got, gd = build([0, n], np.arange(n) - 1, 1)
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy().view(np.uint64), seen) and np.array_equal(gd.cpu().numpy(), depth)
        check(c, queries(c, 4), [(seen, depth, sees)], 0.1)


def test_long_caches_repeat():
    # the same bits run to run, tiles split over many blocks
    with Case("bf16", "fp8", 4096, 1, 128, [31, 8], [20000, 40001], seed=71) as c:
        c.fill()
        trees = trees_for(c, 12, 1, 3000, kinds=("tree",))
        q = queries(c, 4)
        first = check(c, q, trees, 0.1, 3000, rows=[0, 5, 7, 30])
        second = check(c, q, trees, 0.1, 3000, rows=[1])
        assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


# ---------------------------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------------------------
def units(p):
    p = np.nan_to_num(np.asarray(p, np.float64), nan=0.0)
    return np.floor(np.clip(p, 0, 1) * 2.0 ** 44).astype(np.int64)


def level(total, u):
    u = min(max(float(u), 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    return int(total) * int(np.floor(u * 2 ** 31)) >> 31


def verified(parents, drafted, target, u, us, most):
    """(tokens, path [n_seqs][most], n_out) by the definition; parents of each sequence."""
    V = target.shape[1]
    tokens, path = np.full((len(parents), most), -1), np.full((len(parents), most), -1)
    counts, a = [], 0
    for s, parent in enumerate(parents):
        n = len(parent)
        if n == 0:
            counts.append(0)
            continue
        at, taken, on = 0, [0], True
        while on:
            on = False
            raw = units(target[a + at])
            w, left = raw.copy(), 1 << 44
            if len(taken) == most:
                break
            for t in range(at + 1, min(n, 1024)):
                if parent[t] != at:
                    continue
                x = int(drafted[a + t])
                have = int(w[x]) if 0 <= x < V else 0
                if level(left, u[a + t]) < have:
                    tokens[s, len(taken) - 1] = x
                    taken.append(t)
                    at, on = t, True
                    break
                left = max(0, left - have)
                if 0 <= x < V:
                    w[x] = 0
        w = w if w.sum() else raw
        total = int(w.sum())
        tokens[s, len(taken) - 1] = int(np.searchsorted(np.cumsum(w), level(total, us[s]), side="right")) if total else -1
        path[s, :len(taken)] = taken
        counts.append(len(taken))
        a += n
    return tokens, path, np.array(counts)


def verify(parents, drafted, target, u, us, most, stream=None, extra=0):
    S = len(parents)
    starts = i32(np.concatenate([[0], np.cumsum([len(p) for p in parents])]))
    flat = i32(np.concatenate([np.asarray(p, np.int64) for p in parents] or [np.zeros(0)]))
    flat = torch.cat([flat, torch.zeros(target.shape[0] - flat.numel(), dtype=torch.int32, device="cuda")])
    out = [torch.full((S, most), 77, dtype=torch.int32, device="cuda") for _ in range(2)]
    n_out = torch.full((S,), 77, dtype=torch.int32, device="cuda")
    ws = torch.full((L.lora_spec_verify_tree_workspace_size(S, target.shape[1]),), 0xFF, dtype=torch.uint8, device="cuda")
    L.lora_spec_verify_tree(starts, flat, drafted, target, u, us, *out, n_out, ws, stream=stream)
    torch.cuda.synchronize()
    return out[0].cpu().numpy(), out[1].cpu().numpy(), n_out.cpu().numpy()


def same(parents, drafted, target, u, us, most):
    got = verify(parents, drafted, target, u, us, most)
    want = verified(parents, drafted.cpu().numpy(), target.float().cpu().numpy(), u.cpu().numpy(), us.cpu().numpy(), most)
    for x, y, name in zip(got, want, ("tokens", "path", "n_out")):
        assert np.array_equal(x, y), (name, np.argwhere(x != y)[:5], x[x != y][:5], y[x != y][:5])
    return got


def drafts(parents, V, dtype, seed, ld=0, few=6):
    """Rows with a few likely tokens, of which the drafts are drawn: siblings share ids now and then."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(len(p) for p in parents)
    logits = torch.randn((n, V), device="cuda", generator=g)
    hot = torch.randint(0, V, (n, few), device="cuda", generator=g)
    logits.scatter_(1, hot, 3.0 + np.log(V) * torch.rand((n, few), device="cuda", generator=g))
    target = torch.softmax(logits, 1)
    if ld:
        wide = torch.full((n, ld), 5.0, device="cuda")
        wide[:, :V] = target
        target = wide.to(dtype)[:, :V]
    else:
        target = target.to(dtype)
    rows = torch.from_numpy(np.concatenate([[max(x, 0) + a for x in p] for p, a in zip(
        parents, np.concatenate([[0], np.cumsum([len(p) for p in parents])]))]).astype(np.int64)).cuda()
    which = torch.randint(0, few, (n,), device="cuda", generator=g)
    drafted = hot[rows.clamp_max(n - 1), which].to(torch.int32)
    return drafted, target, torch.rand(n, device="cuda", generator=g), torch.rand(len(parents), device="cuda", generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 7, 511, 1000, 32000, 40001])
def test_random_trees(dtype, V):
    rng = np.random.default_rng(V)
    sizes = [1, 25, 0, 64, 7, 130, 0, 2]
    parents = [random_parents(rng, n, ("tree", "tree", "tree", "star", "forest", "tree", "tree", "chain")[s]) for s, n in enumerate(sizes)]
    log("[case] verify trees %s V %d" % (dtype, V))
    for seed in range(3):
        d, t, u, us = drafts(parents, V, dtype, seed, ld=V + 3 if seed == 1 else 0, few=min(6, V))
        same(parents, d, t, u, us, 9 if seed else 130)


def test_the_largest_trees_and_many_sequences():
    rng = np.random.default_rng(1)
    parents = [random_parents(rng, n, k) for n, k in ((1024, "tree"), (1100, "chain"), (1024, "star"))]
    d, t, u, us = drafts(parents, 700, torch.float32, 3)
    same(parents, d, t, u * 1e-6, us, 1030)       # long paths
    same(parents, d, t, u, us, 3)
    parents = [random_parents(rng, int(n), "tree") for n in rng.integers(0, 9, 400)]
    d, t, u, us = drafts(parents, 3001, torch.bfloat16, 4)
    same(parents, d, t, u, us, 9)
    parents = [random_parents(rng, int(n), "tree") for n in rng.integers(1, 9, 4)]
    d, t, u, us = drafts(parents, 1 << 18, torch.float16, 5)
    same(parents, d, t, u, us, 9)


@pytest.mark.parametrize("V", [600, 33000])
def test_rows_of_nothing_levels_and_bad_ids(V):
    # a star: every child is refused in turn; duplicates; ids outside; rows of one token, of nothing, of NaN
    n = 12
    parents = [np.where(np.arange(n), 0, -1)] * 5
    t = torch.zeros((5 * n, V), device="cuda")
    t[0, 3], t[0, 500] = 0.25, 0.75
    t[n, 9] = 1.0
    t[2 * n] = float("nan")
    t[2 * n, 17] = 0.5
    t[4 * n, 100:104] = 0.25
    d = torch.zeros(5 * n, dtype=torch.int32, device="cuda")
    d[:n] = i32([0, 3, 3, -1, V, 2 ** 31 - 1, -2 ** 31, 4, 3, 500, 500, 8])
    d[n:2 * n] = 5
    d[n + 7] = 9
    d[2 * n:3 * n] = 17
    d[4 * n:] = i32([0, 100, 100, 101, 101, 102, 102, 103, 103, 104, 105, 106])
    for u in (0.0, 0.2499999, 0.25, 0.5, 0.9999999, 1.0, 2.0, -1.0, float("nan")):
        for us in (0.0, 0.5, 0.99999994, 1.0, float("nan")):
            same(parents, d, t, torch.full((5 * n,), u, device="cuda"), torch.full((5,), us, device="cuda"), 5)


def test_probabilities_are_the_targets():
    # one row, two of its tokens drafted: how often each token comes out is its probability.  Of 65535 sequences
    # a frequency is off by 6 standard deviations, 6 * 0.5 / 256 = 0.0118, less than once in 10^8.
    S = 65535
    p = torch.tensor([0.4, 0.05, 0.3, 0.15, 0.1], device="cuda")
    parents = [np.array([-1, 0, 0])] * S
    g = torch.Generator(device="cuda").manual_seed(3)
    d = i32([0, 2, 1] * S)
    tokens, path, n_out = verify(parents, d, p.expand(3 * S, 5).contiguous(), torch.rand(3 * S, device="cuda", generator=g),
                                 torch.rand(S, device="cuda", generator=g), 2)
    first = np.bincount(tokens[:, 0], minlength=5) / S
    assert np.abs(first - p.cpu().numpy()).max() < 0.0118
    assert np.abs((n_out == 2).mean() - 0.35) < 0.0118


def test_verification_in_a_graph_and_on_a_stream():
    rng = np.random.default_rng(2)
    parents = [random_parents(rng, n, "tree") for n in (20, 9, 31)]
    for V in (1000, 50000):
        d, t, u, us = drafts(parents, V, torch.float32, 6)
        starts = i32(np.concatenate([[0], np.cumsum([len(p) for p in parents])]))
        flat = i32(np.concatenate(parents))
        tokens, path = (torch.zeros((3, 31), dtype=torch.int32, device="cuda") for _ in range(2))
        n_out = torch.zeros(3, dtype=torch.int32, device="cuda")
        ws = torch.empty(L.lora_spec_verify_tree_workspace_size(3, V), dtype=torch.uint8, device="cuda")
        call = L.prepare_spec_verify_tree(starts, flat, d, t, u, us, tokens, path, n_out, ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(torch.cuda.current_stream())
        for seed in range(4):
            nd, nt, nu, ns = drafts(parents, V, torch.float32, 7 + seed)
            for x, y in zip((d, t, u, us), (nd, nt, nu, ns)):
                x.copy_(y)
            tokens.fill_(50)
            g.replay()
            torch.cuda.synchronize()
            want = same(parents, d, t, u, us, 31)
            for x, y in zip((tokens, path, n_out), want):
                assert np.array_equal(x.cpu().numpy(), y)
