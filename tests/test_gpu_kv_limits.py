"""KV cache and attention at the limits of what their calls describe: lengths past the table, rows past the
call's tokens, values that are not finite anywhere, weights of every size."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gather_lora_matmul_amd as L
from gpu_helpers import log
from kv_formula import UNIT, agree, bound, formula, visible
from test_gpu_kv import TD, Case, attend, dequant, quant, wide_case


def i32(x):
    return torch.tensor(np.asarray(x, np.int32)).cuda()


def host(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------------------------
# terms of the weights
# ---------------------------------------------------------------------------------------------
def one_term(q, k, v, see, scale, p_type):
    """formula()'s result with the weights rounded once to the operand's type."""
    n, Hq, D = q.shape
    out = np.zeros((n, Hq, D))
    for i in range(n):
        at = np.flatnonzero(see[i])
        for h in range(Hq):
            x = scale * (k[at, h * k.shape[1] // Hq] @ q[i, h])
            p = np.exp(x - x.max())
            r = torch.from_numpy(p).to(TD[p_type]).double().numpy()
            out[i, h] = r @ v[at, h * k.shape[1] // Hq] / p.sum()
    return out


def whole_scores(c, n_heads, spread=2):
    """Keys and queries of small whole numbers in eight places: exact scores, a few keys with large weights."""
    c.k[:, :, 8:] = 0
    c.k[:, :, :8] = torch.randint(-3, 4, (*c.k.shape[:2], 8), device="cuda", generator=c.gen).to(c.k.dtype)
    starts = np.concatenate([[0], np.cumsum(c.kv_len)])
    L.lora_kv_write(c.cache, L.KvBatch(i32(starts), c.kvl, torch.from_numpy(c.full_table).cuda(), int(starts[-1]),
                                       max(c.kv_len)), c.k, c.v)
    q = torch.zeros((c.n, n_heads, c.D), device="cuda")
    q[:, :, :8] = torch.randint(-spread, spread + 1, (c.n, n_heads, 8), device="cuda", generator=c.gen).float()
    return q.to(TD[c.act]), [host(x) for x in c.k.split(c.kv_len)]


def check_terms(c, q, kd, vd, p_type, terms, rows=None, batch=None):
    """The kernel's results within the bound of `terms`, which weights of one term are not within."""
    out, lse = attend(c, q, 0.25, batch=batch)
    torch.cuda.synchronize()
    worst, at = 0.0, 0
    for s, (n, m) in enumerate(zip(c.q_len, c.kv_len)):
        if s in (0, 1, len(c.q_len) // 2, len(c.q_len) - 1):
            r = at + (np.arange(n) if rows is None else np.array(rows[s]))
            x = host(q)[r]
            see = visible(m - n + r - at, m)
            want = formula(x, kd[s], vd[s], see, 0.25, whole=True)
            agree(host(out)[r], host(lse)[r], want, p_type, terms, c.act, m, "sequence %d" % s)
            once = np.abs(one_term(x, kd[s], vd[s], see, 0.25, p_type) - want[0])
            worst = max(worst, float((once / bound(want, p_type, 2, c.act, m)).max()))
        at += n
    assert worst > 3, "weights of one term would pass: %g" % worst


TYPES = [("f16", "f16", 128), ("bf16", "bf16", 128), ("bf16", "fp8", 128), ("f16", "fp8", 128),
         ("f16", "f16", 64), ("bf16", "bf16", 64), ("bf16", "fp8", 64), ("f16", "fp8", 64)]


@pytest.mark.parametrize("act,kv,D", TYPES)
@pytest.mark.parametrize("S,H,G,n,m", [(1, 8, 1, 1, 130), (2, 2, 8, 2, 99), (2, 2, 4, 4, 64), (1100, 1, 1, 1, 70)])
def test_weights_of_few_rows_have_two_terms(act, kv, D, S, H, G, n, m):
    with Case(act, kv, 8192, H, D, [n] * min(S, 1024), [m] * min(S, 1024), seed=47, extra_blocks=0) as c:
        log("[case] terms, few rows %s/%s D %d: %d x %d rows of %d heads" % (act, kv, D, S, n * G, H))
        _, vd = c.fill()
        q, kd = whole_scores(c, H * G)
        check_terms(c, q, kd, vd, "bf16" if kv == "fp8" else act, 2)


@pytest.mark.parametrize("act,kv,D", TYPES)
@pytest.mark.parametrize("H,G,q_len,kv_len", [(1, 8, [5], [100]), (2, 4, [60, 1], [131, 80]), (5, 3, [40, 7], [90, 33])])
def test_weights_of_tiles_have_two_terms(act, kv, D, H, G, q_len, kv_len):
    # of the activations' type, over FP8 caches too
    with Case(act, kv, 8192, H, D, q_len, kv_len, seed=48, extra_blocks=0) as c:
        log("[case] terms, tiles %s/%s D %d H %d G %d %s" % (act, kv, D, H, G, q_len))
        _, vd = c.fill()
        q, kd = whole_scores(c, H * G)
        check_terms(c, q, kd, vd, act, 2)


@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")])
def test_weights_of_long_work_have_one_term(act, kv):
    # tiles of 256 rows
    q_len, kv_len = [100, 60], [140, 99]
    with wide_case(act, kv, 4096, 128, 1, 8, q_len, kv_len, seed=49) as c:
        log("[case] terms, wide %s/%s" % (act, kv))
        _, vd = c.fill()
        q, kd = whole_scores(c, 8)
        check_terms(c, q, kd, vd, act, 1, rows=[[0, 31, 32, 99], [0, 1, 59]])


@pytest.mark.parametrize("act,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")])
def test_weights_of_long_work_have_two_terms_for_those_who_ask(act, kv):
    q_len, kv_len = [100, 60], [140, 99]
    with wide_case(act, kv, 4096, 128, 1, 8, q_len, kv_len, seed=49) as c:
        log("[case] terms, wide with two %s/%s" % (act, kv))
        _, vd = c.fill()
        q, kd = whole_scores(c, 8)
        b = L.KvBatch(c.q_start, c.kvl, c.table, c.n, max(q_len), two_terms=True)
        check_terms(c, q, kd, vd, act, 2, rows=[[0, 31, 32, 99], [0, 1, 59]], batch=b)
        one, _ = attend(c, q, 0.25)
        two, _ = attend(c, q, 0.25, batch=b)
        assert not torch.equal(one, two)


# ---------------------------------------------------------------------------------------------
# lengths past the table and rows past the call's tokens: nothing moves
# ---------------------------------------------------------------------------------------------
# q_start, n_tokens, kv_len of one sequence over a table of 64 tokens -> (first kept row, its position)
CUT = [
    ([0, 1], 1, 65, (0, 64)),                # one token past the table
    ([0, 5], 5, 66, (0, 61)),                # the last of five, too
    ([0, 3], 3, 67, (0, 64)),                # all of them
    ([0, 40], 40, 90, (0, 50)),
    ([0, 2], 2, 2 ** 31 - 1, (0, 2 ** 31 - 3)),
    ([0, 10], 8, 40, (0, 30)),               # rows past the call's tokens
    ([0, 30], 20, 80, (0, 50)),              # both
    ([-2, 5], 5, 40, (0, 35)),               # rows before the first
    ([-2 ** 31, 5], 5, 40, (0, 35)),
    ([0, 2 ** 31 - 1], 6, 2 ** 31 - 1, (0, 0)),
    ([3, 9], 7, 64, (3, 58)),
    ([0, 6], 6, -7, (0, -6)),                # a length below none is none
]


def kept(q_start, n, kv_len, first):
    """Rows of the call's tensors that belong to the sequence and their positions."""
    rows = np.arange(first[0], min(n, max(q_start[1], first[0])))
    return rows, first[1] + rows - first[0]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("q_start,n,kv_len,first", CUT)
def test_write_and_read_past_the_table_and_the_tokens(kv, q_start, n, kv_len, first):
    page = 4096 if kv == "bf16" else 2048
    with Case("bf16", kv, page, 2, 128, [0], [64], seed=40, extra_blocks=0) as c:
        assert c.T == 32 and c.full_table.shape[3] == 2
        c.fill()
        before, scales = c.pages.clone(), None if c.scales is None else c.scales.clone()
        k = torch.randn((n, 2, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        v = torch.randn((n, 2, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        b = L.KvBatch(i32(q_start), i32([kv_len]), c.table, n, n)
        rows, pos = kept(q_start, n, kv_len, first)
        has = (pos >= 0) & (pos < 64)
        L.lora_kv_write(c.cache, b, k, v)
        ko, vo = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
        L.lora_kv_read(c.cache, b, ko, vo)
        # the whole cache, the rows' places among it
        ka, va = torch.empty_like(c.k), torch.empty_like(c.v)
        L.lora_kv_read(c.cache, L.KvBatch(i32([0, 64]), c.kvl, c.table, 64, 64), ka, va)
        torch.cuda.synchronize()
        for new, old, out, whole in ((k, c.k, ko, ka), (v, c.v, vo, va)):
            stored = (lambda x: torch.from_numpy(dequant(*quant(host(x)))).to(torch.float32).to(x.dtype).cuda()) if c.fp8 \
                else (lambda x: x)
            want = stored(old).clone()
            want[pos[has]] = stored(new)[rows[has]]
            assert torch.equal(whole, want)
            kept_rows = torch.zeros(n, dtype=torch.bool)
            kept_rows[rows[has]] = True
            assert torch.equal(out[rows[has]], stored(new)[rows[has]])
            assert torch.all(out[~kept_rows.cuda()] == 9.0)      # rows without a place are left
        if not has.any():
            assert torch.equal(c.pages, before) and (scales is None or torch.equal(c.scales, scales))


# few rows, tiles of 128 rows, tiles of 256 (a long table, of which one sequence uses the first blocks)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("group,n,q_start,kv_len", [
    (1, 1, [0, 1], 129), (4, 4, [0, 4], 130), (2, 6, [0, 8], 131), (2, 5, [-3, 5], 100), (1, 2, [0, 2], 2 ** 31 - 1),
    (4, 50, [0, 50], 140), (4, 40, [0, 60], 120), (4, 40, [0, 60], 150), (4, 40, [-5, 40], 110), (4, 30, [0, 30], 10 ** 9),
])
def test_attend_past_the_table_and_the_tokens(kv, window, group, n, q_start, kv_len):
    # pages of 40 (FP8: 80) tokens: the table's end lies inside a tile of keys
    cap = 120 if kv == "bf16" else 160
    with Case("bf16", kv, 5120, 1, 128, [0], [cap], seed=41, extra_blocks=0) as c:
        log("[case] past the table %s group %d rows %d %s kv_len %d window %d" % (kv, group, n, q_start, kv_len, window))
        kd, vd = c.fill()
        assert c.full_table.shape[3] * c.T == cap
        q = torch.randn((n, group, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        b = L.KvBatch(i32(q_start), i32([kv_len]), c.table, n, n)
        out, lse = attend(c, q, 0.1, window, batch=b)
        torch.cuda.synchronize()
        pos = kv_len - (q_start[1] - q_start[0]) + (np.arange(n) - q_start[0])
        see = visible(pos, cap, window)
        agree(host(out), host(lse), formula(host(q), kd[0], vd[0], see, 0.1), "bf16", 2, "bf16", cap)


@pytest.mark.parametrize("kv", ["f16", "fp8"])
def test_attend_wide_past_the_table(kv):
    # 8 waves: the first sequence ends inside its table, the second's lengths pass it
    act, G, n = "f16", 8, [100, 90]
    with wide_case(act, kv, 4096, 128, 1, G, n, [300, 200], seed=42) as c:
        nb = c.full_table.shape[3]
        cap = nb * c.T
        # the second sequence repeats its blocks over the whole table: the keys are those 200's over and over
        used = -(-200 // c.T)
        reps = -(-nb // (used - 1))
        c.table[1] = c.table[1, :, :, :used - 1].repeat(1, 1, reps)[:, :, :nb]
        kd, vd = c.fill()
        lens = [300, cap + 7]
        b = L.KvBatch(c.q_start, i32(lens), c.table, sum(n), 100)
        q = torch.randn((sum(n), G, 128), device="cuda", generator=c.gen).to(TD[act])
        q[100:, :, :] = 0   # all keys alike: the mean of the values
        out, lse = attend(c, q, 0.1, 0, batch=b)
        torch.cuda.synchronize()
        see = visible(300 - 100 + np.arange(100), 300)
        agree(host(out[:100]), host(lse[:100]), formula(host(q[:100]), kd[0], vd[0], see, 0.1), "f16", 1, act, 300)
        m = (used - 1) * c.T
        whole, rest = divmod(cap, m)
        vs = vd[1][:m, 0]
        pos = cap + 7 - 90 + np.arange(90)
        for i in (0, 1, 82, 83, 84, 89):
            keys = min(pos[i] + 1, cap)
            whole, rest = divmod(keys, m)
            want = (whole * vs.sum(0) + vs[:rest].sum(0)) / keys
            # equal weights are powers of two: only the sums and the output round
            tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -24 + (keys + 64) * 2.0 ** -24 * np.abs(vs).mean(0)
            assert np.all(np.abs(host(out[100 + i]) - want) <= tol), i
            assert np.all(np.abs(host(lse[100 + i]) - np.log(keys)) <= 2.0 ** -21 * np.log(keys) + 2.0 ** -21)


# ---------------------------------------------------------------------------------------------
# infinities in V, wherever their token lies
# ---------------------------------------------------------------------------------------------
def rewrite(c):
    """The cache again from c.k, c.v; the dense copies of one sequence with it."""
    m = c.kv_len[0]
    L.lora_kv_write(c.cache, L.KvBatch(i32([0, m]), c.kvl, torch.from_numpy(c.full_table).cuda(), m, m), c.k, c.v)
    c.kd, c.vd = [host(c.k)], [host(c.v)]


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,n", [(1, 1, 1), (1, 4, 4), (2, 2, 40), (600, 1, 1)])
@pytest.mark.parametrize("window", [0, 130])
def test_infinite_values_far_from_every_edge(act, H, G, n, window):
    # tokens that every row sees, in tiles of keys that every row sees whole; weights down to 2^-40
    many = H > 256   # sequences instead of heads: waves that work for themselves
    S, H = (H, 1) if many else (1, H)
    m = 150
    with Case(act, act, 4096, H, 128, [n] * S, [m] * S, seed=43, extra_blocks=0) as c:
        c.fill()
        c.k[:, :, 0] = -4.0 * torch.rand(c.k.shape[:2], device="cuda", generator=c.gen).to(c.k.dtype)
        c.k[m - 1::m, :, 0] = 0                       # the last token has the largest weight
        for s in range(S):
            at = s * m
            c.v[at + 70, 0, 3] = float("inf")
            c.v[at + 71, 0, 4] = -float("inf")
            c.v[at + 40, 0, 5] = float("inf")
            c.v[at + 90, 0, 5] = -float("inf")        # both: NaN
            c.v[at + 60, 0, 6] = float("nan")
        starts = np.arange(S + 1) * m
        L.lora_kv_write(c.cache, L.KvBatch(i32(starts), c.kvl, torch.from_numpy(c.full_table).cuda(), S * m, m), c.k, c.v)
        q = torch.randn((c.n, H * G, 128), device="cuda", generator=c.gen).to(TD[act])
        q[:, :, 0] = 70.0
        out, lse = attend(c, q, 0.1, window)
        torch.cuda.synchronize()
        few = n * G <= 16
        for s in (range(S) if S < 3 else (0, 1, S // 2, S - 1)):
            r = slice(s * n, s * n + n)
            kd, vd = host(c.k[s * m:s * m + m]), host(c.v[s * m:s * m + m])
            see = visible(m - n + np.arange(n), m, window)
            agree(host(out[r]), host(lse[r]), formula(host(q[r]), kd, vd, see, 0.1), act, 2 if few else 1, act, m)


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_infinite_values_of_small_weights_in_long_caches(act, n):
    # the weight of the infinite value is 2^-15 .. 2^-300 of the largest, which comes before it or
    # long after it (other tiles, other blocks' parts): any weight above zero times infinity is infinite
    m = 9000
    for first in (False, True):
        with Case(act, act, 8192, 1, 128, [n], [m], seed=44, extra_blocks=0) as c:
            c.fill()
            for drop in (15, 30, 140, 300):
                c.k[:] = 0
                top = 100 if first else m - 500
                c.k[top, 0, 0] = 8.0
                at = 5000 if first else 1000
                c.v[:] = torch.randn(c.v.shape, device="cuda", generator=c.gen).to(c.v.dtype)
                c.v[at, 0, 3] = float("inf")
                c.v[at + 1, 0, 7] = -float("inf")
                rewrite(c)
                q = torch.zeros((n, 2, 128), device="cuda", dtype=TD[act])
                q[:, :, 0] = drop / 8.0
                out, lse = attend(c, q, float(np.log(2.0)))
                torch.cuda.synchronize()
                see = visible(m - n + np.arange(n), m)
                agree(host(out), host(lse), formula(host(q), c.kd[0], c.vd[0], see, float(np.float32(np.log(2.0)))), act,
                      2 if 2 * n <= 16 else 1, act, m, "drop %d" % drop)


@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_wide_infinite_values_far_from_every_edge(act):
    n, lens = [90, 70], [700, 500]
    with wide_case(act, act, 4096, 128, 1, 8, n, lens, seed=45) as c:
        c.fill()
        c.k[:, :, 0] = -4.0 * torch.rand(c.k.shape[:2], device="cuda", generator=c.gen).to(c.k.dtype)
        for at, d, x in ((70, 3, "inf"), (330, 4, "-inf"), (200, 5, "inf"), (400, 5, "-inf"), (250, 6, "nan"),
                         (700 + 100, 3, "-inf")):
            c.v[at, 0, d] = float(x)
        L.lora_kv_write(c.cache, L.KvBatch(i32([0, 700, 1200]), c.kvl, torch.from_numpy(c.full_table).cuda(), 1200, 700), c.k, c.v)
        q = torch.randn((c.n, 8, 128), device="cuda", generator=c.gen).to(TD[act])
        q[:, :, 0] = 70.0
        out, lse = attend(c, q, 0.1)
        torch.cuda.synchronize()
        for s, (r, k) in enumerate(((slice(0, 90), slice(0, 700)), (slice(90, 160), slice(700, 1200)))):
            see = visible(lens[s] - n[s] + np.arange(n[s]), lens[s])
            agree(host(out[r]), host(lse[r]), formula(host(q[r]), host(c.k[k]), host(c.v[k]), see, 0.1), act, 1, act, lens[s])


# ---------------------------------------------------------------------------------------------
# weights of every size
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("S,n", [(1024, 1), (512, 17), (32, 512)])   # few rows, tiles of 128 and of 256 rows
@pytest.mark.parametrize("exponent", [-20, -26])
def test_many_small_weights_beside_a_large_one(act, S, n, exponent):
    # one key of weight 1 and 16000 of about 2^-20 or 2^-26, whose values are all that is left in half of
    # the elements; many sequences over the same pages, so that a worker walks many keys in one piece
    m = 16000
    with Case(act, act, 8192, 1, 128, [1], [m], seed=46, extra_blocks=0) as c:
        log("[case] small weights %s %d x %d, 2^%d" % (act, S, n, exponent))
        c.fill()
        c.k[:] = 0
        c.k[:, 0, 0] = (1 + 0.05 * torch.rand(m, device="cuda", generator=c.gen)).to(c.k.dtype)
        c.v[:] = (1 + torch.rand(c.v.shape, device="cuda", generator=c.gen)).to(c.v.dtype)
        c.k[7, 0, 0] = 0
        c.v[7, 0, :64] = 0
        L.lora_kv_write(c.cache, L.KvBatch(i32([0, m]), c.kvl, c.table, m, m), c.k, c.v)
        q = torch.zeros((S * n, 1, 128), device="cuda", dtype=TD[act])
        q[:, 0, 0] = float(exponent)
        scale = float(np.float32(np.log(2.0)))
        b = L.KvBatch(i32(np.arange(S + 1) * n), i32([m] * S), c.table.repeat(S, 1, 1, 1), S * n, n)
        out, lse = attend(c, q, scale, batch=b)
        torch.cuda.synchronize()
        rows = np.unique([0, n // 2, n - 1])
        see = visible(m - n + rows, m)
        want = formula(host(q)[rows], host(c.k), host(c.v), see, scale)
        for s in (0, 1, S // 2, S - 1):
            agree(host(out)[s * n + rows], host(lse)[s * n + rows], want, act, 2 if n < 512 else 1, act, m, "sequence %d" % s)


@pytest.mark.parametrize("group", [1, 32])
def test_a_longest_length_of_none_is_only_a_wrong_one(group):
    # max_q_len chooses among kernels: with none given the rows are computed all the same
    with Case("bf16", "bf16", 4096, 1, 128, [3, 1], [70, 33], seed=49) as c:
        kd, vd = c.fill()
        q = torch.randn((4, group, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        out, lse = attend(c, q, 0.1, batch=c.batch(max_q=0))
        torch.cuda.synchronize()
        for s, (r, n, m) in enumerate(((slice(0, 3), 3, 70), (slice(3, 4), 1, 33))):
            see = visible(m - n + np.arange(n), m)
            agree(host(out[r]), host(lse[r]), formula(host(q[r]), kd[s], vd[s], see, 0.1), "bf16", 2, "bf16", m)


# ---------------------------------------------------------------------------------------------
# tiles that go out whole
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("act,kv", [("bf16", "bf16"), ("f16", "fp8")])
@pytest.mark.parametrize("rows,S,H,G,n,length", [(128, 35, 5, 4, 96, 1000), (256, 22, 5, 4, 150, 1800)])
def test_whole_rounds_of_tiles_and_a_cut_rest(act, kv, rows, S, H, G, n, length):
    # tiles about equally long, more than the workers are: whole rounds of them, then the others cut into ranges
    # from the middle of a sequence's tiles on
    q_len, kv_len = [n - (s % 3 == 1) for s in range(S)], [length + 7 * (s % 4) for s in range(S)]
    with Case(act, kv, 8192, H, 128, q_len, kv_len, seed=51, extra_blocks=0) as c:
        workers = torch.cuda.get_device_properties(0).multi_processor_count * (512 // rows) // 2
        tiles = [-(-x * G // rows) for x in q_len]
        # units of 64 keys of each tile, to its last row's position
        units = [sum(-(-(m - x + (min((t + 1) * rows, x * G) - 1) // G + 1) // 64) for t in range(k))
                 for x, m, k in zip(q_len, kv_len, tiles)]
        T, longest = sum(tiles) * H, max(-(-m // 64) for m in kv_len)
        whole = T // workers * workers
        if whole == 0 or whole == T:
            pytest.skip("made for 256 compute units")
        assert S <= 64 and 8 * T * longest <= 9 * sum(units) * H          # the rule of whole tiles
        assert (256 if sum(q_len) * G >= 512 * S else 128) == rows
        first = int(np.searchsorted(np.cumsum(tiles) * H, whole, side="right"))   # sequence of the first cut tile
        assert (whole - sum(tiles[:first]) * H) % tiles[first]
        kd, vd = c.fill()
        q = torch.randn((c.n, H * G, 128), device="cuda", generator=c.gen).to(TD[act])
        out, lse = attend(c, q, 0.1)
        again = attend(c, q, 0.1)
        torch.cuda.synchronize()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        off = np.concatenate([[0], np.cumsum(q_len)])
        for s in sorted({0, first - 1, first, S - 1}):
            r = np.arange(off[s], off[s + 1])[[0, 1, 31, 32, 63, 64, -2, -1]]
            see = visible(kv_len[s] - q_len[s] + r - off[s], kv_len[s])
            agree(host(out)[r], host(lse)[r], formula(host(q)[r], kd[s], vd[s], see, 0.1), act, 2 if rows == 128 else 1,
                  act, kv_len[s], "sequence %d" % s)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("size", [65504.0, 63488.0, 2.0 ** -8, 2.0 ** -14, 2.0 ** -20])
def test_fp8_caches_of_f16_rows_of_every_size(n, size):
    # rows from f16's smallest numbers to its largest, whose codes may stand for 65536 (past f16).  In tiles
    # K and V are f16 numbers at half their size: off by 2^-24 at most
    m = 200
    with Case("f16", "fp8", 4096, 1, 128, [n], [m], seed=50) as c:
        c.fill()
        g = lambda: torch.empty((m, 1, 128), device="cuda").uniform_(-1, 1, generator=c.gen)
        for k_size in (1.0, size):
            c.k = (g() * k_size).to(torch.float16)
            c.v = (g() * size).to(torch.float16)
            c.v[:, 0, 5] = size
            L.lora_kv_write(c.cache, L.KvBatch(i32([0, m]), c.kvl, torch.from_numpy(c.full_table).cuda(), m, m), c.k, c.v)
            kd, vd = dequant(*quant(host(c.k))), dequant(*quant(host(c.v)))
            q = torch.empty((n, 2, 128), device="cuda").uniform_(-1, 1, generator=c.gen).to(torch.float16)
            scale = 0.2 / k_size
            out, lse = attend(c, q, scale)
            torch.cuda.synchronize()
            see = visible(m - n + np.arange(n), m)
            out_, lse_, sz, al, err = formula(host(q), kd, vd, see, scale)
            p_type, terms = ("bf16", 2) if n == 1 else ("f16", 1)
            if n > 1:
                err = err + scale * 2.0 ** -24 * np.abs(host(q)).sum(-1)
                sz = sz + 2.0 ** -24 / UNIT["f16"]      # of V, whole: u of this is 2^-24
            big = np.abs(out_) > 65504                     # rounds to infinity
            o = np.where(big & np.isinf(host(out)), out_, host(out))
            assert np.isinf(host(out)[np.abs(out_) >= 65520 * (1 + 2.0 ** -10)]).all()
            agree(o, host(lse), (out_, lse_, sz, al, err), p_type, terms, "f16", m, "size %g k %g" % (size, k_size))


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("n,G,wide", [(3, 4, False), (100, 1, False), (90, 8, True)])
@pytest.mark.parametrize("window", [0, 250])
def test_infinities_that_some_rows_see_beside_others(act, n, G, wide, window):
    # in columns with an infinity that all rows see: opposite ones that the first or the last rows of a wave see
    m = 400
    base = m - n
    make = wide_case if wide else (lambda a, k, p, D, H, g, ql, kl, **kw: Case(a, k, p, H, D, ql, kl, **kw))
    with make(act, act, 4096, 128, 1, G, [n], [m], seed=52) as c:
        c.fill()
        early = max(base - window, 0) + (n + 1) // 2 if window else 20
        for at, d, x in ((200, 3, "inf"), (base + (n + 1) // 2, 3, "-inf"), (200, 4, "-inf"), (early, 4, "inf"),
                         (m - 1, 5, "inf"), (early, 6, "nan"), (230, 7, "inf"), (230, 8, "nan"), (base, 8, "inf")):
            c.v[at, 0, d] = float(x)
        rewrite(c)
        q = torch.randn((n, G, 128), device="cuda", generator=c.gen).to(TD[act])
        out, lse = attend(c, q, 0.1, window)
        torch.cuda.synchronize()
        see = visible(base + np.arange(n), m, window)
        agree(host(out), host(lse), formula(host(q), c.kd[0], c.vd[0], see, 0.1), act, 1 if wide else 2, act, m)
        assert np.isinf(host(out)[:, :, 7]).all() and np.isnan(host(out)[:, :, 8]).all()
        assert 0 < np.isnan(host(out)[:, 0, 3]).sum() < n and np.isinf(host(out)[0, :, 3]).all()


def test_windows_past_32_bits_are_none():
    with Case("bf16", "bf16", 4096, 1, 128, [2], [70], seed=53) as c:
        c.fill()
        q = torch.randn((2, 2, 128), device="cuda", generator=c.gen).to(TD["bf16"])
        want, lse = attend(c, q, 0.1)
        for window in (10 ** 12, 2 ** 63 - 1, 2 ** 32 + 5, 2 ** 31):
            got, ls = attend(c, q, 0.1, window)
            assert torch.equal(got, want) and torch.equal(ls, lse)
        for window in (-1, -2 ** 31 - 1, -2 ** 32 + 5):
            with pytest.raises(L.LoraError, match="window"):
                attend(c, q, 0.1, window)
