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
from kv_formula import agree, bound, formula, visible
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


def check_terms(c, q, kd, vd, p_type, terms, rows=None):
    """The kernel's results within the bound of `terms`, which weights of one term are not within."""
    out, lse = attend(c, q, 0.25)
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
