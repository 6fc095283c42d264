"""Attention of one sequence in 64 bits and how far the kernels may be from it.

A row's result is sum_j p_j v_j / sum_j p_j.  What a kernel rounds:
  * scores: dot products of D terms in fp32 times a rounded scale, within
    (D + 4) 2^-24 scale sum |q| |k| =: e of the value, so p by a factor of exp(2 e) (products of few small
    whole numbers are exact: 4 instead of D + 4);
  * p, in the second product's operand type of unit roundoff u (2^-8 for bf16's 8-bit significand,
    2^-11 for f16's 11): one term u p, two terms u^2 p.  f16 has no numbers between 0 and 2^-24: p is
    held times 2^7 and is off by at most 2^-32 more (of a maximum's 1), of any size;
  * sums of S keys in fp32, at worst (S + 64) 2^-24 of sum p |v|;
  * the output, once, to its type.
"""
import numpy as np

UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # unit roundoff of the format


def visible(pos, n_keys, window=0, there=None):
    """Of tokens at positions pos: which of the keys 0 .. n_keys - 1 they see."""
    j, pos = np.arange(n_keys)[None], np.asarray(pos, np.int64)[:, None]
    see = j <= pos
    if window:
        see &= j > pos - window
    return see if there is None else see & np.asarray(there)[None]


def formula(q, k, v, see, scale, whole=False):
    """(out, lse, sum p |v|, sum |v|, e) of q [n][Hq][D] over k, v [m][H][D]; see [n][m].  Values of V that are
    not finite reach every row that sees them.  whole: the scores are products of whole numbers."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, size, all_v = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, err = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(n):
            at = np.flatnonzero(see[i])
            if at.size == 0:
                continue
            for h in range(Hq):
                kk, vv = k[at, h // G], v[at, h // G]
                x = scale * (kk @ q[i, h])
                p = np.exp(x - x.max())
                out[i, h] = p @ vv / p.sum()
                size[i, h] = p @ np.abs(vv) / p.sum()
                all_v[i, h] = np.abs(vv).sum(0) / p.sum()
                lse[i, h] = x.max() + np.log(p.sum())
                err[i, h] = (4 if whole else D + 4) * 2.0 ** -24 * scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, size, all_v, err


def bound(want, p_type, terms, act, n_keys):
    """Largest difference of each output element from formula()'s."""
    out, _, size, all_v, err = want
    floor = 2.0 ** -32 * all_v if p_type == "f16" else 0.0
    tiny = 2.0 ** -25 if act == "f16" else 2.0 ** -134
    part = UNIT[p_type] ** terms + (n_keys + 64) * 2.0 ** -24 + np.expm1(2 * err)[..., None]
    return (1 + 2 * UNIT[act]) * (part * size + floor) + UNIT[act] * np.abs(out) + tiny


def agree(out, lse, want, p_type, terms, act, n_keys, what=""):
    ro, rl, _, _, err = want
    with np.errstate(invalid="ignore"):
        tol = bound(want, p_type, terms, act, n_keys)
        fine = np.isfinite(ro)
        assert np.array_equal(np.isnan(out), np.isnan(ro)), what + ": NaN"
        other = ~fine & ~np.isnan(ro)
        assert np.array_equal(out[other], ro[other]), what + ": infinities"
        off = np.abs(out - ro)[fine] / tol[fine]
        assert off.size == 0 or off.max() <= 1, "%s: %.3g of the bound at %d of %d" % (what, off.max(), (off > 1).sum(), off.size)
        if lse is not None:
            assert np.array_equal(np.isneginf(lse), np.isneginf(rl)), what + ": empty rows"
            f = np.isfinite(rl)
            assert np.all(np.abs(lse - rl)[f] <= (err + 2.0 ** -21 * np.maximum(1, np.abs(rl)))[f]), what + ": lse"
    return off
