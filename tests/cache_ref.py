"""64-bit references of the cache operators (numpy, from the definitions) and the bounds their
tests use.

Bounds (u24 = 2^-24, the rounding of one fp32 operation; bf16 rounds by at most 2^-8 of the
value):
  * a score s = scale q.k is a sum of Dqk exact products: its fp32 error is at most
    (Dqk + 8) u24 scale sum_d |q_d k_d| (8 for the scaling and the change to base 2);
  * exp2 of the hardware and the log2 at the end are good to 2^-21 each, and the exponent's
    own rounding adds |s - m| u24 log2(e) <= 2^-23 max|s|;  together `ds` below bounds the error
    of a score, and of lse, which moves by at most the largest change of a score;
  * a weight exp(s - lse) then has the relative error 2 ds + 2^-20, and so has a sum of them
    (positive terms; n terms added in fp32 in runs and a running sum: at most 2^-24 times the
    number of additions in a row, 2^-24 (128 + n / 32));
  * o = sum_j p_j v_j: p is rounded to bf16 for the tensor cores (2^-8), its sum is not, and o
    is rounded to bf16: at most 2^-8 (sum_j p_j |v_j| + |o|), and (2 ds + 2^-20) sum_j p_j |v_j|.
"""
import numpy as np

U24 = 2.0 ** -24


def score_bound(q, k, scale):
    """max error of a score and of the lse for rows q [n, D] over keys k [m, D] (float64)."""
    if k.shape[0] == 0:
        return 2.0 ** -20
    mag = scale * np.abs(q) @ np.abs(k).T
    return (q.shape[1] + 8) * U24 * mag.max() + 2.0 ** -20 + 2.0 ** -22 * mag.max()


def softmax_rows(q, k, v, scale):
    """o [n, Dv], lse [n], p [n, m] and the bound's sum_j p_j |v_j| of rows over a key set."""
    n = q.shape[0]
    if k.shape[0] == 0:
        return (np.zeros((n, v.shape[1])), np.full(n, -np.inf), np.zeros((n, 0)),
                np.zeros((n, v.shape[1])))
    s = scale * (q @ k.T)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(1, keepdims=True)
    p = e / z
    return p @ v, (m + np.log(z))[:, 0], p, p @ np.abs(v)


def cache_attn(q, kc, vc, lens, kp, vp, scale, weights=None):
    """References of cache_attn_fwd on float64 arrays: o, lse, weights_out and their bounds."""
    B, _, HQ, _ = q.shape
    S, HK, Dv = kc.shape[1], kc.shape[2], vc.shape[3]
    G, P = HQ // HK, 0 if kp is None else kp.shape[0]
    o, lse = np.zeros((B, 1, HQ, Dv)), np.zeros((B, HQ, 1))
    w = np.zeros((B, HK, S)) if weights is None else weights.copy()
    o_tol, lse_tol, w_tol = np.zeros_like(o), np.zeros_like(lse), np.zeros_like(w)
    for b in range(B):
        n = int(min(max(lens[b], 0), S))
        for g in range(HK):
            hs = slice(g * G, (g + 1) * G)
            k, v = kc[b, :n, g], vc[b, :n, g]
            if P:
                k, v = np.concatenate([kp[:, g], k]), np.concatenate([vp[:, g], v])
            rows = q[b, 0, hs]
            oo, ll, p, pv = softmax_rows(rows, k, v, scale)
            ds = score_bound(rows, k, scale)
            o[b, 0, hs], lse[b, hs, 0] = oo, ll
            o_tol[b, 0, hs] = 2.0 ** -8 * (pv + np.abs(oo)) + (2 * ds + 2.0 ** -20) * pv + 1e-30
            lse_tol[b, hs, 0] = ds
            step = p[:, P:].sum(0)
            w[b, g, :n] += step
            # (one rounding of the total, G roundings of the step's sum)
            w_tol[b, g, :n] = (2 * ds + 2.0 ** -20 + G * U24) * step + U24 * np.abs(w[b, g, :n])
    return (o, lse, w), (o_tol, lse_tol, w_tol)


def key_weights(q, k, lse, allowed, scale):
    """Reference of sparse_attn_key_weights: allowed is bool [B, HK, Sq, Sk]."""
    B, Sq, HQ, _ = q.shape
    Sk, HK = k.shape[1], k.shape[2]
    G = HQ // HK
    w, tol = np.zeros((B, HK, Sk)), np.zeros((B, HK, Sk))
    for b in range(B):
        for h in range(HQ):
            g = h // G
            s = scale * (q[b, :, h] @ k[b, :, g].T)
            live = np.isfinite(lse[b, h])
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.where(allowed[b, g] & live[:, None], np.exp(s - lse[b, h][:, None]), 0.0)
            w[b, g] += p.sum(0)
            rel = 2 * score_bound(q[b, :, h], k[b, :, g], scale)
            # lse is an fp32 input: its change to base 2 rounds once more
            big = np.abs(lse[b, h][live]).max() if live.any() else 0.0
            tol[b, g] += (rel + 2.0 ** -22 * big) * p.sum(0)
    return w, tol + w * U24 * (128 + Sq * G / 32)


def evict(k, v, weights, lens, budget, sinks, recent):
    """Reference of cache_evict: per sequence and head the kept positions."""
    B, S, HK = k.shape[:3]
    keep = np.full((B, HK, budget), -1, np.int32)
    for b in range(B):
        n = int(min(max(lens[b], 0), S))
        for g in range(HK):
            if n <= budget:
                keep[b, g, :n] = np.arange(n)
                continue
            w = weights[b, g].astype(np.float64)
            w = np.where(np.isnan(w), np.inf, w)
            nan = np.isnan(weights[b, g])
            mid = sorted(range(sinks, n - recent), key=lambda i: (not nan[i], -w[i], i))
            mid = mid[:budget - sinks - recent]
            keep[b, g] = sorted([*range(sinks), *mid, *range(n - recent, n)])
    return keep
