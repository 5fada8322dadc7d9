"""Cached attention in plain form (oracle): append with the position rotation,
mean keys of full pages, choice of pages, attention of single rows.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).  Row by row, from the
definitions in include/tiered_attn_cache.h; fp64 but where a value's own
definition says fp32.  A cache is held as two dicts of arrays,
``{"k": codes-or-values [P, Hkv, ps, d], "ks": scales [P, Hkv, ps] or None}``.
"""

from __future__ import annotations

import math

import numpy as np

from .formats import bf16_rne, e4m3_decode, e4m3_encode


def rows_of(lens, cu, S):
    """(row, sequence, position) of every row in use; position None where a
    row has none."""
    out = []
    for s in range(S):
        rows = range(s, s + 1) if cu is None else range(cu[s], cu[s + 1])
        end = s + 1 if cu is None else cu[s + 1]
        for t in rows:
            p = int(lens[s]) - (end - t)
            out.append((t, s, p if 0 <= p < lens[s] else None))
    return out


def rotate32(x, cos, sin, inter):
    """fp32 rotation of [..., d] with every operation rounded by itself."""
    x = np.asarray(x, np.float32)
    r2 = cos.shape[-1]
    a, b = (x[..., 0:2 * r2:2], x[..., 1:2 * r2:2]) if inter else (x[..., :r2], x[..., r2:2 * r2])
    c, s = np.asarray(cos, np.float32), np.asarray(sin, np.float32)
    u, w = a * c - b * s, b * c + a * s
    y = x.copy()
    if inter:
        y[..., 0:2 * r2:2], y[..., 1:2 * r2:2] = u, w
    else:
        y[..., :r2], y[..., r2:2 * r2] = u, w
    return y


def rotate64(x, cos, sin, inter):
    """The same in fp64 (the products of a bf16 and an fp32 value are exact)."""
    x = np.asarray(x, np.float64)
    r2 = cos.shape[-1]
    a, b = (x[..., 0:2 * r2:2], x[..., 1:2 * r2:2]) if inter else (x[..., :r2], x[..., r2:2 * r2])
    c, s = np.asarray(cos, np.float64), np.asarray(sin, np.float64)
    u, w = a * c - b * s, b * c + a * s
    y = x.copy()
    if inter:
        y[..., 0:2 * r2:2], y[..., 1:2 * r2:2] = u, w
    else:
        y[..., :r2], y[..., r2:2 * r2] = u, w
    return y


def token_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-126 with amax <= 448 s; 1 for 0.  NaN for
    what is not finite in fp32 (a rotated key may pass it)."""
    if not amax < float(np.finfo(np.float32).max):
        return math.nan
    if amax == 0.0:
        return 1.0
    m, e = math.frexp(amax)
    return math.ldexp(1.0, max(e - 9 if m <= 0.875 else e - 8, -126))


def append(k, v, ks, vs, mean, K, V, lens, cu, table, cos=None, sin=None, inter=False, pos=None,
           fp8=False):
    """Write rows K, V [T, Hkv, d] into the cache arrays in place (codes and
    scales, FP8; bf16 values otherwise) and the means of the pages filled."""
    ps = k.shape[2]
    filled = {}
    for t, s, p in rows_of(lens, cu, len(lens)):
        if p is None:
            continue
        a = p if pos is None else pos[t]
        page, slot = table[s][p // ps], p % ps
        if fp8:
            x = rotate64(K[t], cos[a], sin[a], inter) if cos is not None else np.float64(K[t])
            for arr, sc, y in ((k, ks, x), (v, vs, np.float64(V[t]))):
                for h in range(y.shape[0]):
                    f = token_scale(np.abs(y[h]).max() if np.isfinite(y[h]).all() else math.nan)
                    sc[page, h, slot] = f
                    if math.isfinite(f):
                        arr[page, h, slot] = e4m3_encode(y[h] / f)
        else:
            x = rotate32(K[t], cos[a], sin[a], inter) if cos is not None else np.float32(K[t])
            k[page, :, slot] = bf16_rne(np.float64(x))
            v[page, :, slot] = V[t]
        if slot == ps - 1:
            filled[page] = True
    if mean is not None:
        for page in filled:
            x = decoded(k, ks, fp8)[page].astype(np.float32)       # [Hkv, ps, d]
            acc = np.zeros((x.shape[0], x.shape[2]), np.float32)
            for r in range(ps):
                acc = acc + x[:, r]
            mean[page] = acc * np.float32(1.0 / ps)


def decoded(x, scales, fp8):
    return e4m3_decode(x) * np.float64(scales)[..., None] if fp8 else np.float64(x)


def keys_of(x, table_row, n, h):
    """The first n decoded keys or values of a sequence for head h."""
    ps = x.shape[2]
    if n == 0:
        return np.zeros((0, x.shape[3]))
    pages = [table_row[j] for j in range(-(-n // ps))]
    return x[pages, h].reshape(-1, x.shape[3])[:n]


def attend(q, K, V, scale):
    """(O, lse, A, smax): softmax(scale q K^T) V of one query, its log sum,
    sum_i p_i |v_i|, and a bound of the sums' magnitudes scale * sum_c |q_c k_c|."""
    if K.shape[0] == 0:
        return np.zeros(V.shape[1]), -math.inf, np.zeros(V.shape[1]), 0.0
    s = K @ q * scale
    m = s.max()
    e = np.exp(s - m)
    z = e.sum()
    return e @ V / z, m + math.log(z), e @ np.abs(V) / z, float((np.abs(K) @ np.abs(q)).max() * scale)


def select(Q, mean, lens, cu, table, G, ps, n_select, n_first, n_recent, scale):
    """sel [T, Hkv, n_select]; rows not in use keep -2."""
    T, Hkv = Q.shape[0], mean.shape[1]
    out = np.full((T, Hkv, n_select), -2, np.int32)
    for t, s, p in rows_of(lens, cu, len(lens)):
        n = 0 if p is None else p // ps + 1
        for h in range(Hkv):
            if n <= n_select:
                ids = list(range(n))
            else:
                cand = list(range(n_first, n - n_recent))
                mass = np.zeros(len(cand))
                kb = np.float64(mean[[table[s][j] for j in cand], h])
                for g in range(G):
                    with np.errstate(invalid="ignore"):
                        lg = kb @ np.float64(Q[t, h * G + g]) * scale
                    ok = np.isfinite(lg)
                    if ok.any():
                        e = np.where(ok, np.exp(np.where(ok, lg, 0) - lg[ok].max()), 0.0)
                        mass += e / e.sum()
                order = sorted(range(len(cand)), key=lambda i: (-mass[i], i))
                ids = sorted(list(range(n_first)) + list(range(n - n_recent, n)) +
                             [cand[i] for i in order[:n_select - n_first - n_recent]])
            out[t, h] = ids + [-1] * (n_select - len(ids))
    return out
