"""The 8-bit KV cache's append and attention from their definitions, in numpy, for the tests.

Pages are uint8 [num_pages][page_bytes], exponents int8 [num_pages], the block table
[S][max_blocks][n_kv][2].  Nothing here uses the library.
"""
import numpy as np

LIMIT = {"e4m3": 448.0, "int8": 127.0}
MIN_EXPONENT = -40


def _e4m3_table():
    b = np.arange(256)
    sign, ex, man = np.where(b > 127, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = np.where(ex > 0, (1 + man / 8.0) * 2.0 ** (ex - 7.0), man * 2.0 ** -9)
    v = sign * v
    v[[0x7F, 0xFF]] = np.nan
    return v


E4M3 = _e4m3_table()


def decode(codes, fmt):
    """Bytes -> fp64 values in units of the scale."""
    return E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def nearest(x, fmt):
    """fp64 in units of the scale -> the nearest code's value, ties to even, saturating; NaN stays (INT8: 0)."""
    with np.errstate(invalid="ignore"):
        if fmt == "int8":
            return np.clip(np.rint(np.where(np.isnan(x), 0.0, x)), -127, 127)
        y = np.clip(x, -448, 448)
        m = np.maximum(np.abs(y), 2.0 ** -6)
        ulp = 2.0 ** (np.frexp(np.where(np.isnan(m), 1.0, m))[1] - 1 - 3)
        return np.clip(np.rint(y / ulp) * ulp, -448, 448)


def half_step(v, fmt):
    """Half the distance between codes at |v| (in units of the scale)."""
    if fmt == "int8":
        return np.full(v.shape, 0.5)
    m = np.maximum(np.abs(v), 2.0 ** -6)
    return 2.0 ** (np.frexp(m)[1] - 1 - 4)


def fit_exponent(amax, fmt):
    if amax == 0:
        return MIN_EXPONENT
    m, x = np.frexp(amax / LIMIT[fmt])
    return max(MIN_EXPONENT, int(x) - (1 if m == 0.5 else 0))


def rotate(x, cos, sin, interleaved, dtype):
    """x [T][heads][d], cos and sin [T][rot / 2]; products and sums rounded to dtype one by one."""
    x, cos, sin = x.astype(dtype), cos.astype(dtype)[:, None], sin.astype(dtype)[:, None]
    h = cos.shape[-1]
    y = x.copy()
    ia, ib = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    a, b = x[..., ia], x[..., ib]
    with np.errstate(invalid="ignore"):
        y[..., ia] = a * cos - b * sin
        y[..., ib] = b * cos + a * sin
    return y


def append(pages, exps, table, indptr, kv_len, k, v, bt, fmt):
    """Writes rotated keys k and values v [T][n_kv][d] (fp32 or fp64) into the pages, in place; pages hold codes'
    VALUES here: fp64 [num_pages][bt][d]."""
    for s in range(len(kv_len)):
        n = indptr[s + 1] - indptr[s]
        p0 = kv_len[s] - n
        for blk in range(p0 // bt, -(-kv_len[s] // bt) if n else p0 // bt):
            lo, hi = max(p0, blk * bt), min(kv_len[s], (blk + 1) * bt)
            held = lo - blk * bt
            for h in range(k.shape[1]):
                for w, src in enumerate((k, v)):
                    page = table[s, blk, h, w]
                    rows = src[indptr[s] + lo - p0:indptr[s] + hi - p0, h].astype(np.float64)
                    mag = np.abs(rows[np.isfinite(rows)])
                    e = fit_exponent(mag.max() if mag.size else 0.0, fmt)
                    if held:
                        old = int(exps[page])
                        e = max(e, old)
                        pages[page, :held] = nearest(pages[page, :held] * 2.0 ** (old - e), fmt)
                    pages[page, held:held + hi - lo] = nearest(rows * 2.0 ** -float(e), fmt)
                    exps[page] = e


def attend(values, exps, table, indptr, kv_len, q, bt, scale, causal=True, window=0):
    """fp64 (out, lse, tolerance of out, tolerance of lse), from pages of code values.

    The tolerances: a weight is rounded to fp16 once (2^-11 of it), the output once (2^-11, half a
    subnormal step 2^-25 at least); scores are sums of d products in fp32 (d 2^-24 of the sum of
    magnitudes) and the exponential is good to 2^-21 of its value; sums of n weights to n 2^-24.
    """
    T, hq, d = q.shape
    n_kv = table.shape[2]
    out, lse = np.zeros((T, hq, d)), np.full((T, hq), -np.inf)
    t_out, t_lse = np.zeros((T, hq, d)), np.zeros((T, hq))
    q = q.astype(np.float64)
    for s in range(len(kv_len)):
        t0, t1, L = indptr[s], indptr[s + 1], kv_len[s]
        n, nb = t1 - t0, -(-L // bt)
        if n == 0 or L == 0:
            continue
        pos = L - n + np.arange(n)
        j = np.arange(L)
        see = np.ones((n, L), bool)
        if causal:
            see &= j[None] <= pos[:, None]
        if window:
            see &= j[None] > pos[:, None] - window
        used = see.any(0)
        for h in range(n_kv):
            kk, vv = (np.concatenate([values[table[s, b, h, w]] * 2.0 ** float(exps[table[s, b, h, w]])
                                      if used[b * bt:(b + 1) * bt].any() else np.zeros((bt, d))
                                      for b in range(nb)])[:L] for w in (0, 1))
            kk, vv = np.where(used[:, None], kk, 0.0), np.where(used[:, None], vv, 0.0)
            for g in range(h * (hq // n_kv), (h + 1) * (hq // n_kv)):
                z = np.where(see, q[t0:t1, g] @ kk.T * scale, -np.inf)
                m = z.max(1)
                m0 = np.where(np.isinf(m), 0.0, m)
                p = np.exp(z - m0[:, None])
                l = p.sum(1)
                w = p / np.where(l > 0, l, 1.0)[:, None]
                out[t0:t1, g] = w @ vv
                with np.errstate(divide="ignore"):
                    lse[t0:t1, g] = np.where(l > 0, m0 + np.log(l), -np.inf)
                ds = np.where(see, np.abs(q[t0:t1, g]) @ np.abs(kk).T, 0).max(1) * abs(scale) * (d + 8) * 2.0 ** -24
                ds = ds + 2.0 ** -21 + L * 2.0 ** -24
                mag = w @ np.abs(vv)
                t_out[t0:t1, g] = (2.0 ** -11 * 1.01 + 2 * ds[:, None]) * mag + 2.0 ** -11 * np.abs(out[t0:t1, g]) + 2.0 ** -24
                t_lse[t0:t1, g] = ds + 2.0 ** -21 * (1 + np.abs(np.where(l > 0, lse[t0:t1, g], 0)))
    return out, lse, t_out, t_lse
