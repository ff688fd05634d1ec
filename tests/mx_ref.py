"""Plain float64 / numpy forms of the MXFP4 operators, from the format's definition: E2M1 codes with
magnitudes {0, .5, 1, 1.5, 2, 3, 4, 6}, one E8M0 byte b per 32 elements, value = e2m1 * 2^(b - 127)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(v):
    """float64 [R, C] -> (codes [R, C/2] uint8, scale bytes [R, C/32] uint8)."""
    r, c = v.shape
    blk = v.reshape(r, c // 32, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(blk).max(axis=2)
    bad = ~np.isfinite(blk).all(axis=2)
    ex = np.frexp(np.where(bad | (amax == 0), 1.0, amax))[1] - 1  # floor(log2 amax)
    b = np.where(amax == 0, 0, np.clip(ex - 2 + 127, 0, 254))
    y = np.where(bad[..., None], 0.0, blk) / np.ldexp(1.0, b - 127)[..., None]
    dist = np.abs(np.abs(y)[..., None] - E2M1)
    # nearest magnitude; of two equally near, the even code (np.argmin keeps the first, so even codes go first)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[np.argmin(dist[..., order], axis=-1)]
    code = np.where(np.abs(y) >= 6, 7, code)
    code = code | (np.signbit(np.where(bad[..., None], 0.0, blk)).astype(np.int64) << 3)
    code = code.reshape(r, c).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, b).astype(np.uint8)


def dequantize(codes, scales):
    """-> float64 [R, C]; NaN where the scale byte is 255."""
    nib = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], -1)
    v = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)


def fp32_sum_bound(absprod, k):
    """Bound on the error of an fp32 sum of k products whose magnitudes add up to absprod: every partial
    sum is at most absprod and is rounded at most once per eight products, plus the joins."""
    return (k / 8 + 16) * 2.0 ** -24 * absprod


def half_step(t, ref):
    """Largest rounding to the output type ('f32' or 'bf16')."""
    return np.abs(ref) * (2.0 ** -24 if t == "f32" else 2.0 ** -8) + (1e-38 if t == "f32" else 1e-38)


def route(logits, top_k, renorm):
    """ids [T, k] (-1 where fewer), weights [T, k]; a row with NaN or +inf: no ids, zero weights."""
    t, e = logits.shape
    ids = np.full((t, top_k), -1, np.int64)
    wts = np.zeros((t, top_k))
    for i in range(t):
        row = logits[i]
        if np.isnan(row).any() or (row == np.inf).any() or (row == -np.inf).all():
            continue
        order = [j for j in np.argsort(-row, kind="stable") if row[j] > -np.inf][:top_k]
        ids[i, :len(order)] = order
        ex = np.exp(row - row.max())
        wts[i, :len(order)] = ex[order] / (ex[order].sum() if renorm else ex.sum())
    return ids, wts


def moe(x, logits, wgu, wdn, experts, top_k, renorm):
    """(y, bound on the error of y before its rounding, ids, weights); wgu [E * 2I, H], wdn [E * H, I]."""
    t, h = x.shape
    inter = wdn.shape[1]
    ids, wts = route(logits, top_k, renorm)
    y, err, mag = np.zeros((t, h)), np.zeros((t, h)), np.zeros((t, h))
    bad = np.isnan(logits).any(axis=1) | (logits == np.inf).any(axis=1)
    for i in range(t):
        for r in range(top_k):
            e = ids[i, r]
            if e < 0:
                continue
            g_w, u_w = wgu[e * 2 * inter:e * 2 * inter + inter], wgu[e * 2 * inter + inter:(e + 1) * 2 * inter]
            g, u = g_w @ x[i], u_w @ x[i]
            dg = fp32_sum_bound(np.abs(g_w) @ np.abs(x[i]), h)
            du = fp32_sum_bound(np.abs(u_w) @ np.abs(x[i]), h)
            s = g / (1 + np.exp(-g))
            a = s * u
            # |silu'| < 1.1; 2^-16 covers the two bf16 planes (2^-17), exp and the divisions
            da = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -16 * np.abs(a)
            d_w = wdn[e * h:(e + 1) * h]
            y[i] += wts[i, r] * (d_w @ a)
            err[i] += wts[i, r] * (np.abs(d_w) @ da)
            mag[i] += wts[i, r] * (np.abs(d_w) @ np.abs(a))
    err += fp32_sum_bound(mag, inter * top_k)
    y[bad] = np.nan
    return y, err, ids, wts
