"""The attention operators in 64 bits (numpy), from their definitions in
include/r9q.h, and the packed 4-bit cache read byte by byte."""
import numpy as np


def to_bf16(x):
    """fp32 -> the nearest bf16 (ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, np.float32(np.nan))


def rotate(y, cos, sin, interleaved):
    """y [T][H][D]; cos, sin [T][rot/2]."""
    half = cos.shape[-1]
    out = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, None, i], sin[:, None, i]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def norm_rope(x, w, cos, sin, eps, interleaved):
    x = x.astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    return y if cos is None else rotate(y, cos.astype(np.float64), sin.astype(np.float64), interleaved)


def norm_rope_grad(dy, x, w, cos, sin, eps, interleaved):
    """(dx, dw, sum |terms of dw|), the two products of a rotated element's gradient counted apart."""
    x, w, g = x.astype(np.float64), w.astype(np.float64), dy.astype(np.float64)
    terms = np.abs(g)
    if cos is not None:
        cos, sin = cos.astype(np.float64), sin.astype(np.float64)
        own = rotate(g, cos, 0 * sin, interleaved)
        g = rotate(g, cos, -sin, interleaved)
        terms = np.abs(own) + np.abs(g - own)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    return r * (w * g - xh * (w * g * xh).mean(-1, keepdims=True)), (g * xh).sum((0, 1)), (terms * np.abs(xh)).sum((0, 1))


def quantise32(x):
    """(codes, step, lowest) of the last dimension, each step in fp32."""
    x = np.ascontiguousarray(x, np.float32)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        low, step = to_bf16(lo), to_bf16((hi - lo) * np.float32(1 / 15))
        q = np.where(step > 0, (x - low) / np.where(step > 0, step, np.float32(1)), np.float32(0))
        codes = np.clip(np.rint(q), 0, 15)
    return np.where(np.isfinite(codes), codes, 0).astype(np.int64), step, low


def cache_codes(k, v, page, dim):
    """Packed bytes [pages][H][page][D/2] -> (K codes, V codes) [pages][H][page][D]."""
    pages, heads = k.shape[:2]
    kc = np.zeros((pages, heads, page, dim), np.int64)
    kc[..., 0::2], kc[..., 1::2] = k & 15, k >> 4
    vb = v.reshape(pages, heads, page // 16, dim // 64, 8, 4, 4, 4)
    vc = np.zeros((pages, heads, page // 16, 16, dim), np.int64)
    for t in range(16):
        j, b = (t % 8) // 2, 2 * (t % 2) + t // 8
        for d in range(dim):
            c, m, n, r = d // 64, d % 64 // 16, d % 16 // 8, d % 8
            vc[:, :, :, t, d] = (vb[:, :, :, c, r, j, m, b] >> (4 * n)) & 15
    return kc, vc.reshape(pages, heads, page, dim)


def attention(q, k, v, spread, scale, window):
    """One sequence: q [Lq][Hq][D], k, v [len][Hk][D], spread [len][Hk] the range of v's codes.  Returns o, lse, and
    for each the bounds' parts: sum p spread, sum p |v| and the largest sum |q k| scale."""
    n, heads, dim = q.shape
    length, kv = k.shape[:2]
    o, lse = np.zeros((n, heads, dim)), np.full((n, heads), -np.inf)
    wide, mass, top = np.zeros((n, heads)), np.zeros((n, heads, dim)), np.zeros((n, heads))
    for i in range(n):
        p = length - n + i
        first = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(heads):
            kk, vv = k[first:p + 1, h // (heads // kv)], v[first:p + 1, h // (heads // kv)]
            s = kk @ q[i, h] * scale
            m = s.max()
            e = np.exp(s - m)
            w = e / e.sum()
            lse[i, h] = m + np.log(e.sum())
            o[i, h] = w @ vv
            wide[i, h] = w @ spread[first:p + 1, h // (heads // kv)]
            mass[i, h] = w @ np.abs(vv)
            top[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return o, lse, wide, mass, top
