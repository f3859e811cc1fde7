"""Plain numpy oracle of the row operators: norm and rotation of query and key
heads, quantising rows into a cache with fixed scales, reading them back.

TEST INFRASTRUCTURE ONLY: imported by ``tests/``; the product library never
calls it.  Everything is float64 except where the definition names an fp32
rounding (the reciprocal of a scale, its product, the read-back product).
"""
import numpy as np


def norm_rope(x, w=None, eps=1e-6, table=None, positions=None, interleaved=False):
    """(y, m): float64 x [B, H, L, d] normed by w [d] (None: not) and turned by
    table [P, rot/2, 2] at positions [B, L] (None: not); m bounds the magnitudes that were added for each element.
    Rows of negative position are left as x."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    m = np.abs(y)
    if table is None:
        return y, m
    half = table.shape[1]
    out, mag = y.copy(), m.copy()
    for f in range(half):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        for b in range(x.shape[0]):
            p = np.maximum(positions[b], 0)
            c, s = table[p, f, 0].astype(np.float64), table[p, f, 1].astype(np.float64)
            out[b, :, :, i] = y[b, :, :, i] * c - y[b, :, :, j] * s
            out[b, :, :, j] = y[b, :, :, i] * s + y[b, :, :, j] * c
            mag[b, :, :, i] = mag[b, :, :, j] = m[b, :, :, i] + m[b, :, :, j]
    pad = np.asarray(positions) < 0
    out = np.where(pad[:, None, :, None], x, out)
    return out, mag


def codes(x, scale, zero=None, bits=8):
    """Integer codes of float32 x [B, H, L, d]; scale (and zero) [H] or [1]."""
    x = np.asarray(x, np.float32)
    H = x.shape[1]
    s = np.broadcast_to(np.asarray(scale, np.float32), (H,))[None, :, None, None]
    with np.errstate(all="ignore"):
        inv = np.minimum(np.float32(1.0) / s, np.finfo(np.float32).max)
        n = np.rint(x * inv)
    n = np.where(np.isnan(n), 0.0, np.clip(n.astype(np.float64), -1e6, 1e6)).astype(np.int64)
    if zero is None:
        top = 2 ** (bits - 1) - 1
        return np.clip(n, -top, top)
    z = np.broadcast_to(np.asarray(zero, np.int64), (H,))[None, :, None, None]
    return np.clip(n + z, 0, 2 ** bits - 1)


def pack(c, bits, unsigned):
    """Codes [..., d] as the cache stores them."""
    if bits == 8:
        return c.astype(np.uint8 if unsigned else np.int8)
    u = (c & 15).astype(np.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def unpack(p, bits, unsigned):
    if bits == 8:
        return p.astype(np.int64)
    c = np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], -1).astype(np.int64)
    return c if unsigned else np.where(c >= 8, c - 16, c)


def write(cache, x, scale, zero, bits, start, lengths):
    """Writes the codes of x into a copy of cache [B, H, Lmax, ...]."""
    cache = cache.copy()
    c = pack(codes(x, scale, zero, bits), bits, zero is not None)
    for b in range(x.shape[0]):
        for t in range(x.shape[2]):
            r = int(start[b]) + t
            if t < lengths[b] and 0 <= r < cache.shape[2]:
                cache[b, :, r] = c[b, :, t]
    return cache


def values(cache, scale, zero, bits, start, L):
    """float32 values of cache rows start[b] + t, t < L (all inside the cache)."""
    c = unpack(cache, bits, zero is not None)
    H = cache.shape[1]
    s = np.broadcast_to(np.asarray(scale, np.float32), (H,))[:, None, None]
    z = np.broadcast_to(np.asarray(0 if zero is None else zero, np.int64), (H,))[:, None, None]
    return np.stack([s * (c[b, :, int(start[b]):int(start[b]) + L] - z).astype(np.float32)
                     for b in range(cache.shape[0])])
