"""The operators around a layer's LoRA products from their formulas, on the CPU in 64 bits (and,
where the stored bits are defined by fp32 steps, in fp32 with each step rounded once)."""
import math

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


# ------------------------------------------------------------------ number formats

def e4m3_values():
    """The value of each of the 256 e4m3 bytes (NaN for 0x7f and 0xff)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(b >> 7, -v, v)


E4M3 = e4m3_values()


def _nearest_even(grid, x):
    """Index into an ascending grid of the nearest value to x >= 0; ties to the even index."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 0))
    return np.where(x >= grid[-1], len(grid) - 1, np.where(up, i, i - 1))


def to_e4m3(x):
    """Bytes of x >= 0 as e4m3: nearest, ties to even, saturating; NaN -> 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    return np.where(np.isnan(x), 0x7F, _nearest_even(E4M3[:0x7F], np.nan_to_num(x, posinf=1e30)))


def quantise32(x, factor):
    """Codes [..., d] (0..15) and scale bytes [..., d / 16] of float32 x, in fp32 steps."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        w = (x * (np.float32(1) / np.float32(factor))).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
        top = np.abs(w).max(-1)  # keeps a NaN
        s8 = to_e4m3(top / np.float32(6))
        s = E4M3[s8].astype(np.float32)[..., None]
        y = np.where(s > 0, w / np.where(s > 0, s, np.float32(1)), np.float32(0))
    m = _nearest_even(E2M1, np.abs(np.nan_to_num(y, posinf=1e30, neginf=-1e30)).astype(np.float64))
    code = np.where(s > 0, m + 8 * np.signbit(y), 0)
    return code.reshape(x.shape).astype(np.uint8), s8.astype(np.uint8)


def values(code, s8):
    """What codes and scale bytes stand for (without the cache's factor), in 64 bits."""
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    return (v.reshape(*s8.shape, 16) * E4M3[s8][..., None]).reshape(code.shape)


# ------------------------------------------------------------------ the cache

def sections(cache, d):
    """Views of a cache [pages][heads][blocks][18 d]: codes of K and V, scales of K and V."""
    c = cache.reshape(*cache.shape[:3], 18, d) if isinstance(cache, torch.Tensor) else cache
    flat = c.reshape(*cache.shape[:3], 18 * d)
    return (flat[..., :8 * d].reshape(*cache.shape[:3], 16, d // 2),
            flat[..., 8 * d:16 * d].reshape(*cache.shape[:3], 16, d // 2),
            flat[..., 16 * d:17 * d].reshape(*cache.shape[:3], 16, d // 16),
            flat[..., 17 * d:].reshape(*cache.shape[:3], 16, d // 16))


def unpack(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def build_cache(k, v, pages, table, page, k_scale, v_scale, garbage=255):
    """A cache holding sequences k[b], v[b] ([tokens][heads][d] float) at table's pages; what is
    not theirs holds `garbage` bytes (255: NaN scales)."""
    heads, d = k[0].shape[1:]
    cache = np.full((pages, heads, page // 16, 18 * d), garbage, dtype=np.uint8)
    for b in range(len(k)):
        n = k[b].shape[0]
        for x, factor, c0, s0 in ((k[b], k_scale, 0, 16 * d), (v[b], v_scale, 8 * d, 17 * d)):
            code, s8 = quantise32(x, factor)
            code = pack(code)
            for j in range(n):
                blk = cache[table[b][j // page], :, (j % page) // 16]
                r = j % 16
                blk[:, c0 + r * d // 2:c0 + (r + 1) * d // 2] = code[j]
                blk[:, s0 + r * d // 16:s0 + (r + 1) * d // 16] = s8[j]
    return cache


def read_cache(cache, pages, n, page, d):
    """K and V ([n][heads][d], 64 bits, without factors) of a sequence in the given pages."""
    blk = cache[np.asarray(pages, dtype=np.int64)]  # [p][heads][blocks][18 d]
    out = []
    for c, s in ((0, 2), (1, 3)):
        sec = sections(blk, d)
        val = values(unpack(sec[c]), sec[s])          # [p][heads][blocks][16][d]
        val = np.moveaxis(val, 1, 3)                  # [p][blocks][16][heads][d]
        out.append(val.reshape(blk.shape[0] * page, *val.shape[3:])[:n])
    return out


# ------------------------------------------------------------------ the operators

def norm(x, r, w, eps, groups):
    """z, n and the scales, in 64 bits."""
    z = x.astype(np.float64) + (0 if r is None else r.astype(np.float64))
    n = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    top = np.abs(n).reshape(n.shape[0], groups, n.shape[1] // groups).max(-1)
    return z, n, np.maximum(top / 448, 2.0 ** -100)


def rotate(x, cos, sin, interleaved, dtype=np.float64):
    """rot(x [n][heads][d]) by cos, sin [n][rope_dim / 2], each step in dtype."""
    x, c, s = x.astype(dtype), cos.astype(dtype)[:, None], sin.astype(dtype)[:, None]
    half = c.shape[-1]
    out = x.copy()
    if interleaved:
        ia, ib = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        ia, ib = slice(0, half), slice(half, 2 * half)
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def attention(q, k, v, scale, window):
    """One sequence: q [m][heads][d], k and v [n][kv heads][d] -> out, lse, sum p |v|, the largest
    sum |q k| of a row, in 64 bits."""
    m, heads, d = q.shape
    n, kvh = k.shape[:2]
    g = heads // kvh
    out = np.zeros((m, heads, d))
    lse = np.full((m, heads), -math.inf)
    size = np.zeros((m, heads, d))
    span = np.zeros((m, heads))
    for i in range(m):
        pos = n - m + i
        lo = max(0, pos - window + 1) if window else 0
        if pos < lo or pos < 0:
            continue
        for h in range(heads):
            kk, vv = k[lo:pos + 1, h // g], v[lo:pos + 1, h // g]
            x = kk @ q[i, h] * scale
            top = x.max()
            p = np.exp(x - top)
            out[i, h] = p @ vv / p.sum()
            size[i, h] = p @ np.abs(vv) / p.sum()
            lse[i, h] = top + math.log(p.sum())
            span[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, lse, size, span
