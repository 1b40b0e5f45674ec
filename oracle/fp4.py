"""The block-scaled 4-bit cache and the norm + rotary pass, in plain numpy.

Written from the format's definition: 16 dims share an e4m3 scale, an element is
an e2m1 code, its value code * scale * kv_scale.  Encoding follows the definition's
fp32 steps (quotients are IEEE fp32); values, attention and norms are fp64.
"""
from __future__ import annotations

import numpy as np

# magnitudes by code, both formats rising with the code: 0 is even
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def nearest(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table value nearest to each x >= 0 (ties to the even index), saturating."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        dl, dh = x - table[lo], table[hi] - x
    take = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (x > table[-1])
    return np.where(take, hi, lo)


def encode(x: np.ndarray, kv_scale: float):
    """x [..., d] -> (codes uint8 [..., d] in 0..15, scale bytes uint8 [..., d / 16])."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 16)
    kv = np.float32(kv_scale)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(-1)                        # NaN if any is
        quot = amax / (np.float32(6) * kv)
        scale = np.where(np.isnan(quot), 0x7F, nearest(np.nan_to_num(quot, nan=0.0, posinf=1e30), E4M3))
        dec = np.where(scale == 0x7F, np.nan, E4M3[np.minimum(scale, len(E4M3) - 1)]).astype(np.float32)
        step = (dec * kv)[..., None]
        q = np.where(step > 0, g / step, np.float32(0))
        q = np.nan_to_num(q, nan=0.0, posinf=1e30, neginf=-1e30)
    code = nearest(np.abs(q), E2M1) + 8 * np.signbit(q)
    code = np.where(step > 0, code, 0)
    return code.reshape(x.shape).astype(np.uint8), scale.astype(np.uint8)


def decode_e4m3(b: np.ndarray) -> np.ndarray:
    b = np.asarray(b, np.uint8)
    v = np.where((b & 0x7F) == 0x7F, np.nan, E4M3[np.minimum(b & 0x7F, 126)])
    return np.where(b & 0x80, -v, v)


def cache_shape(nb, h, B, d):
    return (nb, h, B, d // 2 + d // 16)


def _split(cache: np.ndarray, d: int):
    nb, h, B, _ = cache.shape
    flat = cache.reshape(nb, h, -1)
    return flat[:, :, :B * d // 2].reshape(nb, h, d // 32, B, 16), \
        flat[:, :, B * d // 2:].reshape(nb, h, B, d // 16)


def values(cache: np.ndarray, d: int, kv_scale: float) -> np.ndarray:
    """fp64 values [nb, h, B, d] of a cache."""
    body, scales = _split(cache, d)
    nb, h, _, B, _ = body.shape
    code = np.stack([body & 15, body >> 4], -1).reshape(nb, h, d // 32, B, 32)
    code = code.transpose(0, 1, 3, 2, 4).reshape(nb, h, B, d)
    v = np.where(code & 8, -E2M1[code & 7], E2M1[code & 7])
    return v * np.repeat(decode_e4m3(scales), 16, -1) * np.float64(np.float32(kv_scale))


def write(x: np.ndarray, cache: np.ndarray, slots: np.ndarray, kv_scale: float) -> None:
    """x fp32-valued [T, h, d] -> the cache's bytes at slots (negative or outside: skipped)."""
    T, h, d = x.shape
    body, scales = _split(cache, d)          # views
    B = body.shape[3]
    code, sc = encode(x, kv_scale)
    for t, s in enumerate(np.asarray(slots).tolist()):
        if s < 0 or s >= cache.shape[0] * B:
            continue
        pair = code[t].reshape(h, d // 32, 16, 2)
        body[s // B, :, :, s % B] = pair[..., 0] | (pair[..., 1] << 4)
        scales[s // B, :, s % B] = sc[t]


def attention(q, k_rows, v_rows, scale):
    """q [Hq, d], k_rows / v_rows [h, n, d] in fp64 -> [Hq, d]; n = 0 gives zeros."""
    hq, d = q.shape
    h, n, _ = k_rows.shape
    if n == 0:
        return np.zeros((hq, d))
    z = np.einsum("hgd,hnd->hgn", q.reshape(h, hq // h, d), k_rows) * scale
    p = np.exp(z - z.max(-1, keepdims=True))
    return (np.einsum("hgn,hnd->hgd", p, v_rows) / p.sum(-1, keepdims=True)).reshape(hq, d)


def norm_rope(x, weight, cos_sin, positions, eps, interleaved):
    """x fp64 [T, heads, d]; weight [d] or None; the rotated rows in fp64."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = cos_sin.shape[1] // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    cs = np.asarray(cos_sin, np.float64)[positions][:, None]
    c, s = cs[..., :half], cs[..., half:]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y
