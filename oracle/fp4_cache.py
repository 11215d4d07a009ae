"""The 4-bit key/value cache, restated from its definition.

A section (one head of one page of 64 tokens) holds 64 rows of dim / 2 key code
bytes, 64 rows of value code bytes, then 64 rows of scale bytes: the key's
dim / 16 padded to R = 4 ceil(dim / 64), and the value's likewise.  A block of 16
columns x gets s = E4M3(max |x| / (6 g)) and codes E2M1(x / (s g)), the products
and quotients in FP32; a code c reads as (c s) g.

Caches are numpy arrays uint8 [pages, heads, section].
"""

from __future__ import annotations

import numpy as np

from .codecs import E2M1_TABLE, e2m1_encode, e4m3_decode, e4m3_encode, pack_e2m1, unpack_e2m1

PAGE = 64
F32 = np.float32


def scale_row(dim):
    return 4 * -(-dim // 64)


def section_bytes(dim):
    return PAGE * (dim + 2 * scale_row(dim))


def views(cache, dim):
    """Key codes, value codes [pages, 64, heads, dim / 2], key scales, value scales [pages, 64, heads, dim / 16]:
    views of the cache."""
    w, r, n = dim // 2, scale_row(dim), dim // 16
    shape = cache.shape[:2]
    k = cache[..., :PAGE * w].reshape(shape + (PAGE, w))
    v = cache[..., PAGE * w: 2 * PAGE * w].reshape(shape + (PAGE, w))
    s = cache[..., 2 * PAGE * w:].reshape(shape + (PAGE, 2 * r))
    return [np.moveaxis(x, 1, 2) for x in (k, v, s[..., :n], s[..., r: r + n])]


def values(codes, scales, g):
    """(c s) g in 64 bits (c s is exact)."""
    c = E2M1_TABLE[unpack_e2m1(codes)]
    return c * np.repeat(e4m3_decode(scales), 16, axis=-1) * float(F32(g))


def decode(cache, dim, k_scale=1.0, v_scale=1.0):
    """Keys and values [pages, 64, heads, dim] in 64 bits."""
    kc, vc, ks, vs = views(cache, dim)
    return values(kc, ks, k_scale), values(vc, vs, v_scale)


def quantise(x, g):
    """Codes [..., dim / 2] and scales [..., dim / 16] of FP32 rows."""
    x = np.asarray(x, dtype=F32)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    g = F32(g)
    with np.errstate(all="ignore"):
        amax = np.abs(b).max(axis=-1)
        nan = np.isnan(b).any(axis=-1)
        ratio = np.minimum(amax / (F32(6) * g), F32(448))
        s = e4m3_encode(np.where(nan, 0, ratio))
        d = (e4m3_decode(s).astype(F32) * g)[..., None]
        y = np.where(d > 0, np.clip(b / np.where(d > 0, d, F32(1)), -8, 8), np.copysign(F32(0), b))
    s = np.where(nan, np.uint8(0x7F), s)
    y = np.where(nan[..., None], F32(6), np.where(np.isnan(y), 0, y))   # a NaN becomes the largest code
    codes = e2m1_encode(y).reshape(x.shape)
    return pack_e2m1(codes), s


def rotate(x, cos, sin, interleaved):
    """x [n, heads, dim] FP32 with its first columns turned by angles [n, rot / 2]: products and sums in FP32."""
    x = np.array(x, dtype=F32)
    half = cos.shape[1]
    c, s = (np.asarray(t, dtype=F32)[:, None, :] for t in (cos, sin))
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, w = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    x[..., a], x[..., b] = u, w
    return x


def append(k, v, slots, cache, dim, positions=None, cos_sin=None, interleaved=False, k_scale=1.0, v_scale=1.0):
    """Keys and values [n, heads, dim] into the cache, in place (slots outside the pool are skipped)."""
    if cos_sin is not None and cos_sin.shape[1]:
        p = np.clip(np.asarray(positions), 0, len(cos_sin) - 1)
        half = cos_sin.shape[1] // 2
        k = rotate(k, cos_sin[p, :half], cos_sin[p, half:], interleaved)
    new = quantise(k, k_scale) + quantise(v, v_scale)
    to = views(cache, dim)
    slots = np.asarray(slots)
    at = np.nonzero((slots >= 0) & (slots < cache.shape[0] * PAGE))[0]
    page, off = slots[at] // PAGE, slots[at] % PAGE
    for view, x in zip(to, (new[0], new[2], new[1], new[3])):
        view[page, off] = x[at]
