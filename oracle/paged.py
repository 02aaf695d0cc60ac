"""fp64 CPU oracle of what stands around the attention: the norm and rotation of queries and keys with its gradient, the
4-bit rows of a paged key/value cache, and decode over such a cache.  Plain NumPy, float64, from the definitions; it
shares no code with the CUDA package."""

from __future__ import annotations

import math

import numpy as np

from .attention import _f64

__all__ = ["rope_table", "qk_norm_rope", "qk_norm_rope_backward", "four_bit_rows", "four_bit_pack", "four_bit_unpack",
           "page_slots", "cache_rows", "decode_paged"]


def rope_table(rows: int, rot_dim: int, base: float):
    """cos and sin [rows, rot_dim/2] of p·base^(−2i/rot_dim)."""
    i = np.arange(rot_dim // 2, dtype=np.float64)
    ang = np.arange(rows, dtype=np.float64)[:, None] * np.power(base, -2.0 * i / rot_dim)
    return np.cos(ang), np.sin(ang)


def _angles(cos, sin, positions, sections):
    """[T, rot/2] cos and sin: pair i by the position of the axis whose section holds i."""
    cos, sin, pos = _f64(cos), _f64(sin), np.atleast_2d(np.asarray(positions))
    n = cos.shape[1]
    axis = np.zeros(n, int) if sections is None else np.repeat(np.arange(len(sections)), sections)
    at = pos[axis].T  # [T, n]
    return cos[at, np.arange(n)], sin[at, np.arange(n)]


def _turn(x, c, s, rot, interleaved):
    """Rotation of the first rot features of x [T, H, d] by the angles of c, s [T, rot/2]."""
    a = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    b = a + 1 if interleaved else a + rot // 2
    y = x.copy()
    c, s = c[:, None], s[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def qk_norm_rope(x, w, cos, sin, positions, eps=1e-6, interleaved=False, sections=None):
    """x [T, H, d] → each head divided by √(mean x² + eps) and times w (w None: as it is), then rotated."""
    x = _f64(x)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * _f64(w)
    c, s = _angles(cos, sin, positions, sections)
    return _turn(x, c, s, 2 * c.shape[1], interleaved)


def qk_norm_rope_backward(dy, x, w, cos, sin, positions, eps=1e-6, interleaved=False, sections=None):
    """(dx, dw) of ⟨qk_norm_rope(x), dy⟩; dw None without norm."""
    c, s = _angles(cos, sin, positions, sections)
    g = _turn(_f64(dy), c, -s, 2 * c.shape[1], interleaved)
    if w is None:
        return g, None
    x, w = _f64(x), _f64(w)
    d = x.shape[-1]
    ms = (x * x).mean(-1, keepdims=True) + eps
    gw = g * w
    dx = gw / np.sqrt(ms) - x * (gw * x).sum(-1, keepdims=True) / (d * ms ** 1.5)
    return dx, (g * x / np.sqrt(ms)).sum((0, 1))


def four_bit_rows(x):
    """Rows x [..., d] (16-bit values) in 4 bits: numbers [..., d], scales and minima [..., d/32] (fp16 values, as float64).
    The real-number rule: min in fp16, scale = (largest − least)/15 in fp16, number = (x − min)/scale to nearest even."""
    x = _f64(x)
    v = x.reshape(*x.shape[:-1], -1, 32)
    lo, hi = v.min(-1), v.max(-1)
    mn = np.clip(lo, -65504, 65504).astype(np.float16).astype(np.float64)
    # (largest − least)/15 goes through fp32 as the division does there
    sc = np.minimum((hi - lo).astype(np.float32) / np.float32(15), np.float32(65504)).astype(np.float16).astype(np.float64)
    q = (v - mn[..., None]).astype(np.float32) / np.where(sc > 0, sc, 1.0).astype(np.float32)[..., None]
    n = np.where(sc[..., None] > 0, np.clip(np.rint(q), 0, 15), 0)
    return n.reshape(x.shape).astype(np.uint8), sc, mn


def _nibble_of(d: int, value: bool):
    """Nibble index in a row of d/2 bytes of each feature: keys 32w + 8t + n → 8(tW + w) + n, values 32w + 4g + n →
    4(gW + w) + n."""
    f, words = np.arange(d), d // 32
    w, r = f // 32, f % 32
    return ((r // 4) * words + w) * 4 + r % 4 if value else ((r // 8) * words + w) * 8 + r % 8


def four_bit_pack(n, sc, mn, value: bool):
    """Blocks [..., page, d] of numbers with their scales and minima → uint8 [..., page·5d/8] as the cache holds them."""
    page, d = n.shape[-2:]
    nib = np.zeros(n.shape, np.uint8)
    nib[..., _nibble_of(d, value)] = n
    rows = (nib[..., 0::2] | (nib[..., 1::2] << 4)).reshape(*n.shape[:-2], page * d // 2)
    pairs = np.stack([sc, mn], -1).astype(np.float16).reshape(*n.shape[:-2], page * d // 16)
    return np.concatenate([rows, pairs.view(np.uint8)], -1)


def four_bit_unpack(blocks, page: int, d: int, value: bool):
    """(numbers, scales, minima) of uint8 blocks [..., page·5d/8]."""
    blocks = np.ascontiguousarray(blocks)
    rows = blocks[..., : page * d // 2].reshape(*blocks.shape[:-1], page, d // 2)
    nib = np.stack([rows & 15, rows >> 4], -1).reshape(*rows.shape[:-1], d)
    pairs = np.ascontiguousarray(blocks[..., page * d // 2:]).view(np.float16).astype(np.float64)
    pairs = pairs.reshape(*blocks.shape[:-1], page, d // 32, 2)
    return nib[..., _nibble_of(d, value)], pairs[..., 0], pairs[..., 1]


def page_slots(table, b: int, positions, page: int):
    """(page, slot) of positions of sequence b."""
    positions = np.asarray(positions)
    return np.asarray(table)[b, positions // page], positions % page


def cache_rows(cache, table, b: int, positions, d: int, value: bool):
    """float64 rows [n, Hk, d] of sequence b at `positions`: 16-bit caches as they are ([pages, Hk, page, d], any float
    array), 4-bit ones (uint8) as number·scale + min, with the parts (numbers·scale, min) beside them."""
    if str(cache.dtype).endswith("uint8"):
        c = np.asarray(cache)
        pages, hk, page, _ = c.shape
        p, s = page_slots(table, b, positions, page)
        n, sc, mn = four_bit_unpack(c.reshape(pages, hk, -1), page, d, value)
        n, sc, mn = n[p, :, s].astype(np.float64), np.repeat(sc[p, :, s], 32, -1), np.repeat(mn[p, :, s], 32, -1)
        return n * sc + mn, n * sc, mn, sc
    c = _f64(cache)
    p, s = page_slots(table, b, positions, c.shape[2])
    x = c[p, :, s]
    return x, x, np.zeros_like(x), np.zeros_like(x)


def decode_paged(q, k_rows, v_rows, scale: float):
    """o [Nq, H, d] and lse [Nq, H] of one sequence: q [Nq, H, d] its last tokens, k_rows, v_rows [L, Hk, d]; query i sees
    keys 0 .. L − Nq + i, query head h key head h // (H / Hk); no key: o = 0, lse = −inf."""
    q, k, v = _f64(q), _f64(k_rows), _f64(v_rows)
    nq, H, d = q.shape
    L, hk = k.shape[:2]
    o, lse = np.zeros((nq, H, d)), np.full((nq, H), -math.inf)
    for i in range(nq):
        m = L - nq + i + 1
        if m <= 0:
            continue
        for h in range(H):
            s = (k[:m, h // (H // hk)] @ q[i, h]) * scale
            top = s.max()
            p = np.exp(s - top)
            lse[i, h] = top + math.log(p.sum())
            o[i, h] = (p / p.sum()) @ v[:m, h // (H // hk)]
    return o, lse
