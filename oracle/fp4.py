"""Plain fp64 forms of the 4-bit cache, the read-back and the head norm with
rotation (numpy; shares nothing with the CUDA path)."""
from __future__ import annotations

import numpy as np

from . import bf16_to_f64, e4m3_from_f32, e4m3_to_f64, f16_to_f64

PAGE = 64
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(x, head):
    """x float [..., D] and head scales broadcast over [..., 1] -> (codes uint8
    [..., D], scale bytes uint8 [..., D/16]).  Quotients are fp32 ones."""
    x = np.asarray(x, np.float32)
    head = np.broadcast_to(np.asarray(head, np.float32), x.shape[:-1] + (1,))
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    with np.errstate(all="ignore"):
        amax = np.abs(blocks).max(-1)  # NaN if any is NaN
        want = (amax / (head * np.float32(6))).astype(np.float32)
        nan = np.isnan(want)
        byte = np.where(nan, 0x7F, e4m3_from_f32(np.where(nan, 0, np.minimum(want, np.float32(448)))))
        step = (e4m3_to_f64(byte.astype(np.uint8)).astype(np.float32) * head).astype(np.float32)[..., None]
        quotient = (np.abs(blocks) / step).astype(np.float32).astype(np.float64)
    usable = (byte != 0)[..., None] & ~nan[..., None] & (step > 0)
    quotient = np.where(usable, quotient, 0.0)
    code = np.zeros(quotient.shape, np.int64)
    for i in range(1, 8):  # past the middle between two values, or on it where the upper code is even
        mid = (GRID[i - 1] + GRID[i]) / 2
        code = np.where((quotient > mid) | ((quotient == mid) & (i % 2 == 0)), i, code)
    code = np.where(usable, code + 8 * np.signbit(blocks), 0)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def rows_of_slab(pool, head_dim):
    """uint8 pool [P, Hk, slab] -> views (code bytes [P, Hk, 64, D/2], scale bytes [P, Hk, 64, D/16])."""
    n = PAGE * head_dim // 2
    p, hk, _ = pool.shape
    return (pool[:, :, :n].reshape(p, hk, PAGE, head_dim // 2), pool[:, :, n:].reshape(p, hk, PAGE, head_dim // 16))


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def decode_pool(pool, head, head_dim):
    """uint8 pool [P, Hk, slab], head scales [Hk] -> (code * block scale, head scale) as float64 values [P, Hk, 64, D]."""
    codes, scales = rows_of_slab(pool, head_dim)
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], head_dim).astype(np.int64)
    v = np.where(n >= 8, -1.0, 1.0) * GRID[n & 7]
    s = np.repeat(e4m3_to_f64(np.ascontiguousarray(scales)), 16, axis=-1)
    return v * s * np.asarray(head, np.float64)[None, :, None, None]


def make_pool(x, head):
    """Rows x float [P, Hk, 64, D] -> a uint8 pool [P, Hk, slab]."""
    codes, scales = encode(x, np.asarray(head, np.float32)[None, :, None, None])
    p, hk = x.shape[:2]
    return np.concatenate([pack(codes).reshape(p, hk, -1), scales.reshape(p, hk, -1)], -1)


def append(k_new_bits, cu, start, block_table, pool, head, head_dim):
    """bf16 bits [T, Hk, D] written into a copy of a 4-bit pool."""
    out = pool.copy()
    codes, scales = rows_of_slab(out, head_dim)
    x = bf16_to_f64(k_new_bits).astype(np.float32)
    c, s = encode(x, np.asarray(head, np.float32)[None, :, None])
    c = pack(c)
    for b in range(len(start)):
        for i in range(int(cu[b]), int(cu[b + 1])):
            p = int(start[b]) + i - int(cu[b])
            page = int(block_table[b, p // PAGE])
            codes[page, :, p % PAGE] = c[i]
            scales[page, :, p % PAGE] = s[i]
    return out


def attend(q_bits, k, v, block_table, seq_lens, scale):
    """q bf16 bits [B, Hq, D], k and v float64 values [P, Hk, 64, D].  Returns
    (out, lse, spread, reach, top): spread = sum_j p_j |v_j|, reach = the
    largest scale * sum |q k| of a row, top = the largest |v| of a row."""
    q = bf16_to_f64(q_bits)
    nb, hq, d = q.shape
    hk = k.shape[1]
    out, spread, top = np.zeros((nb, hq, d)), np.zeros((nb, hq, d)), np.zeros((nb, hq, d))
    lse, reach = np.full((nb, hq), -np.inf), np.zeros((nb, hq))
    for b in range(nb):
        n = int(seq_lens[b])
        if n == 0:
            continue
        pages = block_table[b, : (n + PAGE - 1) // PAGE]
        for h in range(hq):
            g = h // (hq // hk)
            kk, vv = k[pages, g].reshape(-1, d)[:n], v[pages, g].reshape(-1, d)[:n]
            s = scale * (kk @ q[b, h])
            lse[b, h] = s.max() + np.log(np.exp(s - s.max()).sum())
            p = np.exp(s - lse[b, h])
            out[b, h], spread[b, h], top[b, h] = p @ vv, p @ np.abs(vv), np.abs(vv).max(0)
            reach[b, h] = abs(scale) * (np.abs(kk) @ np.abs(q[b, h])).max()
    return out, lse, spread, reach, top


def to_f64(bits, dtype):
    return f16_to_f64(bits) if dtype == "f16" else bf16_to_f64(bits)


def norm_rope(x, weight, positions, cos_sin, rope_dim, interleaved, sections, eps, norm=True):
    """x float64 [T, H, D] -> (y float64, size): size bounds the terms each output is a sum of."""
    y = np.array(x, np.float64)
    d = y.shape[-1]
    if norm:
        y = y / np.sqrt((y * y).sum(-1, keepdims=True) / d + eps)
        if weight is not None:
            y = y * weight
    out, size = y.copy(), np.abs(y)
    axis = np.repeat(np.arange(len(sections)), sections)
    for pair in range(rope_dim // 2):
        i, j = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + rope_dim // 2)
        row = cos_sin[positions[axis[pair]]].astype(np.float64)
        c, s = row[:, None, pair], row[:, None, rope_dim // 2 + pair]
        out[..., i], out[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
        size[..., i] = size[..., j] = np.abs(y[..., i]) + np.abs(y[..., j])
    return out, size
