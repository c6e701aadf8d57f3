"""Float64 (and, where the operators fix their roundings, float32) definitions of the serving operators.

Rotary append, the 4-bit pool format, and causal attention with a sliding window and sinks, written from their
formulas with one plain loop per query row.
"""

from __future__ import annotations

import numpy as np

BS = 16


def rotate(x, positions, cos_sin, interleaved: bool, dtype=np.float64):
    """x [T, H, D] with its first rot_dim channels turned by the tokens' positions, in ``dtype`` arithmetic."""
    x = np.asarray(x, dtype=dtype).copy()
    r = cos_sin.shape[1]
    rows = np.asarray(cos_sin, dtype=dtype)[np.asarray(positions)]
    c, s = rows[:, None, : r // 2], rows[:, None, r // 2:]
    if interleaved:
        a, b = x[..., 0:r:2].copy(), x[..., 1:r:2].copy()
        x[..., 0:r:2], x[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., : r // 2].copy(), x[..., r // 2:r].copy()
        x[..., : r // 2], x[..., r // 2:r] = a * c - b * s, b * c + a * s
    return x


def q4_quantise(x):
    """x [..., D] float32 -> (codes uint8 [..., D], step fp16, low fp16 [..., D/32]) with the format's roundings."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(g).all(-1)
    g = np.clip(np.where(bad[..., None], np.float32(0), g), np.float32(-32768), np.float32(32768))
    lo, hi = g.min(-1), g.max(-1)
    low = lo.astype(np.float16)
    step = ((hi - lo) * np.float32(1.0 / 15.0)).astype(np.float16)
    s32 = step.astype(np.float32)
    inv = np.where(s32 == 0, np.float32(0), np.float32(1) / np.where(s32 == 0, np.float32(1), s32)).astype(np.float32)
    n = np.clip(np.rint((g - low.astype(np.float32)[..., None]) * inv[..., None]), 0, 15).astype(np.uint8)
    step, low = np.where(bad, np.float16(np.nan), step), np.where(bad, np.float16(np.nan), low)
    return n.reshape(x.shape), step, low


def q4_values(codes, step, low):
    """The fp16 numbers the codes stand for, as float64."""
    n = np.asarray(codes, dtype=np.float64)
    n = n.reshape(*n.shape[:-1], -1, 32)
    v = n * step.astype(np.float64)[..., None] + low.astype(np.float64)[..., None]
    return v.astype(np.float16).astype(np.float64).reshape(codes.shape)


def q4_store(pool, slots, x):
    """Quantise x [T, H, D] into the records of a uint8 pool [blocks, H, 10 * D]; negative slots are skipped."""
    d = x.shape[-1]
    codes, step, low = q4_quantise(x)
    for t, s in enumerate(slots):
        if s < 0:
            continue
        rec, at = pool[s // BS], s % BS
        rec[:, at * d // 2:(at + 1) * d // 2] = codes[t, :, 0::2] | (codes[t, :, 1::2] << 4)
        pairs = np.stack([step[t], low[t]], -1).astype(np.float16).view(np.uint8).reshape(x.shape[1], -1)
        rec[:, BS * d // 2 + at * d // 8:BS * d // 2 + (at + 1) * d // 8] = pairs


def q4_load(pool):
    """Every value of a pool [blocks, H, 10 * D] as float64 [blocks * 16, H, D]."""
    n, h, size = pool.shape
    d = size // 10
    byte = pool[:, :, : BS * d // 2].reshape(n, h, BS, d // 2)
    codes = np.stack([byte & 15, byte >> 4], -1).reshape(n, h, BS, d)
    pairs = np.ascontiguousarray(pool[:, :, BS * d // 2:]).view(np.float16).reshape(n, h, BS, d // 32, 2)
    return q4_values(codes, pairs[..., 0], pairs[..., 1]).transpose(0, 2, 1, 3).reshape(n * BS, h, d)


def visible(p: int, length: int, window: int, sinks: int):
    """Keys that the query at position p sees, in order."""
    return [j for j in range(min(p + 1, length)) if window == 0 or j < sinks or p - j < window]


def window_attention(q, k_pool, v_pool, block_table, query_start_loc, seq_lens, scale, window, sinks):
    """(out, spread, reach): out [Tq, Hq, D] float64; spread = sum of p |v| and reach = max over the row's keys of
    scale * sum |q k|, the two magnitudes that roundings of the probabilities and of the scores scale with."""
    q = np.asarray(q, dtype=np.float64)
    hkv, g = k_pool.shape[1], q.shape[1] // k_pool.shape[1]
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    reach = np.zeros(q.shape[:2])
    for b in range(len(seq_lens)):
        q0, sq, length = int(query_start_loc[b]), int(query_start_loc[b + 1] - query_start_loc[b]), int(seq_lens[b])
        for i in range(sq):
            keys = np.asarray(visible(length - sq + i, length, window, sinks), dtype=np.int64)
            if keys.size == 0:
                continue
            rows = block_table[b][keys // BS].astype(np.int64) * BS + keys % BS
            k, v = k_pool[rows].astype(np.float64), v_pool[rows].astype(np.float64)
            for h in range(q.shape[1]):
                x = q[q0 + i, h]
                s = scale * (k[:, h // g] @ x)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[q0 + i, h] = p @ v[:, h // g]
                spread[q0 + i, h] = p @ np.abs(v[:, h // g])
                reach[q0 + i, h] = abs(scale) * (np.abs(k[:, h // g]) @ np.abs(x)).max()
    return out, spread, reach
