"""Inputs and tolerances shared by the tests of the serving operators."""

import numpy as np
import torch

from oracle import serving as sv

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def table_of(seed, lens, W, spare=3):
    """A scattered block table [B, W] over one pool; entries past a row's keys are out of the pool."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // 16) for n in lens]
    blocks = sum(need) + spare
    perm = torch.randperm(blocks, generator=g).numpy().astype(np.int32)
    table = np.full((len(lens), max(W, 1)), 10 ** 6, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, blocks


def seen_blocks(rows, b, window, sinks):
    """Logical blocks that some query of row b = (Sq, L) sees."""
    sq, length = rows[b]
    got = set()
    for i in range(sq):
        got |= {j // 16 for j in sv.visible(length - sq + i, length, window, sinks)}
    return got


def random_q4_pool(blocks, hkv, d, seed):
    """A pool of quantised normal values."""
    rng = np.random.default_rng(seed)
    pool = np.zeros((blocks, hkv, 10 * d), dtype=np.uint8)
    sv.q4_store(pool, np.arange(blocks * 16), rng.standard_normal((blocks * 16, hkv, d)).astype(np.float32))
    return pool


def tolerance(want, spread, reach, n_keys, d, dtype, p_eps):
    """How far an output may be from the 64-bit one.

    With u = 2^-24 and A = sum p |v|: the scores carry d + 4 roundings of terms of size reach (products summed in
    fp32, the scale, the subtraction of the maximum; and the exponent's own 2^-22), which moves each probability by
    that factor, numerator and denominator alike; the sums over n keys carry n + 8 roundings each; a probability
    rounded to 16 bits moves by p_eps; the result is rounded once to dtype.  First order, times 1.01 for the rest.
    """
    u = 2.0 ** -24
    score = (d + 4) * u * reach[..., None] + 2.0 ** -22
    rel = 2 * score + 2 * (n_keys + 8) * u + p_eps
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    tiny = 2.0 ** -25 if dtype == "f16" else 1e-38  # half of the smallest fp16 step near zero
    return 1.01 * (rel * spread + half * (np.abs(want) + rel * spread)) + tiny
