"""CPU: the serving operators' oracle against closed forms and brute force."""

import numpy as np
import pytest

from oracle import serving as sv


def test_rotation_is_a_turn_by_the_angle():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 64))
    angle = rng.uniform(0, 7, (9, 16))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos = np.array([0, 8, 3, 3, 1])
    for inter in (False, True):
        y = sv.rotate(x, pos, cs, inter)
        a, b = (x[..., 0:32:2], x[..., 1:32:2]) if inter else (x[..., :16], x[..., 16:32])
        c, d = (y[..., 0:32:2], y[..., 1:32:2]) if inter else (y[..., :16], y[..., 16:32])
        z = (a + 1j * b) * np.exp(1j * angle[pos])[:, None]
        assert np.allclose(c, z.real, atol=1e-14) and np.allclose(d, z.imag, atol=1e-14)
        assert np.array_equal(y[..., 32:], x[..., 32:])


def test_relative_positions_only_enter_scores():
    rng = np.random.default_rng(1)
    inv = 10000.0 ** -(np.arange(0, 64, 2) / 64)
    ang = np.arange(64)[:, None] * inv
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    dots = [float((sv.rotate(q, [p + 7], cs, False) * sv.rotate(k, [p], cs, False)).sum()) for p in (0, 5, 41)]
    assert np.allclose(dots, dots[0], atol=1e-12)


def test_q4_round_trip_is_within_half_a_step():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((40, 3, 128)) * rng.choice([1e-3, 1, 300], (40, 3, 1))).astype(np.float32)
    codes, step, low = sv.q4_quantise(x)
    v = sv.q4_values(codes, step, low).reshape(40, 3, 4, 32)
    g = x.astype(np.float64).reshape(40, 3, 4, 32)
    s, lo = step.astype(np.float64)[..., None], low.astype(np.float64)[..., None]
    # half a step, plus the fp16 roundings of low, step (15 of them at the top) and the value itself
    h = 2.0 ** -11
    assert (np.abs(v - g) <= 0.5 * s + h * (np.abs(lo) + 15 * s + np.abs(g)) + 2.0 ** -24).all()
    assert codes.max() == 15 and codes.min() == 0


def test_q4_edges():
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, 32:] = 7.25
    codes, step, low = sv.q4_quantise(x)
    assert (codes == 0).all() and (step == 0).all() and list(low[0, 0]) == [0, 7.25]
    x[0, 0, 3], x[0, 0, 40] = np.nan, 1e9
    codes, step, low = sv.q4_quantise(x)
    v = sv.q4_values(codes, step, low)[0, 0]
    assert np.isnan(v[:32]).all() and np.isfinite(v[32:]).all() and abs(v[40] - 32768) <= 16


def test_q4_store_load_and_layout():
    rng = np.random.default_rng(3)
    pool = np.full((3, 2, 640), 0xAB, np.uint8)
    x = rng.standard_normal((4, 2, 64)).astype(np.float32)
    sv.q4_store(pool, [17, -1, 0, 47], x)
    codes, step, low = sv.q4_quantise(x)
    assert pool[1, 1, 32 + 5] == codes[0, 1, 10] | codes[0, 1, 11] << 4
    assert pool[0, 0, 512:516].view(np.float16).tolist() == [step[2, 0, 0], low[2, 0, 0]]
    v = sv.q4_load(pool)
    assert np.array_equal(v[47], sv.q4_values(codes, step, low)[3])
    assert (pool[2, :, :480] == 0xAB).all()  # other tokens of a block keep their bytes


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 9), (1, 0), (3, 2), (5, 40), (100, 1)])
def test_window_attention_against_a_dense_mask(window, sinks):
    rng = np.random.default_rng(4)
    rows = [(3, 20), (1, 0), (4, 2), (0, 6), (7, 33)]
    hq, hkv, d = 4, 2, 8
    table = rng.permutation(20)[:15].reshape(5, 3)
    k, v = rng.standard_normal((2, 320, hkv, d))
    qsl = np.concatenate([[0], np.cumsum([r[0] for r in rows])])
    q = rng.standard_normal((qsl[-1], hq, d))
    out, spread, reach = sv.window_attention(q, k, v, table, qsl, [r[1] for r in rows], 0.4, window, sinks)
    for b, (sq, length) in enumerate(rows):
        at = (table[b][:, None] * 16 + np.arange(16)).ravel()[:length]
        p, j = np.arange(length - sq, length)[:, None], np.arange(length)[None]
        mask = j <= p
        if window:
            mask &= (j < sinks) | (j > p - window)
        for h in range(hq):
            s = np.where(mask, 0.4 * q[qsl[b]:qsl[b + 1], h] @ k[at, h // 2].T, -np.inf)
            e = np.where(mask, np.exp(s - s.max(-1, initial=-1e30, keepdims=True)), 0)
            want = e @ v[at, h // 2] / np.maximum(e.sum(-1, keepdims=True), 1e-300)
            assert np.allclose(out[qsl[b]:qsl[b + 1], h], want, atol=1e-12)
    assert (spread >= np.abs(out) - 1e-12).all() and (reach >= 0).all()
