"""GPU: rotary append, 4-bit pools and window/sinks attention against their 64-bit definitions."""

import numpy as np
import pytest
import torch

from oracle import serving as sv

from . import serving_cases as sc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_181_gb300 import _lib

    return _lib


# ---------------------------------------------------------------- append


def append_inputs(T, hq, hkv, d, dtype, rot, seed, fused, blocks, skip=()):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, hq + 2 * hkv, d, generator=g).to(sc.DT[dtype])
    if fused:
        dev = qkv.cuda()
        q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    else:
        q, k, v = (x.contiguous().cuda() for x in (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]))
    angle = torch.rand(50, max(rot // 2, 1), generator=g) * 300
    cs = torch.cat([angle.cos(), angle.sin()], 1) if rot else None
    pos = torch.randint(0, 50, (T,), generator=g, dtype=torch.int32)
    slots = torch.randperm(blocks * 16, generator=g)[:T].to(torch.int64)
    for t in skip:
        slots[t] = -1
    return qkv, q, k, v, pos, cs, slots


def bits(t):
    t = t.contiguous().cpu()
    return t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()]).numpy()


def rotated(x, pos, cs, interleaved):
    """Bit-exact fp32 rotation, then one rounding to x's type."""
    if cs is None:
        return x, x.float().numpy()
    y = sv.rotate(x.float().numpy(), pos.numpy(), cs.numpy(), interleaved, np.float32)
    return torch.from_numpy(y).to(x.dtype), y


APPEND = [
    # T, hq, hkv, d, rot, interleaved, fused
    (1, 32, 8, 128, 128, False, True),
    (1, 1, 1, 64, 64, False, False),
    (5, 6, 2, 64, 32, True, True),
    (33, 7, 1, 128, 64, False, True),
    (17, 40, 8, 128, 128, True, False),
    (257, 3, 3, 64, 16, False, True),
    (19, 5, 5, 128, 112, False, False),
    (9, 4, 2, 128, 48, True, True),
    (40, 8, 2, 128, 0, False, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,fused", APPEND)
def test_append_bit_exact(lib, T, hq, hkv, d, rot, inter, fused, dtype):
    blocks, skip = T // 16 + 3, ((1, 3) if T > 4 else ())
    qkv, q, k, v, pos, cs, slots = append_inputs(T, hq, hkv, d, dtype, rot, T + d, fused, blocks, skip)
    kp = torch.full((blocks * 16, hkv, d), 3.0, dtype=sc.DT[dtype], device="cuda")
    vp = torch.full_like(kp, -5.0)
    want_k, want_v = kp.cpu(), vp.cpu()
    out = lib.paged_kv_append(q, k, v, pos.cuda(), None if cs is None else cs.cuda(), slots.cuda(), kp, vp,
                              interleaved=inter, flags=lib.PKV_CHECK_BOUNDS)
    assert lib.check() == 0 and lib.last_launches() == 1
    keep = slots >= 0
    want_k[slots[keep]] = rotated(qkv[:, hq:hq + hkv], pos, cs, inter)[0][keep]
    want_v[slots[keep]] = qkv[:, hq + hkv:][keep]
    assert np.array_equal(bits(out), bits(rotated(qkv[:, :hq], pos, cs, inter)[0]))
    assert np.array_equal(bits(kp), bits(want_k)) and np.array_equal(bits(vp), bits(want_v))
    if cs is not None and dtype == "f32":  # and near the 64-bit rotation: two products and a sum, rounded each
        w = sv.rotate(qkv[:, :hq].double().numpy(), pos.numpy(), cs.double().numpy(), inter)
        size = sv.rotate(qkv[:, :hq].abs().double().numpy(), pos.numpy(),
                         np.concatenate([cs[:, : rot // 2].abs(), -cs[:, rot // 2:].abs()], 1), inter)
        other = sv.rotate(qkv[:, :hq].abs().double().numpy(), pos.numpy(), cs.abs().double().numpy(), inter)
        assert (np.abs(out.double().cpu().numpy() - w) <= 2 * 2.0 ** -24 * np.maximum(size, other) + 1e-38).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,fused", APPEND)
def test_append_q4_and_gather_bit_exact(lib, T, hq, hkv, d, rot, inter, fused, dtype):
    blocks, skip = T // 16 + 3, ((0, 2) if T > 4 else ())
    qkv, q, k, v, pos, cs, slots = append_inputs(T, hq, hkv, d, dtype, rot, 3 * T + d, fused, blocks, skip)
    pools = [sc.random_q4_pool(blocks, hkv, d, s) for s in (1, 2)]
    kp, vp = (torch.from_numpy(p.copy()).cuda() for p in pools)
    out = lib.paged_kv_append_q4(q, k, v, pos.cuda(), None if cs is None else cs.cuda(), slots.cuda(), kp, vp,
                                 interleaved=inter, flags=lib.PKV_CHECK_BOUNDS)
    assert lib.check() == 0 and lib.last_launches() == 1
    sv.q4_store(pools[0], slots.tolist(), rotated(qkv[:, hq:hq + hkv], pos, cs, inter)[1])
    sv.q4_store(pools[1], slots.tolist(), qkv[:, hq + hkv:].float().numpy())
    assert np.array_equal(bits(out), bits(rotated(qkv[:, :hq], pos, cs, inter)[0]))
    assert np.array_equal(kp.cpu().numpy(), pools[0]) and np.array_equal(vp.cpu().numpy(), pools[1])
    # Read two rows' blocks back, from the second listed block on.
    table = torch.randint(0, blocks, (2, 3), dtype=torch.int32, generator=torch.Generator().manual_seed(T))
    stage = [torch.full((2, 50, hkv, d), 9.0, dtype=sc.DT[dtype], device="cuda") for _ in range(2)]
    lib.paged_kv_gather_q4(kp, vp, table.cuda(), *stage, first_block=1, n_blocks=2, flags=lib.PKV_CHECK_BOUNDS)
    assert lib.check() == 0
    for pool, got in zip(pools, stage):
        want = torch.full((2, 50, hkv, d), 9.0, dtype=sc.DT[dtype])
        values = torch.from_numpy(sv.q4_load(pool)).view(blocks, 16, hkv, d)
        want[:, 16:48] = values[table[:, 1:].long()].reshape(2, 32, hkv, d).to(sc.DT[dtype])
        assert np.array_equal(bits(got), bits(want))


def test_append_q4_odd_values(lib):
    """Groups that are constant, huge, tiny, non-finite: stored as the format says."""
    T, hkv, d = 6, 1, 64
    x = np.random.default_rng(5).standard_normal((T, hkv, d)).astype(np.float32)
    x[0, 0, :32] = 2.5
    x[1, 0, 5] = 1e30
    x[2, 0, 40] = np.inf
    x[3, 0, 2] = np.nan
    x[4] *= 1e-7
    x[5, 0, :32] = 0
    pool = np.zeros((1, hkv, 640), np.uint8)
    v = torch.from_numpy(x).cuda()
    slots = torch.arange(T, device="cuda")
    kp, vp = torch.from_numpy(pool.copy()).cuda(), torch.from_numpy(pool.copy()).cuda()
    assert lib.paged_kv_append_q4(None, v, v, None, None, slots, kp, vp) is None
    sv.q4_store(pool, range(T), x)
    want, got = sv.q4_load(pool), sv.q4_load(vp.cpu().numpy())
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    assert torch.equal(kp, vp)


def test_append_in_place_and_on_another_stream(lib):
    qkv, q, k, v, pos, cs, slots = append_inputs(37, 8, 2, 128, "bf16", 128, 3, False, 4)
    kp, vp = (torch.zeros(64, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = lib.paged_kv_append(q, k, v, pos.cuda(), cs.cuda(), slots.cuda(), kp, vp).clone()
    wk = kp.clone()
    kp.zero_()
    pos, cs, slots = pos.cuda(), cs.cuda(), slots.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.paged_kv_append(q, k, v, pos, cs, slots, kp, vp, q_out=q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got is q and torch.equal(q, want) and torch.equal(kp, wk)


@pytest.mark.parametrize("q4", [False, True])
def test_append_flags_bad_metadata(lib, q4):
    qkv, q, k, v, pos, cs, slots = append_inputs(4, 2, 1, 64, "f16", 64, 8, False, 2)
    pos[1], pos[2] = 50, -1
    slots = torch.tensor([3, 4, 5, 32])
    shape = (2, 1, 640) if q4 else (32, 1, 64)
    kp, vp = (torch.zeros(shape, dtype=torch.uint8 if q4 else torch.float16, device="cuda") for _ in range(2))
    out = torch.full((4, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    fn = lib.paged_kv_append_q4 if q4 else lib.paged_kv_append
    fn(q, k, v, pos.cuda(), cs.cuda(), slots.cuda(), kp, vp, q_out=out, flags=lib.PKV_CHECK_BOUNDS)
    assert lib.check() == lib.PKV_DEVERR_SLOT | lib.PKV_DEVERR_POSITION
    assert (out[1:3] == 7).all() and not (out[0] == 7).any() and not (out[3] == 7).any()
    held = sv.q4_load(vp.cpu().numpy())[:, 0] if q4 else vp[:, 0].float().cpu().numpy()
    assert held[3].any() and not np.delete(held, 3, 0).any()


def test_gather_q4_flags_bad_blocks(lib):
    pool = torch.from_numpy(sc.random_q4_pool(2, 1, 64, 1)).cuda()
    table = torch.tensor([[1, 2, -1, 0]], dtype=torch.int32).cuda()
    stage = [torch.full((1, 64, 1, 64), 9.0, device="cuda") for _ in range(2)]
    lib.paged_kv_gather_q4(pool, pool, table, *stage, flags=lib.PKV_CHECK_BOUNDS)
    assert lib.check() == lib.PKV_DEVERR_BLOCK
    assert (stage[0][0, 16:48] == 9).all() and not (stage[1][0, :16] == 9).any() and not (stage[0][0, 48:] == 9).any()


# ---------------------------------------------------------------- attention


def attention(lib, rows, hq, hkv, d, dtype, window, sinks, q4=False, seed=0, flags=0, scale=None, poison=True, tail=0,
              table_pad=0, workspace=None):
    """Run one call; returns (got, want, tolerance).  What no query sees is NaN, its blocks are not listed."""
    g = torch.Generator().manual_seed(seed)
    lens = [r[1] for r in rows]
    table, blocks = sc.table_of(seed, lens, max(-(-max(lens) // 16), 1) + table_pad)
    scale = d ** -0.5 if scale is None else scale
    qsl = np.concatenate([[0], np.cumsum([r[0] for r in rows])]).astype(np.int32)
    q = torch.randn(int(qsl[-1]) + tail, hq, d, generator=g).to(sc.DT[dtype])
    if q4:
        kn, vn = (sc.random_q4_pool(blocks, hkv, d, seed + s) for s in (1, 2))
        k64, v64 = sv.q4_load(kn), sv.q4_load(vn)
        kp, vp = torch.from_numpy(kn), torch.from_numpy(vn)
    else:
        kp, vp = (torch.randn(blocks * 16, hkv, d, generator=g).to(sc.DT[dtype]) for _ in range(2))
        k64, v64 = kp.double().numpy(), vp.double().numpy()
    want, spread, reach = sv.window_attention(q[: qsl[-1]].double().numpy(), k64, v64, table, qsl, lens, scale, window,
                                              sinks)
    if poison:
        nan_pair = torch.tensor([float("nan")], dtype=torch.float16).view(torch.uint8)
        kept = torch.zeros(blocks * 16, dtype=torch.bool)
        for b, (sq, length) in enumerate(rows):
            seen = sorted({j for i in range(sq) for j in sv.visible(length - sq + i, length, window, sinks)})
            at = np.asarray(seen, dtype=np.int64)
            if at.size:
                kept[torch.from_numpy(table[b][at // 16].astype(np.int64) * 16 + at % 16)] = True
        for b in range(len(rows)):
            seen = sc.seen_blocks(rows, b, window, sinks)
            for w in range(table.shape[1]):
                if w not in seen:
                    table[b, w] = -7 if w % 2 else 10 ** 6
        for pool in (kp, vp):
            if q4:  # NaN pairs for the unseen tokens
                pairs = pool[:, :, 8 * d:].view(blocks, hkv, 16, d // 32, 2, 2).transpose(1, 2).reshape(blocks * 16, -1, 2)
                pairs[~kept] = nan_pair
                pool[:, :, 8 * d:] = pairs.view(blocks, 16, hkv, d // 8).transpose(1, 2).reshape(blocks, hkv, 2 * d)
            else:
                pool[~kept] = float("nan")
    out = torch.full((q.shape[0], hq, d), 77.0, dtype=sc.DT[dtype], device="cuda")
    fn = lib.paged_attn_q4 if q4 else lib.paged_attn_window
    fn(q.cuda(), kp.cuda(), vp.cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(qsl).cuda(),
       torch.tensor(lens, dtype=torch.int32).cuda(), max(1, max(r[0] for r in rows)), max(lens), scale, window=window,
       sinks=sinks, out=out, workspace=workspace, flags=flags | lib.PKV_CHECK_BOUNDS)
    assert lib.check() == 0 and lib.last_launches() in (1, 2)
    out = out.double().cpu().numpy()
    assert (out[qsl[-1]:] == 77).all()
    half = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    if q4 and dtype == "bf16":
        half = 2.0 ** -11  # probabilities meet fp16 values
    tol = sc.tolerance(want, spread, reach, max(lens), d, dtype, 0.0 if flags & lib.PKV_FORCE_SIMT else half)
    return out[: qsl[-1]], want, tol


def agree(got, want, tol):
    off = np.abs(got - want)
    assert not np.isnan(got).any()
    assert (off <= tol).all(), (float(off.max()), float((off / tol).max()), np.unravel_index(np.argmax(off / tol), off.shape))


ROWS = {
    "tokens": [(1, 1), (1, 17), (1, 0), (1, 16), (1, 333), (1, 100), (1, 700)],
    "few": [(2, 40), (0, 9), (5, 3), (3, 0), (4, 260), (8, 8), (3, 515)],
    "chunks": [(40, 90), (1, 5), (17, 300), (130, 130)],
    "long": [(1, 2600), (2, 1500)],
}
MASKS = [(0, 0), (1, 0), (7, 3), (64, 4), (100, 20), (33, 700)]
PATHS = [("f32", False, 0), ("bf16", False, 0), ("f16", False, 0), ("bf16", True, 0), ("f16", True, 0), ("f32", True, 0),
         ("bf16", False, 2), ("f16", True, 2)]


@pytest.mark.parametrize("dtype,q4,flags", PATHS, ids=lambda v: str(v))
@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("rows", list(ROWS))
def test_attention_masks_and_lengths(lib, rows, window, sinks, dtype, q4, flags):
    d = 128 if (window + len(rows)) % 2 else 64
    agree(*attention(lib, ROWS[rows], 6, 2, d, dtype, window, sinks, q4, seed=window + 7, flags=flags))


@pytest.mark.parametrize("q4,dtype", [(False, "bf16"), (False, "f32"), (True, "bf16"), (True, "f16")])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (8, 8), (16, 2), (40, 8), (33, 3), (64, 1), (12, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_head_layouts(lib, hq, hkv, d, q4, dtype):
    agree(*attention(lib, [(1, 129), (3, 70), (20, 64)], hq, hkv, d, dtype, 50, 5, q4, seed=hq + d))


@pytest.mark.parametrize("q4,dtype", [(False, "bf16"), (False, "f16"), (False, "f32"), (True, "bf16")])
@pytest.mark.parametrize("scale", [1.0, 0.01])
def test_attention_scales_and_padded_batch(lib, q4, dtype, scale):
    agree(*attention(lib, [(1, 300), (70, 200)], 4, 2, 128, dtype, 90, 2, q4, seed=5, scale=scale, tail=9, table_pad=3))


@pytest.mark.parametrize("q4", [False, True])
def test_attention_negative_scale_by_name(lib, q4):
    agree(*attention(lib, [(3, 50)], 4, 2, 64, "bf16", 20, 2, q4, seed=6, scale=-0.2, flags=lib.PKV_FORCE_SIMT))
    agree(*attention(lib, [(3, 50)], 4, 2, 64, "f32", 20, 2, q4, seed=6, scale=-0.2))


@pytest.mark.parametrize("q4", [False, True])
def test_attention_flags_bad_metadata(lib, q4):
    hq, hkv, d = 4, 2, 64
    pool = (torch.from_numpy(sc.random_q4_pool(8, hkv, d, 1)) if q4 else torch.randn(128, hkv, d).bfloat16()).cuda()
    q = torch.randn(5, hq, d).bfloat16().cuda()
    fn = lib.paged_attn_q4 if q4 else lib.paged_attn_window

    def call(table, qsl, lens, mq=4, ml=64):
        fn(q, pool, pool, torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(qsl, dtype=torch.int32).cuda(),
           torch.tensor(lens, dtype=torch.int32).cuda(), mq, ml, 0.1, window=20, sinks=2, flags=lib.PKV_CHECK_BOUNDS)
        return lib.check()

    good = [[0, 1, 2, 3], [4, 5, 6, 7]]
    assert call(good, [0, 2, 5], [64, 40]) == 0
    assert call([[0, 1, 9, 3], [4, 5, 6, 7]], [0, 2, 5], [64, 40]) == lib.PKV_DEVERR_BLOCK
    assert call(good, [0, 2, 5], [65, 40]) == lib.PKV_DEVERR_SEQLEN
    assert call(good, [0, 2, 5], [64, -3]) == lib.PKV_DEVERR_SEQLEN
    assert call(good, [0, 4, 3], [64, 40]) == lib.PKV_DEVERR_QUERY
    assert call(good, [0, 0, 5], [64, 40]) == lib.PKV_DEVERR_QUERY  # 5 queries, max_query_len 4
    assert call(good, [0, 2, 5], [64, 40]) == 0


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("q4", [False, True])
def test_prompt_and_decode_steps_together(lib, q4):
    """A prompt of two sequences, then decode steps: append with rotation, then attention, on one stream; every
    step's output against the 64-bit definitions on the cache as it should stand."""
    hq, hkv, d, window, sinks = 8, 2, 64, 48, 4
    g = torch.Generator().manual_seed(11)
    inv = 10000.0 ** -(torch.arange(0, d, 2, dtype=torch.float64) / d)
    ang = torch.arange(256, dtype=torch.float64)[:, None] * inv
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    table, blocks = sc.table_of(3, [160, 160], 10)
    held = [np.zeros((blocks, hkv, 10 * d), np.uint8) if q4 else np.full((blocks * 16, hkv, d), np.nan) for _ in range(2)]
    pools = [torch.from_numpy(h.copy()).cuda() if q4 else torch.from_numpy(h.copy()).bfloat16().cuda() for h in held]
    lens = [0, 0]
    for step in [(70, 33)] + [(1, 1)] * 5 + [(3, 1)] + [(0, 2)]:
        qsl = np.array([0, step[0], sum(step)], np.int32)
        pos = np.concatenate([np.arange(n, n + s) for n, s in zip(lens, step)]).astype(np.int32)
        slots = np.concatenate([table[b][np.arange(lens[b], lens[b] + s) // 16].astype(np.int64) * 16
                                + np.arange(lens[b], lens[b] + s) % 16 for b, s in enumerate(step)])
        lens = [n + s for n, s in zip(lens, step)]
        qkv = torch.randn(sum(step), hq + 2 * hkv, d, generator=g).bfloat16()
        dev = qkv.cuda()
        append, attend = ((lib.paged_kv_append_q4, lib.paged_attn_q4) if q4 else
                          (lib.paged_kv_append, lib.paged_attn_window))
        q = append(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], torch.from_numpy(pos).cuda(), cs.cuda(),
                   torch.from_numpy(slots).cuda(), *pools, flags=lib.PKV_CHECK_BOUNDS)
        out = attend(q, *pools, torch.from_numpy(table).cuda(), torch.from_numpy(qsl).cuda(),
                     torch.tensor(lens, dtype=torch.int32).cuda(), max(step), 160, d ** -0.5, window=window,
                     sinks=sinks, flags=lib.PKV_CHECK_BOUNDS)
        assert lib.check() == 0
        turned = [rotated(qkv[:, a:b], torch.from_numpy(pos), cs, False) for a, b in ((0, hq), (hq, hq + hkv))]
        if q4:
            sv.q4_store(held[0], slots, turned[1][1])
            sv.q4_store(held[1], slots, qkv[:, hq + hkv:].float().numpy())
            k64, v64 = sv.q4_load(held[0]), sv.q4_load(held[1])
        else:
            held[0][slots], held[1][slots] = turned[1][0].double().numpy(), qkv[:, hq + hkv:].double().numpy()
            k64, v64 = held
        want, spread, reach = sv.window_attention(turned[0][0].double().numpy(), k64, v64, table, qsl, lens, d ** -0.5,
                                                  window, sinks)
        tol = sc.tolerance(want, spread, reach, 160, d, "bf16", 2.0 ** -8)
        agree(out.double().cpu().numpy(), want, tol)


@pytest.mark.parametrize("q4", [False, True])
def test_captured_step_replays_with_new_contents(lib, q4):
    """Append and attention captured once; replays follow the buffers' contents, two graphs on two streams agree."""
    hq, hkv, d, B = 8, 2, 128, 3
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    cs = torch.randn(64, d, generator=g).cuda()
    table = torch.arange(B * 4, dtype=torch.int32).view(B, 4).cuda()
    qsl = torch.arange(B + 1, dtype=torch.int32).cuda()

    class State:
        def __init__(self):
            if q4:
                self.kp, self.vp = (torch.from_numpy(sc.random_q4_pool(B * 4, hkv, d, s)).cuda() for s in (1, 2))
            else:
                gg = torch.Generator().manual_seed(9)
                self.kp, self.vp = (torch.randn(B * 64, hkv, d, generator=gg).bfloat16().cuda() for _ in range(2))
            self.q, self.out = torch.empty(B, hq, d).bfloat16().cuda(), torch.empty(B, hq, d).bfloat16().cuda()
            self.qkv = torch.empty(B, hq + 2 * hkv, d).bfloat16().cuda()
            self.pos, self.slots = torch.empty(B, dtype=torch.int32).cuda(), torch.empty(B, dtype=torch.int64).cuda()
            self.lens = torch.empty(B, dtype=torch.int32).cuda()

        def load(self, qkv, lens):
            self.qkv.copy_(qkv)
            self.lens.copy_(lens)
            self.pos.copy_(lens - 1)
            at = (lens - 1).long()
            self.slots.copy_(table.long().gather(1, (at // 16)[:, None])[:, 0] * 16 + at % 16)

        def step(self):
            append, attend = ((lib.paged_kv_append_q4, lib.paged_attn_q4) if q4 else
                              (lib.paged_kv_append, lib.paged_attn_window))
            append(self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:], self.pos, cs, self.slots,
                   self.kp, self.vp, q_out=self.q)
            attend(self.q, self.kp, self.vp, table, qsl, self.lens, 1, 64, 0.1, window=30, sinks=3, out=self.out)

    eager, graphs, states = State(), [], [State(), State()]
    first = torch.tensor([20, 41, 5], dtype=torch.int32).cuda()
    x = rnd(B, hq + 2 * hkv, d)
    for s in states:
        s.load(x, first)
        s.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
        graphs.append(graph)
    eager.load(x, first)
    eager.step()
    for n in range(3):
        x, lens = rnd(B, hq + 2 * hkv, d), first + n + 1
        eager.load(x, lens)
        eager.step()
        for s in states:
            s.load(x, lens)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for s in states:
            assert torch.equal(s.out, eager.out) and torch.equal(s.kp, eager.kp) and torch.equal(s.q, eager.q)


@pytest.mark.parametrize("q4", [False, True])
def test_repeated_calls_give_the_same_bits(lib, q4):
    a = attention(lib, [(1, 3000), (2, 900)], 8, 2, 128, "bf16", 0, 0, q4, seed=3, poison=False)[0]
    for _ in range(3):
        assert np.array_equal(a, attention(lib, [(1, 3000), (2, 900)], 8, 2, 128, "bf16", 0, 0, q4, seed=3, poison=False)[0])


@pytest.mark.parametrize("q4,dtype", [(False, "bf16"), (False, "f16"), (True, "bf16"), (True, "f16")])
@pytest.mark.parametrize("rows,hq,hkv,d,window,sinks", [
    ([(300, 300), (0, 40), (257, 900)], 2, 2, 128, 0, 0),       # one head a tile: 128 tokens each
    ([(300, 700), (129, 129)], 4, 1, 64, 150, 20),
    ([(77, 1900), (26, 1300)], 5, 1, 128, 400, 130),            # 25 tokens a tile, 125 of its 128 rows
    ([(50, 5000)], 8, 1, 64, 0, 0),                             # few items over many keys: clusters share them
    ([(40, 4100), (33, 2050)], 4, 2, 128, 3000, 17),
    ([(5, 600), (3, 130)], 64, 1, 128, 64, 33),                 # two tokens a tile
    ([(3, 64), (1, 20)], 128, 1, 64, 0, 0),                     # one token a tile
    ([(2, 40)], 130, 1, 64, 9, 1),                              # more heads than a tile has rows
    ([(200, 100), (50, 0)], 2, 1, 128, 30, 2),                  # more queries than keys
])
def test_prompt_tiles(lib, rows, hq, hkv, d, window, sinks, dtype, q4):
    agree(*attention(lib, rows, hq, hkv, d, dtype, window, sinks, q4, seed=hq + len(rows), tail=3))


@pytest.mark.parametrize("q4,dtype", [(False, "bf16"), (True, "bf16"), (True, "f16")])
@pytest.mark.parametrize("rows,hq,hkv,d,window,sinks", [
    ([(1, 30000)], 8, 1, 128, 0, 0),
    ([(1, 5000), (1, 0), (2, 700)], 4, 2, 64, 1500, 40),  # so few keys that a cluster is quicker than a second launch
    ([(1, 40000), (1, 0), (2, 700)], 4, 2, 64, 33000, 40),
    ([(3, 25000)], 5, 1, 128, 0, 0),              # 15 rows
    ([(4, 26500), (1, 33)], 7, 1, 64, 25900, 1),  # 28 rows
])
def test_few_sequences_share_keys(lib, rows, hq, hkv, d, window, sinks, q4, dtype):
    """CTAs of one tile merge through a workspace (the caller's, the binding's) or, without one, in clusters."""
    size = lib.window_workspace_size(10 ** 4, hq, hkv, d, sc.DT[dtype], len(rows), max(r[0] for r in rows),
                                     max(r[1] for r in rows), window, sinks, q4)
    if rows[0][1] < 9000:
        assert size == 0
        agree(*attention(lib, rows, hq, hkv, d, dtype, window, sinks, q4, seed=4, tail=2))
        assert lib.last_launches() == 1
        return
    assert size > 0 and size % 16 == 0
    for ws in (None, torch.full((size,), 255, dtype=torch.uint8, device="cuda"), torch.empty(0, device="cuda"),
               torch.empty(size - 16, dtype=torch.uint8, device="cuda")):
        got = attention(lib, rows, hq, hkv, d, dtype, window, sinks, q4, seed=4, workspace=ws, tail=2)
        assert lib.last_launches() == (2 if ws is None or ws.numel() >= size else 1)
        agree(*got)


def test_shared_keys_on_another_stream(lib):
    """The binding's own scratch belongs to the stream of the call."""
    g = torch.Generator().manual_seed(0)
    pool = torch.randn(4096, 1, 64, generator=g).bfloat16().cuda()
    q = torch.randn(1, 4, 64, generator=g).bfloat16().cuda()
    meta = (torch.arange(256, dtype=torch.int32)[None].cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda(),
            torch.tensor([4096], dtype=torch.int32).cuda())
    want = lib.paged_attn_window(q, pool, pool, *meta, 1, 4096, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(q) for _ in range(20)]
    for out in outs:
        lib.paged_attn_window(q, pool, pool, *meta, 1, 4096, 0.1, out=out, stream=side)
        torch.full((1 << 16,), 3.0, device="cuda")  # would land in scratch freed too early
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_ordinary_calls_take_the_fast_way(lib, monkeypatch):
    def no(*a, **k):
        raise AssertionError("the careful path ran")

    pool = torch.zeros(64, 2, 64, dtype=torch.bfloat16, device="cuda")
    four = torch.zeros(4, 2, 640, dtype=torch.uint8, device="cuda")
    qkv = torch.zeros(3, 8, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    table, qsl, lens = torch.zeros(1, 4, **i32), torch.tensor([0, 3], **i32), torch.tensor([20], **i32)
    pos, slots, cs = torch.arange(3, **i32), torch.arange(3, device="cuda"), torch.zeros(9, 64, device="cuda")
    lib._code("f", torch.float32)
    monkeypatch.setattr(lib, "_attn_window", no)
    monkeypatch.setattr(lib, "_append", no)
    monkeypatch.setattr(lib, "_refuse_placement", no)
    q = lib.paged_kv_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, cs, slots, pool, pool)
    lib.paged_kv_append_q4(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, cs, slots, four, four, interleaved=True)
    stage = torch.zeros(1, 64, 2, 64, device="cuda")
    lib.paged_kv_gather_q4(four, four, table, stage, stage)
    lib.paged_attn_window(q, pool, pool, table, qsl, lens, 3, 64, 0.1, stream=torch.cuda.current_stream())
    lib.paged_attn_q4(q, four, four, table, qsl, lens, 3, 64, 0.1, window=4)
    torch.cuda.synchronize()


@pytest.mark.parametrize("q4", [False, True])
def test_many_prompt_tiles_in_turn(lib, q4):
    """More items than SMs, of one and of two query tiles, whole and ragged, with keys and without: what one CTA works
    through in turn."""
    rows = [(70, 90), (130, 130), (0, 50), (33, 400), (64, 70), (200, 100), (129, 300)] * 6
    agree(*attention(lib, rows, 8, 8, 64, "bf16", 45, 3, q4, seed=21, tail=1))
    rows = [(97, 97), (40, 41), (64, 64), (17, 200), (5, 0)] * 9
    agree(*attention(lib, rows, 16, 4, 128, "f16", 0, 0, q4, seed=22))


@pytest.mark.parametrize("q4", [False, True])
def test_offsets_past_32_bits(lib, q4):
    """Blocks, query rows and output rows whose byte offsets pass 2^32 (and element offsets 2^31): the same bits as from
    a small cache."""
    hq, hkv, d = 16, 8, 128
    small = 40
    blocks = (1 << 32) // (10 * d * hkv) + 77 if q4 else (1 << 31) // (16 * hkv * d) + 77
    lead = (1 << 31) // (hq * d) + 11  # query tokens before the ones of interest
    g = torch.Generator().manual_seed(5)
    rows = [(1, 300), (70, 200), (9, 40)]
    tokens = sum(r[0] for r in rows)
    fill = torch.randn(3, sum(r[1] for r in rows), hkv, d, generator=g).bfloat16().cuda()
    q = torch.randn(tokens, hq, d, generator=g).bfloat16().cuda()
    table, used = sc.table_of(1, [r[1] for r in rows], 19, spare=1)
    assert used <= small
    append, attend = ((lib.paged_kv_append_q4, lib.paged_attn_q4) if q4 else (lib.paged_kv_append, lib.paged_attn_window))
    lens = torch.tensor([r[1] for r in rows], dtype=torch.int32).cuda()
    slots = np.concatenate([table[b][np.arange(r[1]) // 16].astype(np.int64) * 16 + np.arange(r[1]) % 16
                            for b, r in enumerate(rows)])
    cs = torch.randn(512, d, generator=g).cuda()
    pos = torch.from_numpy(np.concatenate([np.arange(r[1]) for r in rows]).astype(np.int32)).cuda()
    got = []
    for n, first in ((small, 0), (blocks, blocks - used)):
        shape, kind = ((n, hkv, 10 * d), torch.uint8) if q4 else ((n * 16, hkv, d), torch.bfloat16)
        kp, vp = (torch.empty(shape, dtype=kind, device="cuda") for _ in range(2))
        tb = torch.from_numpy(np.where(table < used, table + first, table).astype(np.int32)).cuda()
        append(None, fill[0], fill[1], pos, cs, torch.from_numpy(slots + first * 16).cuda(), kp, vp,
               flags=lib.PKV_CHECK_BOUNDS)
        for flags in (0, lib.PKV_FORCE_SIMT):
            for ahead in (0, lead) if first else (0,):
                qs = q if not ahead else torch.empty(ahead + tokens, hq, d, dtype=q.dtype, device="cuda")
                out = torch.zeros_like(qs)
                if ahead:
                    qs[ahead:] = q
                for b, most in ((0, 1), (1, 70), (2, 9)):  # a decode step, a prompt, many rows of one tile
                    at = ahead + sum(r[0] for r in rows[:b])
                    qsl = torch.tensor([at, at + rows[b][0]], dtype=torch.int32).cuda()
                    attend(qs, kp, vp, tb[b:b + 1], qsl, lens[b:b + 1], most, 300, 0.09, window=150, sinks=5, out=out,
                           flags=flags | lib.PKV_CHECK_BOUNDS)
                got.append((flags, out[ahead:].clone()))
                assert ahead == 0 or not out[:ahead].any()
        assert lib.check() == 0
        if q4:
            stage = [torch.empty(3, 19 * 16, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            for b, r in enumerate(rows):
                n_blocks = -(-r[1] // 16)
                lib.paged_kv_gather_q4(kp, vp, tb[b:b + 1], stage[0][b:b + 1], stage[1][b:b + 1], n_blocks=n_blocks)
                got.append(("stage", torch.stack([s[b, : r[1]] for s in stage])))
        del kp, vp
    for what in {w for w, _ in got}:
        same = [x for w, x in got if w == what]
        if what == "stage":
            assert all(torch.equal(a, b) for a, b in zip(same[:3], same[3:]))
        else:
            assert len(same) == 3 and all(torch.equal(same[0], x) for x in same[1:]) and same[0].any()


@pytest.mark.parametrize("q4", [False, True])
def test_seventy_thousand_sequences(lib, q4):
    """More sequences than a grid's second dimension holds, some without keys, one key or one block each."""
    B, hq, hkv, d = 70001, 2, 1, 64
    g = torch.Generator().manual_seed(6)
    n = torch.randint(0, 17, (B,), generator=g, dtype=torch.int32)
    qkv = torch.randn(B, hq + 2 * hkv, d, generator=g).half()
    kp, vp = (torch.zeros((64, hkv, 10 * d) if q4 else (1024, hkv, d), dtype=torch.uint8 if q4 else torch.float16,
                          device="cuda") for _ in range(2))
    slots = torch.full((B,), -1, dtype=torch.int64)
    at = torch.arange(0, B, 69)[:1000]
    slots[at] = torch.arange(1000)
    append, attend = ((lib.paged_kv_append_q4, lib.paged_attn_q4) if q4 else (lib.paged_kv_append, lib.paged_attn_window))
    dev = qkv.cuda()
    q = append(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], None, None, slots.cuda(), kp, vp)
    assert torch.equal(q, dev[:, :hq])
    table = torch.arange(B, dtype=torch.int32)[:, None] % 62
    out = attend(q, kp, vp, table.cuda(), torch.arange(B + 1, dtype=torch.int32).cuda(), n.cuda(), 1, 16, 0.125)
    if q4:
        k, v = (torch.from_numpy(sv.q4_load(p.cpu().numpy())).view(64, 16, d) for p in (kp, vp))
    else:
        k, v = (p.cpu().double().view(64, 16, d) for p in (kp, vp))
    x = qkv[:, :hq].double()
    s = torch.einsum("bhd,bkd->bhk", x, k[table[:, 0].long()]) * 0.125
    seen = torch.arange(16)[None, None] < n[:, None, None]
    p = torch.where(seen, s, torch.tensor(-float("inf"))).softmax(-1).nan_to_num(0)
    w = v[table[:, 0].long()]
    want, spread = torch.einsum("bhk,bkd->bhd", p, w), torch.einsum("bhk,bkd->bhd", p, w.abs())
    reach = (torch.einsum("bhd,bkd->bhk", x.abs(), k[table[:, 0].long()].abs()) * 0.125).amax(-1)
    agree(out.double().cpu().numpy(), want.numpy(),
          sc.tolerance(want.numpy(), spread.numpy(), reach.numpy(), 16, d, "f16", 2.0 ** -11))


@pytest.mark.parametrize("dtype,q4,flags", PATHS, ids=lambda v: str(v))
@pytest.mark.parametrize("rows", [[(90, 60), (2, 40)], [(9, 7), (1, 5)]], ids=["prompt", "few"])
def test_widest_window_with_queries_before_the_keys(lib, rows, dtype, q4, flags):
    """A window as large as the type allows, and rows whose first queries see no key."""
    agree(*attention(lib, rows, 4, 2, 64, dtype, 2 ** 31 - 1, 2, q4, seed=8, flags=flags))


@pytest.mark.parametrize("q4,dtype", [(False, "bf16"), (True, "f16"), (False, "f32")])
@pytest.mark.parametrize("group", [128, 160])
def test_heads_that_fill_or_pass_a_tile(lib, group, q4, dtype):
    """128 query heads a kv head are a whole tile for each token; more take the few-rows kernel at every length."""
    agree(*attention(lib, [(5, 90), (1, 33), (40, 40)], group, 1, 64, dtype, 30, 1, q4, seed=group))


@pytest.mark.parametrize("q4", [False, True])
def test_two_billion_keys(lib, q4):
    """The longest sequence a call takes (its table repeats four blocks): the answer is that of the four."""
    n, hq, d = 2 ** 31 - 256, 8, 64
    g = torch.Generator().manual_seed(4)
    if q4:
        kn, vn = (sc.random_q4_pool(4, 1, d, s) for s in (1, 2))
        kp, vp, k, v = torch.from_numpy(kn).cuda(), torch.from_numpy(vn).cuda(), sv.q4_load(kn), sv.q4_load(vn)
    else:
        kp, vp = (torch.randn(64, 1, d, generator=g).bfloat16().cuda() for _ in range(2))
        k, v = kp.cpu().double().numpy(), vp.cpu().double().numpy()
    q = torch.randn(1, hq, d, generator=g).bfloat16().cuda()
    table = (torch.arange(n // 16, device="cuda", dtype=torch.int32) % 4)[None]
    fn = lib.paged_attn_q4 if q4 else lib.paged_attn_window
    out = fn(q, kp, vp, table, torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
             1, n, 0.125, flags=lib.PKV_CHECK_BOUNDS)
    assert lib.check() == 0
    want, spread, reach = sv.window_attention(q.cpu().double().numpy(), k, v, np.arange(4)[None], [0, 1], [64], 0.125, 0, 0)
    # Sums in fp32 run over the keys of one lane (at most n / (64 CTAs x 4 warps x 8 lanes) roundings of a sum, and the
    # merges of 64 x 32 of them), in place of the four blocks' 64.
    agree(out.double().cpu().numpy(), want, sc.tolerance(want, spread, reach, n // 2048 + 2048, d, "bf16", 2.0 ** -8))


@pytest.mark.parametrize("q4", [False, True])
def test_captured_calls_keep_their_own_scratch(lib, q4):
    """Two graphs of calls that split their keys over a workspace of the binding's, replayed at the same time."""
    n, d = 32768, 64
    size = lib.window_workspace_size(n // 16, 4, 1, d, torch.bfloat16, 1, 1, n, 0, 0, q4)
    assert size > 0
    g = torch.Generator().manual_seed(3)
    if q4:
        kp, vp = (torch.from_numpy(sc.random_q4_pool(n // 16, 1, d, s)).cuda() for s in (1, 2))
    else:
        kp, vp = (torch.randn(n, 1, d, generator=g).bfloat16().cuda() for _ in range(2))
    meta = (torch.arange(n // 16, dtype=torch.int32)[None].cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda(),
            torch.tensor([n], dtype=torch.int32).cuda(), 1, n, 0.125)
    fn = lib.paged_attn_q4 if q4 else lib.paged_attn_window
    qs = [torch.randn(1, 4, d, generator=g).bfloat16().cuda() for _ in range(2)]
    want = [fn(q, kp, vp, *meta) for q in qs]
    assert lib.last_launches() == 2
    graphs, outs = [], [[torch.zeros_like(q) for _ in range(4)] for q in qs]
    for q, out in zip(qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for o in out:
                fn(q, kp, vp, *meta, out=o)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for out in outs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(o, w) for o in out)


@pytest.mark.parametrize("q4", [False, True])
def test_captured_prompts_on_two_streams(lib, q4):
    """Prompt calls of one launch and of two (whole waves, and clusters for the rest), captured and replayed at once."""
    d, hkv, n = 128, 8, 8192
    g = torch.Generator().manual_seed(13)
    if q4:
        kp, vp = (torch.randint(0, 50, (n // 16, hkv, 10 * d), generator=g, dtype=torch.uint8).cuda() for _ in range(2))
    else:
        kp, vp = (torch.randn(n, hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.randperm(n // 16, generator=g).int()[None].cuda()
    fn = lib.paged_attn_q4 if q4 else lib.paged_attn_window
    calls, inputs = [], []
    for tokens, hq, window, launches in ((2048, 40, 0, 2), (300, 16, 700, 1)):
        q = torch.randn(tokens, hq, d, generator=g).bfloat16().cuda()
        meta = (torch.tensor([0, tokens], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda(), tokens, n)
        run = lambda out, q=q, meta=meta, window=window: fn(q, kp, vp, table, *meta, 0.09, window=window, out=out,  # noqa: E731
                                                                  flags=lib.PKV_CHECK_BOUNDS)
        want = run(None)
        assert lib.last_launches() == launches and want.isfinite().all()
        graph, outs = torch.cuda.CUDAGraph(), [torch.zeros_like(q) for _ in range(3)]
        with torch.cuda.graph(graph):
            for o in outs:
                run(o)
        calls.append((graph, outs, want))
        inputs.append((q, meta))  # a graph reads them where they are: they have to live as long as it does
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for _, outs, _ in calls:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        for st, (graph, _, _) in zip(streams, calls):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for _, outs, want in calls for o in outs)
    assert lib.check() == 0
