"""CPU: what the serving operators refuse, in C and in the binding."""

import pytest
import torch

from paged_kv_cache_181_gb300 import _lib as lib

P = 4096  # a 16-byte aligned stand-in for a pointer: every call below is refused before it is used


def append(name="paged_kv_append", q=P, qs=512, k=P, ks=128, v=P, vs=128, pos=P, cs=P, maxpos=64, rot=64, slots=P, T=4,
           hq=8, qo=P, kp=P, vp=P, n=64, hkv=2, d=64, dt=lib.PKV_BF16, flags=0):
    return getattr(lib.lib, name)(q, qs, k, ks, v, vs, pos, cs, maxpos, rot, slots, T, hq, qo, kp, vp, n, hkv, d, dt,
                                  flags, None)


@pytest.mark.parametrize("name", ["paged_kv_append", "paged_kv_append_q4"])
@pytest.mark.parametrize("change,status,word", [
    (dict(T=-1), lib.PKV_ERR_INVALID_ARG, "negative"),
    (dict(hkv=0), lib.PKV_ERR_INVALID_ARG, "zero size"),
    (dict(d=96), lib.PKV_ERR_UNSUPPORTED, "head dim"),
    (dict(dt=7), lib.PKV_ERR_UNSUPPORTED, "dtype"),
    (dict(rot=80), lib.PKV_ERR_INVALID_ARG, "rot_dim"),
    (dict(rot=24), lib.PKV_ERR_UNSUPPORTED, "multiple of 16"),
    (dict(q=None), lib.PKV_ERR_INVALID_ARG, "NULL"),
    (dict(cs=None), lib.PKV_ERR_INVALID_ARG, "NULL"),
    (dict(slots=None), lib.PKV_ERR_INVALID_ARG, "NULL"),
    (dict(k=P + 8), lib.PKV_ERR_INVALID_ARG, "aligned"),
    (dict(vs=129), lib.PKV_ERR_INVALID_ARG, "aligned"),
    (dict(cs=P + 4), lib.PKV_ERR_INVALID_ARG, "aligned"),
    (dict(qs=1024), lib.PKV_ERR_INVALID_ARG, "contiguous"),  # q_out is q, but q has gaps
    (dict(T=2 ** 31), lib.PKV_ERR_UNSUPPORTED, "too many"),
    (dict(hq=70000), lib.PKV_ERR_UNSUPPORTED, "too many"),
])
def test_append_refusals(name, change, status, word):
    assert append(name, **change) == status
    assert word in lib.last_error() and name in lib.last_error()
    assert lib.last_launches() == 0


@pytest.mark.parametrize("name", ["paged_kv_append", "paged_kv_append_q4"])
def test_append_of_nothing_is_a_no_op(name):
    assert append(name, T=0, q=None, k=None, v=None, slots=None) == lib.PKV_OK
    assert lib.last_launches() == 0


def attn(name="paged_attn_window", q=P, Tq=4, hq=4, kp=P, vp=P, nblk=8, bs=16, hkv=2, d=64, dt=lib.PKV_BF16, table=P,
         B=1, W=2, qsl=P, lens=P, mq=4, ml=32, scale=0.125, window=0, sinks=0, out=P, ws=None, nws=0,
         flags=0):
    return getattr(lib.lib, name)(q, Tq, hq, kp, vp, nblk, bs, hkv, d, dt, table, B, W, qsl, lens, mq, ml, scale,
                                  window, sinks, out, ws, nws, flags, None)


@pytest.mark.parametrize("name", ["paged_attn_window", "paged_attn_q4"])
@pytest.mark.parametrize("change,status,word", [
    (dict(B=-1), lib.PKV_ERR_INVALID_ARG, "negative"),
    (dict(hq=3), lib.PKV_ERR_INVALID_ARG, "multiple"),
    (dict(bs=32), lib.PKV_ERR_UNSUPPORTED, "block_size"),
    (dict(d=80), lib.PKV_ERR_UNSUPPORTED, "head dim"),
    (dict(dt=3), lib.PKV_ERR_UNSUPPORTED, "dtype"),
    (dict(window=-1), lib.PKV_ERR_INVALID_ARG, "window"),
    (dict(sinks=-2), lib.PKV_ERR_INVALID_ARG, "sinks"),
    (dict(scale=float("nan")), lib.PKV_ERR_INVALID_ARG, "finite"),
    (dict(scale=0.0), lib.PKV_ERR_UNSUPPORTED, "PKV_FORCE_SIMT"),
    (dict(scale=-1.0, dt=lib.PKV_F16), lib.PKV_ERR_UNSUPPORTED, "PKV_FORCE_SIMT"),
    (dict(ml=33), lib.PKV_ERR_INVALID_ARG, "max_seq_len"),
    (dict(table=None), lib.PKV_ERR_INVALID_ARG, "NULL"),
    (dict(out=P + 2), lib.PKV_ERR_INVALID_ARG, "aligned"),
    (dict(ws=P + 8), lib.PKV_ERR_INVALID_ARG, "workspace"),
    (dict(nblk=0), lib.PKV_ERR_INVALID_ARG, "without blocks"),
    (dict(mq=2 ** 31 - 1), lib.PKV_ERR_UNSUPPORTED, "too many"),
    (dict(W=2 ** 27, ml=2 ** 31 - 255), lib.PKV_ERR_UNSUPPORTED, "max_seq_len"),
])
def test_attention_refusals(name, change, status, word):
    assert attn(name, **change) == status
    assert word in lib.last_error() and name in lib.last_error()
    assert lib.last_launches() == 0


@pytest.mark.parametrize("name", ["paged_attn_window", "paged_attn_q4"])
def test_attention_of_nothing_is_a_no_op(name):
    for change in (dict(Tq=0), dict(B=0), dict(mq=0)):
        assert attn(name, q=None, out=None, **change) == lib.PKV_OK


@pytest.mark.parametrize("change,status,word", [
    (dict(first=1, n=2), lib.PKV_ERR_INVALID_ARG, "table width"),
    (dict(rows=31), lib.PKV_ERR_INVALID_ARG, "staging rows"),
    (dict(d=32), lib.PKV_ERR_UNSUPPORTED, "head dim"),
    (dict(dt=9), lib.PKV_ERR_UNSUPPORTED, "dtype"),
    (dict(kp=None), lib.PKV_ERR_INVALID_ARG, "NULL"),
    (dict(sk=P + 4), lib.PKV_ERR_INVALID_ARG, "aligned"),
    (dict(B=-1), lib.PKV_ERR_INVALID_ARG, "negative"),
])
def test_gather_refusals(change, status, word):
    a = dict(kp=P, nblk=8, B=2, W=2, first=0, n=2, sk=P, rows=32, d=64, dt=lib.PKV_BF16) | change
    got = lib.lib.paged_kv_gather_q4(a["kp"], P, a["nblk"], P, a["B"], a["W"], a["first"], a["n"], a["sk"], P,
                                     a["rows"], 2, a["d"], a["dt"], 0, None)
    assert got == status and word in lib.last_error()


def test_record_size():
    assert [lib.lib.pkv_q4_block_bytes(d) for d in (64, 128, 96, 0, -1)] == [640, 1280, 0, 0, 0]
    assert lib.q4_block_bytes(128) == 1280
    with pytest.raises(lib.PkvError):
        lib.q4_block_bytes(80)


def _append_args(**change):
    T, hq, hkv, d = 3, 4, 2, 64
    a = dict(q=torch.zeros(T, hq, d), k=torch.zeros(T, hkv, d), v=torch.zeros(T, hkv, d),
             positions=torch.zeros(T, dtype=torch.int32), cos_sin=torch.zeros(8, 64),
             slot_mapping=torch.zeros(T, dtype=torch.int64), key_pool=torch.zeros(32, hkv, d),
             value_pool=torch.zeros(32, hkv, d))
    return a | change


@pytest.mark.parametrize("change,word", [
    (dict(v=torch.zeros(3, 2, 32)), "k and v"),
    (dict(q=torch.zeros(2, 4, 64)), "q must be"),
    (dict(q_out=torch.zeros(3, 5, 64)), "q_out shape"),
    (dict(q=None, q_out=torch.zeros(3, 4, 64)), "without q"),
    (dict(value_pool=torch.zeros(16, 2, 64)), "one shape"),
    (dict(key_pool=torch.zeros(32, 1, 64), value_pool=torch.zeros(32, 1, 64)), "pools must be"),
    (dict(k=torch.zeros(3, 2, 64).half()), "share one dtype"),
    (dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), "int64"),
    (dict(positions=torch.zeros(3, dtype=torch.int64)), "int32"),
    (dict(positions=None), "int32"),
    (dict(cos_sin=torch.zeros(8, 64).double()), "float32"),
    (dict(), "CUDA"),  # everything right, but on the host
])
def test_binding_refuses_append_arguments(change, word):
    with pytest.raises(ValueError, match=word):
        lib.paged_kv_append(**_append_args(**change))


def test_binding_refuses_pools_of_the_other_kind():
    with pytest.raises(ValueError, match="pools must be"):
        lib.paged_kv_append_q4(**_append_args())
    q = torch.zeros(3, 4, 64)
    meta = (torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    plain, four = torch.zeros(32, 2, 64), torch.zeros(2, 2, 640, dtype=torch.uint8)
    with pytest.raises(ValueError, match="pools must be"):
        lib.paged_attn_q4(q, plain, plain, *meta, 3, 32, 1.0)
    with pytest.raises(ValueError, match="pools must be"):
        lib.paged_attn_window(q, four, four, *meta, 3, 32, 1.0)
    with pytest.raises(ValueError, match="B\\+1"):
        lib.paged_attn_window(q, plain, plain, meta[0], meta[2], meta[2], 3, 32, 1.0)
    with pytest.raises(ValueError, match="out shape"):
        lib.paged_attn_window(q, plain, plain, *meta, 3, 32, 1.0, out=torch.zeros(3, 4, 32))
    with pytest.raises(ValueError, match="CUDA"):
        lib.paged_attn_window(q, plain, plain, *meta, 3, 32, 1.0)


def test_binding_refuses_torn_heads():
    base = torch.zeros(3, 64, 4).transpose(1, 2)
    with pytest.raises(ValueError, match="contiguous"):
        lib._token_stride("f", "q", base)
    assert lib._token_stride("f", "q", torch.zeros(3, 8, 64)[:, 2:6]) == 512
    assert lib._token_stride("f", "q", torch.zeros(1, 8, 64)[:, 2:6]) == 256


class FakeTensor:
    """What csrc/fastcall.c asks of a tensor, without a GPU."""

    def __init__(self, shape, dtype, device=0, contiguous=True, stride=None, at=P):
        self.shape, self.dtype, self.device, self.contiguous = torch.Size(shape), dtype, device, contiguous
        self.at = at
        self.strides = stride or torch.empty(shape, dtype=torch.uint8).stride()

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return self.at

    def stride(self):
        return self.strides


@pytest.fixture
def fast(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("has a GPU: the addresses here are not memory")
    from paged_kv_cache_181_gb300 import _fastcall as f

    f.setup((torch.float32, torch.bfloat16, torch.float16), torch.uint8, torch.int32, torch.int64, lambda: 0, lambda d: 0)
    yield f
    monkeypatch.setattr(lib, "_DTYPES", {})  # the binding sets it up again with torch's own
    lib._code("f", torch.float32)


def fast_attend(**change):
    f = FakeTensor
    a = dict(q4=False, q=f((3, 4, 64), torch.bfloat16), kp=f((32, 2, 64), torch.bfloat16), vp=f((32, 2, 64), torch.bfloat16),
             table=f((1, 2), torch.int32), qsl=f((2,), torch.int32), lens=f((1,), torch.int32), mq=3, ml=32, scale=0.1,
             window=0, sinks=0, out=f((3, 4, 64), torch.bfloat16), ws=None, flags=0, bs=16, stream=None)
    return list((a | change).values())


def test_fast_attention_makes_the_call(fast):
    assert fast.attend(*fast_attend()) == lib.PKV_ERR_CUDA  # it got as far as the device
    assert fast.attend(*fast_attend(window=-1)) == lib.PKV_ERR_INVALID_ARG and "window" in lib.last_error()
    four = FakeTensor((2, 2, 640), torch.uint8)
    assert fast.attend(*fast_attend(q4=True, kp=four, vp=four)) == lib.PKV_ERR_CUDA


@pytest.mark.parametrize("change", [
    dict(q=FakeTensor((3, 4, 64), torch.float64)), dict(q=FakeTensor((3, 4, 64), torch.bfloat16, device=1)),
    dict(q=FakeTensor((3, 4, 64), torch.bfloat16, device=-1)), dict(kp=FakeTensor((32, 2, 64), torch.float16)),
    dict(vp=FakeTensor((16, 2, 64), torch.bfloat16)), dict(kp=FakeTensor((30, 2, 64), torch.bfloat16)),
    dict(table=FakeTensor((1, 2), torch.int64)), dict(table=FakeTensor((2,), torch.int32)),
    dict(lens=FakeTensor((2,), torch.int32)), dict(qsl=FakeTensor((3,), torch.int32)),
    dict(out=FakeTensor((3, 4, 32), torch.bfloat16)), dict(out=FakeTensor((3, 4, 64), torch.bfloat16, contiguous=False)),
    dict(ws=FakeTensor((64,), torch.uint8, device=1)), dict(bs=32), dict(mq=2.0), dict(mq=2 ** 40), dict(scale="x"), dict(q4=True),
    dict(q=None), dict(stream=7), dict(flags=None),
])
def test_fast_attention_leaves_the_rest_alone(fast, change):
    assert fast.attend(*fast_attend(**change)) is None


def fast_append(**change):
    f = FakeTensor
    row = (8 * 64, 64, 1)
    a = dict(q4=False, q=f((3, 4, 64), torch.float16, stride=row), k=f((3, 2, 64), torch.float16, stride=row),
             v=f((3, 2, 64), torch.float16, stride=row), pos=f((3,), torch.int32), cs=f((9, 32), torch.float32),
             slots=f((3,), torch.int64), kp=f((32, 2, 64), torch.float16), vp=f((32, 2, 64), torch.float16), inter=False,
             q_out=f((3, 4, 64), torch.float16, at=2 * P), flags=0, stream=None)
    return list((a | change).values())


def test_fast_append_makes_the_call(fast):
    assert fast.append(*fast_append()) == lib.PKV_ERR_CUDA
    assert fast.append(*fast_append(cs=FakeTensor((9, 24), torch.float32))) == lib.PKV_ERR_UNSUPPORTED
    assert fast.gather(FakeTensor((4, 2, 640), torch.uint8), FakeTensor((4, 2, 640), torch.uint8),
                       FakeTensor((1, 2), torch.int32), FakeTensor((1, 32, 2, 64), torch.float16),
                       FakeTensor((1, 32, 2, 64), torch.float16), 1, None, 0, None) == lib.PKV_ERR_CUDA


@pytest.mark.parametrize("change", [
    dict(q=None), dict(cs=None), dict(q_out=None), dict(k=FakeTensor((3, 2, 64), torch.float16, stride=(512, 1, 2))),
    dict(q=FakeTensor((2, 4, 64), torch.float16)), dict(v=FakeTensor((3, 2, 64), torch.bfloat16)),
    dict(pos=FakeTensor((3,), torch.int64)), dict(pos=FakeTensor((4,), torch.int32)), dict(cs=FakeTensor((9, 0), torch.float32)),
    dict(slots=FakeTensor((3,), torch.int32)), dict(kp=FakeTensor((32, 1, 64), torch.float16)), dict(q4=True),
    dict(slots=FakeTensor((3,), torch.int64, contiguous=False)), dict(v=FakeTensor((3, 2, 64), torch.float16, device=1)),
])
def test_fast_append_leaves_the_rest_alone(fast, change):
    assert fast.append(*fast_append(**change)) is None


def test_scratch_is_allocated_on_the_calls_stream(monkeypatch):
    """Memory of the current stream could still be in use by work queued there."""
    import contextlib
    import types
    active, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    fake = types.SimpleNamespace(cuda=types.SimpleNamespace(stream=on),
                                 empty=lambda n, dtype, device: made.append((n, active[-1])))
    monkeypatch.setattr(lib, "_torch", lambda: fake)
    q = types.SimpleNamespace(device="cuda:0")
    lib._scratch(64, q, "side")
    lib._scratch(32, q, None)
    assert made == [(64, "side"), (32, None)]


@pytest.mark.parametrize("source,kernel,variants,spilling,most", [
    ("attn_win_dec.cu", "attn_win_dec_kernel", 12, "Li128ELi4E", 450),  # 32 rows of 128 channels
    ("attn_q4_dec.cu", "attn_q4_dec_kernel", 12, "Li128ELi2E", 8),
    ("attn_win_tc.cu", "attn_win_tc_kernel", 8, "", 300),  # a few words of the roles' bookkeeping, none a row's scores
])
def test_serving_kernels_fit_their_registers(source, kernel, variants, spilling, most):
    """The library built in this tree: a toolchain that allocated otherwise would be slower, not wrong."""
    import os

    from paged_kv_cache_181_gb300 import build as b
    log = os.path.join(b.OUT_DIR, source + ".ptxas.txt")
    if not os.path.exists(log):
        pytest.skip(f"no ptxas report of {source} in this tree")
    with open(log) as f:
        got = b.spills(f.read(), kernel)
    assert len(got) == variants, got
    for name, st, ld in got:
        assert max(st, ld) <= (most if spilling in name else 0), (name, st, ld)
