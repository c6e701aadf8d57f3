// Rotary append: q_out = rot(q), pool[slot] = rot(k), pool[slot] = v, into 16-bit/fp32 pools or, quantised on the
// way, into 4-bit records; and the read-back of 4-bit blocks into staging buffers.
//
// All three are bound by memory: the append reads (Hq + 2 Hkv) D values a token and writes as many (Q and K rotated,
// V as it is), with about one operation per byte.  8192 tokens, 40 heads over 8 kv heads, D = 128, bf16: 38.6 us, 91 %
// of the measured copy bandwidth; into 4-bit records and read back from them 50.2 us, 76 %; one token 2.7 us, a launch.
//
// A thread takes two vectors of 8 channels that the rotation pairs (rot_dim/2 apart) or, where it does not, two
// others, and keeps their cosines and sines in registers while it walks over the heads of its token, loading four
// heads' vectors (4-bit pools: two, and the next two meanwhile) before it uses the first.  In fp32: two products and one sum, each rounded, so that results do not
// depend on how a compiler contracts them.
//
// 4-bit pools: the four lanes that hold a group of 32 channels in one of their two vectors find its range with two
// shuffles each.  The pairs of vectors keep groups on four neighbouring lanes for every rot_dim that is a multiple of
// 64; any other takes a kernel with one vector a thread, which loads its partner's vector as well.

#include "q4.cuh"

namespace {

constexpr int kThreads = 256;

template <typename T>
PKV_DEVINLINE void load8(const T* p, float (&x)[8]);
template <>
PKV_DEVINLINE void load8<float>(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <typename T>
PKV_DEVINLINE void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = pkv_to_f32<T>(reinterpret_cast<const T*>(&w[i])[0]);
    x[2 * i + 1] = pkv_to_f32<T>(reinterpret_cast<const T*>(&w[i])[1]);
  }
}
template <>
PKV_DEVINLINE void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  unpack8<__nv_bfloat16>(*reinterpret_cast<const uint4*>(p), x);
}
template <>
PKV_DEVINLINE void load8<__half>(const __half* p, float (&x)[8]) {
  unpack8<__half>(*reinterpret_cast<const uint4*>(p), x);
}

template <typename T>
PKV_DEVINLINE void store8(T* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    reinterpret_cast<T*>(&w[i])[0] = pkv_from_f32<T>(x[2 * i]);
    reinterpret_cast<T*>(&w[i])[1] = pkv_from_f32<T>(x[2 * i + 1]);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
PKV_DEVINLINE void store8<float>(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Quantise the group of 32 channels that four neighbouring lanes hold (8 each) and store the lane's code word
// and, by the group's first lane, the pair.  `mask`: the warp's lanes that came here, whole groups of four.
template <int D>
PKV_DEVINLINE void store_q4(unsigned mask, uint8_t* record, int token, int vec, float (&x)[8]) {
  float lo = x[0], hi = x[0], fine = 0.f;  // fine: 0, or NaN when a value is not finite
#pragma unroll
  for (int i = 0; i < 8; ++i) fine = fmaf(x[i], 0.f, fine);
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
  for (int m = 1; m < 4; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, m));
    fine += __shfl_xor_sync(mask, fine, m);
  }
  if (lo < -32768.f || hi > 32768.f) {  // the four lanes agree
    lo = fminf(fmaxf(lo, -32768.f), 32768.f), hi = fminf(fmaxf(hi, -32768.f), 32768.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -32768.f), 32768.f);
  }
  const __half low = __float2half_rn(lo);
  const __half step = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), (float)(1.0 / 15.0)));
  const float lowf = __half2float(low), stepf = __half2float(step);
  const float inv = stepf == 0.f ? 0.f : __frcp_rn(stepf);
  // Adding 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the low bits of 0x4b400000 + n; what those
  // constants add up to over the eight nibbles is taken off at the end.
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float n = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], lowf), inv), 0.f), 15.f);
    w = w * 16u + __float_as_uint(__fadd_rn(n, 12582912.f));
  }
  w -= 0x4b400000u * 0x11111111u;
  *reinterpret_cast<uint32_t*>(record + token * Q4<D>::kRowBytes + vec * 4) = w;
  if ((vec & 3) == 0) {
    const __half nan = __ushort_as_half(0x7fff);
    *reinterpret_cast<__half2*>(record + Q4<D>::kPairs + (token * Q4<D>::kGroups + (vec >> 2)) * 4) =
        fine == 0.f ? __halves2half2(step, low) : __halves2half2(nan, nan);
  }
}

// A vector of 8 channels as it lies in memory.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
  PKV_DEVINLINE void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  PKV_DEVINLINE void get(float (&x)[8]) const {
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = pkv_to_f32<T>(e[i]);
  }
};

// Block: one token; of its HG groups of D/16 threads each walks every HG-th head.
// Heads that a thread loads at once (NH), whether it loads the next ones before it works on these (AHEAD), and threads an
// SM, measured at 8192 tokens, 40/8 heads.  16-bit pools: 4 heads, 704 threads 38.6 us (640: 42.0, 768: 39.5, 896: 45.5;
// 2 heads 40.7, ahead 39.1).  4-bit ones, which compute longer, with their read-back: 2 heads ahead, 832 threads 50.4 us (not
// ahead 52.8, 4 heads 55.7).
template <typename T, int D, bool Q4POOL, int HG>
__global__ void __launch_bounds__(D / 16 * HG, sizeof(T) == 2 && HG == 8 ? (Q4POOL ? 832 : 704) / (D / 16 * HG) : 0)
    append_pairs_kernel(const PkvAppendArgs a) {
  constexpr bool AHEAD = Q4POOL && HG == 8;
  constexpr int U = D / 16, NH = sizeof(T) == 4 || AHEAD ? 2 : 4;
  const int64_t t = blockIdx.x;
  const int u = threadIdx.x % U, hg = threadIdx.x / U;
  const int64_t slot = a.slots[t];
  const int heads = a.Hq + 2 * a.Hkv, half = a.rot_dim / 2;
  int64_t pos = 0;
  if (a.rot_dim) {
    pos = a.positions[t];
    if (a.check && (pos < 0 || pos >= a.max_position)) {
      if (u == 0 && hg == 0) pkv_raise(a.err, PKV_DEVERR_POSITION);
      return;
    }
  }
  int stop = heads;  // a token without a slot has Q heads only
  if (slot < 0) stop = a.Hq;
  if (a.check && slot >= a.num_slots) {
    if (u == 0 && hg == 0) pkv_raise(a.err, PKV_DEVERR_SLOT);
    stop = a.Hq;
  }
  // The thread's vectors, v0 and v1, of rotated heads (Q, K), and w0, w1 of V heads.
  const int w0 = Q4POOL || a.interleaved ? (u & ~3) * 2 + (u & 3) : 2 * u, w1 = Q4POOL || a.interleaved ? w0 + 4 : w0 + 1;
  int v0 = w0, v1 = w1;
  const bool paired = !a.interleaved && u < a.rot_dim / 16;
  if (!a.interleaved) {
    if (paired) {
      v0 = u, v1 = u + a.rot_dim / 16;
    } else {
      const int k = u - a.rot_dim / 16;  // behind the rotated channels
      v0 = a.rot_dim / 8 + (Q4POOL ? (k & ~3) * 2 + (k & 3) : 2 * k);
      v1 = v0 + (Q4POOL ? 4 : 1);
    }
  }
  float cc[8], ss[8];
  const float* row = a.cos_sin + pos * a.rot_dim;
  if (paired) {
    load8<float>(row + 8 * u, cc);
    load8<float>(row + half + 8 * u, ss);
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float4 c = make_float4(1.f, 1.f, 1.f, 1.f), z = make_float4(0.f, 0.f, 0.f, 0.f);
      const int v = k ? v1 : v0;
      if (a.interleaved && 8 * v < a.rot_dim) {
        c = *reinterpret_cast<const float4*>(row + 4 * v);
        z = *reinterpret_cast<const float4*>(row + half + 4 * v);
      }
      cc[4 * k] = c.x, cc[4 * k + 1] = c.y, cc[4 * k + 2] = c.z, cc[4 * k + 3] = c.w;
      ss[4 * k] = z.x, ss[4 * k + 1] = z.y, ss[4 * k + 2] = z.z, ss[4 * k + 3] = z.w;
    }
  }
  const bool turn0 = a.interleaved && 8 * v0 < a.rot_dim, turn1 = a.interleaved && 8 * v1 < a.rot_dim;
  const T* const q = (const T*)a.q + t * a.q_stride;
  const T* const k = (const T*)a.k + t * a.k_stride;
  const T* const v = (const T*)a.v + t * a.v_stride;
  Raw<T> r0[NH], r1[NH];
  auto fetch = [&](int h0, Raw<T>(&to0)[NH], Raw<T>(&to1)[NH]) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int h = h0 + i * HG;
      if (h < stop) {
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        const T* src = is_q ? q + (int64_t)h * D : is_v ? v + (int64_t)(h - a.Hq - a.Hkv) * D : k + (int64_t)(h - a.Hq) * D;
        to0[i].load(src + 8 * (is_v ? w0 : v0));
        to1[i].load(src + 8 * (is_v ? w1 : v1));
      }
    }
  };
  if (AHEAD) fetch(hg, r0, r1);
  for (int h0 = hg; h0 < stop; h0 += NH * HG) {
    Raw<T> n0[NH], n1[NH];
    if (AHEAD)
      fetch(h0 + NH * HG, n0, n1);
    else
      fetch(h0, r0, r1);
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int h = h0 + i * HG;
      if (h >= stop) break;
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      float x[8], y[8];
      r0[i].get(x);
      r1[i].get(y);
      if (!is_v) {
        if (paired) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xe = x[e];
            x[e] = __fsub_rn(__fmul_rn(xe, cc[e]), __fmul_rn(y[e], ss[e]));
            y[e] = __fadd_rn(__fmul_rn(y[e], cc[e]), __fmul_rn(xe, ss[e]));
          }
        } else if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float xa = x[2 * e], xb = x[2 * e + 1], ya = y[2 * e], yb = y[2 * e + 1];
            if (turn0) {
              x[2 * e] = __fsub_rn(__fmul_rn(xa, cc[e]), __fmul_rn(xb, ss[e]));
              x[2 * e + 1] = __fadd_rn(__fmul_rn(xb, cc[e]), __fmul_rn(xa, ss[e]));
            }
            if (turn1) {
              y[2 * e] = __fsub_rn(__fmul_rn(ya, cc[4 + e]), __fmul_rn(yb, ss[4 + e]));
              y[2 * e + 1] = __fadd_rn(__fmul_rn(yb, cc[4 + e]), __fmul_rn(ya, ss[4 + e]));
            }
          }
        }
      }
      const int o0 = is_v ? w0 : v0, o1 = is_v ? w1 : v1;
      if (Q4POOL && !is_q) {
        const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
        uint8_t* record = (uint8_t*)(is_v ? a.v_pool : a.k_pool) + ((slot >> 4) * a.Hkv + hk) * Q4<D>::kRecord;
        const unsigned mask = 0xfu << (threadIdx.x & 28);  // the four lanes of a group share its head
        store_q4<D>(mask, record, (int)(slot & 15), o0, x);
        store_q4<D>(mask, record, (int)(slot & 15), o1, y);
      } else {
        T* dst = is_q ? (T*)a.q_out + (t * a.Hq + h) * D
                      : (T*)(is_v ? a.v_pool : a.k_pool) + (slot * a.Hkv + (is_v ? h - a.Hq - a.Hkv : h - a.Hq)) * D;
        store8<T>(dst + 8 * o0, x);
        store8<T>(dst + 8 * o1, y);
      }
    }
    if (AHEAD) {
#pragma unroll
      for (int i = 0; i < NH; ++i) r0[i] = n0[i], r1[i] = n1[i];
    }
  }
}

// One vector a thread: 4-bit pools with a rot_dim that splits groups over more than four lanes.
// Grid: x = token, y = groups of kThreads / (D/8) heads (Q heads, then K, then V).
template <typename T, int D, bool Q4POOL>
__global__ void __launch_bounds__(kThreads) append_kernel(const PkvAppendArgs a) {
  constexpr int VECS = D / 8;
  const int64_t t = blockIdx.x;
  const int vec = threadIdx.x % VECS;
  const int h = blockIdx.y * (kThreads / VECS) + threadIdx.x / VECS;
  const int heads = a.Hq + 2 * a.Hkv;
  const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
  const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
  bool live = h < heads;  // lanes past the last head keep the warp whole for the shuffles below
  const int64_t slot = a.slots[t];
  int64_t pos = 0;
  if (a.rot_dim) {
    pos = a.positions[t];
    if (a.check && (pos < 0 || pos >= a.max_position)) {
      if (threadIdx.x == 0 && blockIdx.y == 0) pkv_raise(a.err, PKV_DEVERR_POSITION);
      live = false;
      pos = 0;
    }
  }
  if (live && !is_q) {
    live = slot >= 0;
    if (a.check && slot >= a.num_slots) {
      if (vec == 0 && hk == 0 && !is_v) pkv_raise(a.err, PKV_DEVERR_SLOT);
      live = false;
    }
  }
  float x[8] = {};
  if (live) {
    const T* src = is_q ? (const T*)a.q + t * a.q_stride + (int64_t)h * D
                        : (is_v ? (const T*)a.v + t * a.v_stride : (const T*)a.k + t * a.k_stride) + (int64_t)hk * D;
    const int c = vec * 8;
    load8<T>(src + c, x);
    if (!is_v && c < a.rot_dim) {
      const float* row = a.cos_sin + pos * a.rot_dim;
      const int half = a.rot_dim / 2;
      if (a.interleaved) {
        const float4 cs = *reinterpret_cast<const float4*>(row + c / 2);
        const float4 sn = *reinterpret_cast<const float4*>(row + half + c / 2);
        const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = x[2 * i], w = x[2 * i + 1];
          x[2 * i] = __fsub_rn(__fmul_rn(u, cc[i]), __fmul_rn(w, ss[i]));
          x[2 * i + 1] = __fadd_rn(__fmul_rn(w, cc[i]), __fmul_rn(u, ss[i]));
        }
      } else {
        const bool second = c >= half;
        const int i0 = second ? c - half : c;
        float y[8], cc[8], ss[8];
        load8<T>(src + (second ? c - half : c + half), y);
        load8<float>(row + i0, cc);
        load8<float>(row + half + i0, ss);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = __fmul_rn(x[i], cc[i]), r = __fmul_rn(y[i], ss[i]);
          x[i] = second ? __fadd_rn(p, r) : __fsub_rn(p, r);
        }
      }
    }
  }
  __syncwarp();  // q_out may be q: every lane of the head has read before any stores
  if (is_q) {
    if (live) store8<T>((T*)a.q_out + (t * a.Hq + h) * D + vec * 8, x);
  } else if (!Q4POOL) {
    if (live) store8<T>((T*)(is_v ? a.v_pool : a.k_pool) + (slot * a.Hkv + hk) * D + vec * 8, x);
  }
  if (Q4POOL) {
    const bool keep = live && !is_q;
    uint8_t* record = (uint8_t*)(is_v ? a.v_pool : a.k_pool) + ((slot >> 4) * a.Hkv + hk) * Q4<D>::kRecord;
    // a head's lanes agree on `keep`, and a group's four lanes are of one head
    const unsigned mask = __ballot_sync(0xffffffffu, keep);
    if (keep) store_q4<D>(mask, record, (int)(slot & 15), vec, x);
  }
}

// stage[b][first*16 + i] = the values of token i of the listed blocks.  Grid: x = listed block, y = (row, K|V); a thread
// takes 8 channels at a time, several in flight, in the order of the staging rows.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    gather_q4_kernel(const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp, int64_t num_blocks,
                     const int32_t* __restrict__ table, int W, int first_block, T* __restrict__ sk, T* __restrict__ sv,
                     int64_t stage_rows, int Hkv, unsigned int* err, int check) {
  constexpr int VECS = D / 8, NU = 4;
  const int b = blockIdx.y >> 1, page = first_block + blockIdx.x;
  const bool is_v = blockIdx.y & 1;
  const int blk = __ldg(table + (int64_t)b * W + page);
  if (check && (blk < 0 || blk >= num_blocks)) {
    if (threadIdx.x == 0) pkv_raise(err, PKV_DEVERR_BLOCK);
    return;
  }
  const uint8_t* recs = (is_v ? vp : kp) + (int64_t)blk * Hkv * Q4<D>::kRecord;
  T* dst = (is_v ? sv : sk) + (b * stage_rows + (int64_t)page * 16) * Hkv * D;
  const int per_token = Hkv * VECS, n = 16 * per_token;
  for (int e0 = threadIdx.x; e0 < n; e0 += NU * kThreads) {
    uint32_t w[NU];
    __half2 pair[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int e = e0 + i * kThreads;
      if (e < n) {
        const int token = e / per_token, r = e - token * per_token, h = r / VECS, vec = r % VECS;
        const uint8_t* rec = recs + (int64_t)h * Q4<D>::kRecord;
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(rec + token * Q4<D>::kRowBytes) + vec);
        pair[i] = __ldg(reinterpret_cast<const __half2*>(rec + Q4<D>::kPairs) + token * Q4<D>::kGroups + (vec >> 2));
      }
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int e = e0 + i * kThreads;
      if (e < n) {
        __half2 hv[4];
        q4_values(w[i], pair[i], hv);
        float x[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = __low2float(hv[c]), x[c + 4] = __high2float(hv[c]);
        store8<T>(dst + (int64_t)e * 8, x);
      }
    }
  }
}

template <typename T, int D, bool Q4POOL>
int launch_append(const PkvAppendArgs& a, cudaStream_t s) {
  if (Q4POOL && !a.interleaved && a.rot_dim % 64) {
    constexpr int per = kThreads / (D / 8);
    const dim3 grid((unsigned)a.T, (unsigned)((a.Hq + 2 * a.Hkv + per - 1) / per));
    append_kernel<T, D, Q4POOL><<<grid, kThreads, 0, s>>>(a);
    return (int)cudaGetLastError();
  }
  // Few tokens of many heads: enough threads that each has at most four heads, whose loads it issues at once.  Else 8
  // groups, so that a thread's cosines and sines serve more heads.  A block per token either way: several tokens a
  // block measured 3 % slower at 8192 tokens.
  if (a.T < 1024 && a.Hq + 2 * a.Hkv > 32)
    append_pairs_kernel<T, D, Q4POOL, 16><<<(unsigned)a.T, D, 0, s>>>(a);
  else
    append_pairs_kernel<T, D, Q4POOL, 8><<<(unsigned)a.T, D / 2, 0, s>>>(a);
  return (int)cudaGetLastError();
}

template <typename T>
int launch_append_t(const PkvAppendArgs& a, bool q4, cudaStream_t s) {
  if (q4) return a.D == 64 ? launch_append<T, 64, true>(a, s) : launch_append<T, 128, true>(a, s);
  return a.D == 64 ? launch_append<T, 64, false>(a, s) : launch_append<T, 128, false>(a, s);
}

}  // namespace

int pkv_launch_append(const PkvAppendArgs& a, pkv_dtype dt, bool q4, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  switch (dt) {
    case PKV_F32: return launch_append_t<float>(a, q4, s);
    case PKV_BF16: return launch_append_t<__nv_bfloat16>(a, q4, s);
    case PKV_F16: return launch_append_t<__half>(a, q4, s);
  }
  return (int)cudaErrorInvalidValue;
}

namespace {
template <typename T, int D>
int launch_gather(const void* kp, const void* vp, int64_t num_blocks, const int32_t* table, int B, int W,
                  int first_block, int n_blocks, void* sk, void* sv, int64_t stage_rows, int Hkv, unsigned int* err,
                  int check, cudaStream_t s) {
  for (int b0 = 0; b0 < B; b0 += 32767) {  // a grid's y extent
    const int nb = B - b0 < 32767 ? B - b0 : 32767;
    const int64_t at = (int64_t)b0 * stage_rows * Hkv * D;
    gather_q4_kernel<T, D><<<dim3((unsigned)n_blocks, (unsigned)(2 * nb)), kThreads, 0, s>>>(
        (const uint8_t*)kp, (const uint8_t*)vp, num_blocks, table + (int64_t)b0 * W, W, first_block, (T*)sk + at,
        (T*)sv + at, stage_rows, Hkv, err, check);
  }
  return (int)cudaGetLastError();
}
}  // namespace

int pkv_launch_gather_q4(const void* kp, const void* vp, int64_t num_blocks, const int32_t* table, int B, int W,
                         int first_block, int n_blocks, void* sk, void* sv, int64_t stage_rows, int Hkv, int D,
                         pkv_dtype dt, unsigned int* err, int check, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
#define PKV_GATHER(T)                                                                                               \
  (D == 64 ? launch_gather<T, 64>(kp, vp, num_blocks, table, B, W, first_block, n_blocks, sk, sv, stage_rows, Hkv, \
                                  err, check, s)                                                                    \
           : launch_gather<T, 128>(kp, vp, num_blocks, table, B, W, first_block, n_blocks, sk, sv, stage_rows, Hkv, \
                                   err, check, s))
  switch (dt) {
    case PKV_F32: return PKV_GATHER(float);
    case PKV_BF16: return PKV_GATHER(__nv_bfloat16);
    case PKV_F16: return PKV_GATHER(__half);
  }
#undef PKV_GATHER
  return (int)cudaErrorInvalidValue;
}
