// Rotary append: q_out = rot(q), pool[slot] = rot(k), pool[slot] = v, into 16-bit/fp32 pools or, quantised on the
// way, into 4-bit records; and the read-back of 4-bit blocks into staging buffers.
//
// All three are bound by memory: the append reads (Hq + 2 Hkv) D values a token and writes as many (Q and K rotated,
// V as it is), with about one operation per byte.
//
// One thread produces one vector of 8 channels of one head.  A rotated channel needs its partner (rot_dim/2 away,
// or its neighbour): the thread loads both vectors; the partner's bytes are another lane's own, in the same warp
// (a head is D/8 = 8 or 16 lanes), so they come from L1.  In fp32: two products and one sum, each rounded, so that
// results do not depend on how a compiler contracts them.

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
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    fine = fine && fabsf(x[i]) <= 3.402823466e38f;
    x[i] = fminf(fmaxf(x[i], -32768.f), 32768.f);
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
  for (int m = 1; m < 4; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, m));
    fine = __shfl_xor_sync(mask, fine ? 1 : 0, m) && fine;
  }
  const __half low = __float2half_rn(lo);
  const __half step = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), (float)(1.0 / 15.0)));
  const float lowf = __half2float(low), stepf = __half2float(step);
  const float inv = stepf == 0.f ? 0.f : __frcp_rn(stepf);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(x[i], lowf), inv)), 0.f), 15.f);
    w |= (uint32_t)n << (4 * i);
  }
  uint8_t* codes = record + token * Q4<D>::kRowBytes + vec * 4;
  *reinterpret_cast<uint32_t*>(codes) = w;
  if ((vec & 3) == 0) {
    const __half nan = __ushort_as_half(0x7fff);
    *reinterpret_cast<__half2*>(record + Q4<D>::kPairs + (token * Q4<D>::kGroups + (vec >> 2)) * 4) =
        fine ? __halves2half2(step, low) : __halves2half2(nan, nan);
  }
}

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

// stage[b][first*16 + i] = the values of token i of the listed blocks.  One thread per 8 channels.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    gather_q4_kernel(const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp, int64_t num_blocks,
                     const int32_t* __restrict__ table, int W, int first_block, int n_blocks, T* __restrict__ sk,
                     T* __restrict__ sv, int64_t stage_rows, int Hkv, int64_t n, unsigned int* err, int check) {
  constexpr int VECS = D / 8;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < n; u += (int64_t)gridDim.x * kThreads) {
    const int vec = (int)(u % VECS);
    int64_t r = u / VECS;
    const int h = (int)(r % Hkv);
    r /= Hkv;
    const int token = (int)(r & 15);
    r >>= 4;
    const int page = (int)(r % n_blocks);
    r /= n_blocks;
    const bool is_v = r & 1;
    const int64_t b = r >> 1;
    const int blk = __ldg(table + b * W + first_block + page);
    if (check && (blk < 0 || blk >= num_blocks)) {
      if (token == 0 && vec == 0 && h == 0) pkv_raise(err, PKV_DEVERR_BLOCK);
      continue;
    }
    const uint8_t* rec = (is_v ? vp : kp) + ((int64_t)blk * Hkv + h) * Q4<D>::kRecord;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(rec + token * Q4<D>::kRowBytes) + vec);
    const __half2 pair = __ldg(reinterpret_cast<const __half2*>(rec + Q4<D>::kPairs) + token * Q4<D>::kGroups + (vec >> 2));
    __half2 hv[4];
    q4_values(w, pair, hv);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __low2float(hv[i]), x[i + 4] = __high2float(hv[i]);
    const int64_t row = b * stage_rows + (int64_t)(first_block + page) * 16 + token;
    store8<T>((is_v ? sv : sk) + (row * Hkv + h) * D + vec * 8, x);
  }
}

template <typename T, int D>
int launch_append(const PkvAppendArgs& a, bool q4, cudaStream_t s) {
  constexpr int per = kThreads / (D / 8);
  const dim3 grid((unsigned)a.T, (unsigned)((a.Hq + 2 * a.Hkv + per - 1) / per));
  if (q4)
    append_kernel<T, D, true><<<grid, kThreads, 0, s>>>(a);
  else
    append_kernel<T, D, false><<<grid, kThreads, 0, s>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace

int pkv_launch_append(const PkvAppendArgs& a, pkv_dtype dt, bool q4, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  switch (dt) {
    case PKV_F32: return a.D == 64 ? launch_append<float, 64>(a, q4, s) : launch_append<float, 128>(a, q4, s);
    case PKV_BF16:
      return a.D == 64 ? launch_append<__nv_bfloat16, 64>(a, q4, s) : launch_append<__nv_bfloat16, 128>(a, q4, s);
    case PKV_F16: return a.D == 64 ? launch_append<__half, 64>(a, q4, s) : launch_append<__half, 128>(a, q4, s);
  }
  return (int)cudaErrorInvalidValue;
}

namespace {
template <typename T, int D>
int launch_gather(const void* kp, const void* vp, int64_t num_blocks, const int32_t* table, int B, int W,
                  int first_block, int n_blocks, void* sk, void* sv, int64_t stage_rows, int Hkv, unsigned int* err,
                  int check, cudaStream_t s) {
  int sms = pkv_sm_count();
  if (sms <= 0) sms = 152;
  const int64_t n = (int64_t)B * 2 * n_blocks * 16 * Hkv * (D / 8);
  int64_t grid = (n + kThreads - 1) / kThreads;
  if (grid > (int64_t)sms * 32) grid = (int64_t)sms * 32;
  gather_q4_kernel<T, D><<<(unsigned)grid, kThreads, 0, s>>>((const uint8_t*)kp, (const uint8_t*)vp, num_blocks, table,
                                                             W, first_block, n_blocks, (T*)sk, (T*)sv, stage_rows, Hkv,
                                                             n, err, check);
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
