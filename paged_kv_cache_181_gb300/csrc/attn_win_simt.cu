// Window/sinks attention on the CUDA cores, every type of pool: fp32 arithmetic throughout.
//
// One cluster = 32 packed query rows (attn_win.cuh) of one (sequence, kv head); its CTAs take the 32-key tiles in
// turn and merge at the end.  A CTA has 4 warps of 8 rows: scores with a lane per key (K rows padded by 16 bytes, so
// the lanes' float4 reads spread over the banks; Q rows are broadcast reads), an online softmax with the
// running maximum and sum in registers, then P.V with a lane per D/32 channels.  This is the path of fp32 calls
// (tensor cores have no fp32 product) and of PKV_FORCE_SIMT.

#include <atomic>

#include "attn_win.cuh"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kRows = 32;  // query rows per CTA
constexpr int kKeys = 32;  // keys per tile
constexpr int kWarpRows = kRows / 4;

struct PoolQ4 {};

template <int D>
struct Smem {
  float q[kRows][D];
  float k[kKeys][D + 4];
  float v[kKeys][D];
  float p[kRows][kKeys];
  float m[kRows], l[kRows];
};

// CH channels [c, c + CH) of key `slot` (pool row) of head kvh, as fp32.
template <typename T, int D, int CH>
struct Loader {
  static PKV_DEVINLINE void load(const void* pool, int64_t blk, int token, int Hkv, int kvh, int c, float (&x)[CH]) {
    const T* p = (const T*)pool + ((blk * 16 + token) * Hkv + kvh) * D + c;
    alignas(16) T v[CH];
    if constexpr (CH * sizeof(T) == 16)
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (CH * sizeof(T) == 8)
      *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
    else
      *reinterpret_cast<uint32_t*>(v) = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < CH; ++i) x[i] = pkv_to_f32<T>(v[i]);
  }
};
template <int D, int CH>
struct Loader<PoolQ4, D, CH> {
  static PKV_DEVINLINE void load(const void* pool, int64_t blk, int token, int Hkv, int kvh, int c, float (&x)[CH]) {
    const uint8_t* rec = (const uint8_t*)pool + (blk * Hkv + kvh) * Q4<D>::kRecord;
    const __half2 pair = *reinterpret_cast<const __half2*>(rec + Q4<D>::kPairs + (token * Q4<D>::kGroups + c / 32) * 4);
    const uint8_t* code = rec + token * Q4<D>::kRowBytes + c / 2;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int n = (code[i / 2] >> (4 * (i & 1))) & 15;
      x[i] = __half2float(__hfma(__int2half_rn(n), __low2half(pair), __high2half(pair)));
    }
  }
};

template <typename T, typename Pool, int D>
__global__ void __launch_bounds__(kThreads) attn_win_simt_kernel(const PkvWinArgs a) {
  constexpr int CH = D / 32;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.Hq / a.Hkv;
  const int64_t n_qt = ((int64_t)a.max_query_len * g + kRows - 1) / kRows;
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  int64_t item = blockIdx.x / n_cta;
  const int64_t qt = item % n_qt;
  item /= n_qt;
  const int kvh = (int)(item % a.Hkv), b = (int)(item / a.Hkv);
  const WinRow row = win_row(a, b, tid == 0 && qt == 0 && kvh == 0 && rank == 0);
  const int64_t total = (int64_t)row.Sq * g;
  if (qt * kRows >= total) return;  // the whole cluster leaves
  const int r0 = (int)(qt * kRows);
  const int rows = total - r0 < kRows ? (int)(total - r0) : kRows;
  const int base = row.L - row.Sq;
  const WinPages pg = win_pages(base + r0 / g, base + (r0 + rows - 1) / g, a.window, a.sinks);

  const float sl2 = a.scale * 1.4426950408889634f;
  for (int e = tid; e < kRows * D; e += kThreads) {
    const int r = e / D, c = e % D;
    float x = 0.f;
    if (r < rows) {
      const int64_t tok = (int64_t)row.q0 + (r0 + r) / g;
      x = pkv_to_f32<T>(((const T*)a.q)[(tok * a.Hq + kvh * g + (r0 + r) % g) * D + c]);
    }
    sm.q[r][c] = x;
  }
  float m[kWarpRows], l[kWarpRows], o[kWarpRows][CH] = {};
#pragma unroll
  for (int i = 0; i < kWarpRows; ++i) m[i] = -INFINITY, l[i] = 0.f;

  const int n_tiles = (pg.n + 1) / 2;
  for (int kt = rank; kt < n_tiles; kt += n_cta) {
    __syncthreads();  // the previous tile is used up (and Q is in place)
    for (int i = warp; i < kKeys; i += 4) {
      const int v = 2 * kt + (i >> 4);
      const int j = v < pg.n ? pg.page(v) * 16 + (i & 15) : 0;
      float x[CH] = {}, y[CH] = {};
      if (v < pg.n && pg.any(j)) {  // unseen keys stay zero: 0 * NaN would not
        const int64_t blk = win_block(a, b, j >> 4);
        Loader<Pool, D, CH>::load(a.k_pool, blk, i & 15, a.Hkv, kvh, lane * CH, x);
        Loader<Pool, D, CH>::load(a.v_pool, blk, i & 15, a.Hkv, kvh, lane * CH, y);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) sm.k[i][lane * CH + c] = x[c], sm.v[i][lane * CH + c] = y[c];
    }
    __syncthreads();
    float s[kWarpRows] = {};
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 kk = *reinterpret_cast<const float4*>(&sm.k[lane][c]);
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(&sm.q[warp * kWarpRows + i][c]);
        s[i] = fmaf(q.x, kk.x, fmaf(q.y, kk.y, fmaf(q.z, kk.z, fmaf(q.w, kk.w, s[i]))));
      }
    }
    const int v = 2 * kt + (lane >> 4);
    const int j = v < pg.n ? pg.page(v) * 16 + (lane & 15) : 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
      const int r = warp * kWarpRows + i;
      const int p = base + (r0 + r) / g;
      const bool seen = r < rows && win_sees(p, j, a.window, a.sinks);
      const float x = seen ? s[i] * sl2 : -INFINITY;
      float top = x;
#pragma unroll
      for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float m_new = fmaxf(m[i], top);
      const float mu = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = m[i] == m_new ? 1.f : ptx::ex2(m[i] - mu);
      const float e = seen ? ptx::ex2(x - mu) : 0.f;
      float sum = e;
#pragma unroll
      for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      l[i] = l[i] * alpha + sum;
      m[i] = m_new;
#pragma unroll
      for (int c = 0; c < CH; ++c) o[i][c] *= alpha;
      sm.p[r][lane] = e;
    }
    __syncwarp();
#pragma unroll 4
    for (int k = 0; k < kKeys; ++k) {
      float vv[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) vv[c] = sm.v[k][lane * CH + c];
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i) {
        const float p = sm.p[warp * kWarpRows + i][k];
#pragma unroll
        for (int c = 0; c < CH; ++c) o[i][c] = fmaf(p, vv[c], o[i][c]);
      }
    }
  }
  __syncthreads();
  float* so = &sm.v[0][0];  // [kRows][D]: kRows == kKeys
#pragma unroll
  for (int i = 0; i < kWarpRows; ++i) {
    const int r = warp * kWarpRows + i;
#pragma unroll
    for (int c = 0; c < CH; ++c) so[r * D + lane * CH + c] = o[i][c];
    if (lane == 0) sm.m[r] = m[i], sm.l[r] = l[i];
  }
  win_merge_store<T, D>(so, D, sm.m, sm.l, rows, r0, g, kvh, a.Hq, row.q0, (T*)a.out, tid, kThreads);
}

template <typename T, typename Pool, int D>
int launch(const PkvWinArgs& a, cudaStream_t s) {
  auto kernel = attn_win_simt_kernel<T, Pool, D>;
  const size_t smem = sizeof(Smem<D>);
  static PkvKernelState state;
  const int rc = pkv_prepare_kernel((const void*)kernel, (int)smem, kThreads, 0, state);
  if (rc) return rc;
  const int g = a.Hq / a.Hkv;
  const int64_t items = (int64_t)a.B * a.Hkv * (((int64_t)a.max_query_len * g + kRows - 1) / kRows);
  const int ctas = pkv_plan_cluster(state, items, pkv_visible_keys(a, kRows / g + 1) / kKeys + 1, 2.0);
  void* args[] = {const_cast<PkvWinArgs*>(&a)};
  return pkv_launch_cluster((const void*)kernel, items, ctas, kThreads, smem, args, false, s);
}

template <typename T, typename Pool>
int launch_d(const PkvWinArgs& a, int D, cudaStream_t s) {
  return D == 64 ? launch<T, Pool, 64>(a, s) : launch<T, Pool, 128>(a, s);
}

}  // namespace

int pkv_launch_win_simt(const PkvWinArgs& a, pkv_dtype dt, int D, bool q4, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  switch (dt) {
    case PKV_F32: return q4 ? launch_d<float, PoolQ4>(a, D, s) : launch_d<float, float>(a, D, s);
    case PKV_BF16:
      return q4 ? launch_d<__nv_bfloat16, PoolQ4>(a, D, s) : launch_d<__nv_bfloat16, __nv_bfloat16>(a, D, s);
    case PKV_F16: return q4 ? launch_d<__half, PoolQ4>(a, D, s) : launch_d<__half, __half>(a, D, s);
  }
  return (int)cudaErrorInvalidValue;
}
