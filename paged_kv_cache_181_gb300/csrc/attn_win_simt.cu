// Window/sinks attention on the CUDA cores, every type of pool: fp32 arithmetic throughout.
//
// One cluster = a tile of packed query rows (attn_win.cuh) of one (sequence, kv head); its CTAs take the keys in turn and
// merge at the end.  This is the path of fp32 calls (tensor cores have no fp32 product) and of PKV_FORCE_SIMT.
//
// Tiles of 32 rows: a CTA's 4 warps have 8 rows each and share tiles of 32 keys in shared memory.  Scores with a lane
// per key (K rows padded by 16 bytes, so the lanes' float4 reads spread over the banks; Q rows are broadcast reads), an
// online softmax with the running maximum and sum in registers, then P.V with a lane per D/32 channels.  16 warps an SM
// hide what each waits for; tiles of 64 keys, two a lane, and register tiles of 8 x 4 scores need fewer reads for an FMA
// but leave 8 warps, and measured slower (3 sequences, 333 queries, window 501: 72 and 90 us instead of 50).

// Calls of at most 8 rows (decode): bound by memory, so keys and values go from memory to registers.  Half a warp
// takes a key, a lane D/16 of its channels for every row; four keys at a time, whose scores are summed over the half
// warp by four shuffles each; each half warp has a softmax state of its own until the end.

#include <atomic>

#include "attn_win.cuh"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kWarpRows = 8;  // query rows of a warp
constexpr int kRows = kWarps * kWarpRows, kKeys = 32;  // of a CTA's tile

struct PoolQ4 {};

template <int D>
struct Smem {
  float q[kRows][D];
  float k[kKeys][D + 4];
  float v[kKeys][D];  // at the end, the rows' sums
  float p[kRows][kKeys];
  float m[kRows], l[kRows];
};

template <int D>
struct FewSmem {
  static constexpr int kStates = 2 * kWarps;  // a half warp's each
  static constexpr int kStride = D + 4;
  float o[kStates][kWarpRows][kStride];
  float wm[kStates][kWarpRows], wl[kStates][kWarpRows];
  float m[kWarpRows], l[kWarpRows];
};

// CH channels [c, c + CH) of key `slot` (pool row) of head kvh, as fp32.
template <typename T, int D, int CH>
struct Loader {
  static PKV_DEVINLINE void load(const void* pool, int64_t blk, int token, int Hkv, int kvh, int c, float (&x)[CH]) {
    const T* p = (const T*)pool + ((blk * 16 + token) * Hkv + kvh) * D + c;
    alignas(16) T v[CH];
    if constexpr (CH * sizeof(T) == 32)
      reinterpret_cast<uint4*>(v)[0] = reinterpret_cast<const uint4*>(p)[0],
      reinterpret_cast<uint4*>(v)[1] = reinterpret_cast<const uint4*>(p)[1];
    else if constexpr (CH * sizeof(T) == 16)
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
__global__ void __launch_bounds__(kThreads, 2) attn_win_simt_few_kernel(const PkvWinArgs a) {
  constexpr int CH = D / 16, U = 4;  // channels of a lane; keys of a half warp per step
  using S = FewSmem<D>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = lane >> 4, c0 = (lane & 15) * CH;
  const int g = a.Hq / a.Hkv;
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  const uint32_t item = blockIdx.x / n_cta;
  const int kvh = item % a.Hkv, b = item / a.Hkv;
  const WinRow row = win_row(a, b, tid == 0 && kvh == 0 && rank == 0);
  const int rows = row.Sq * g;
  if (rows <= 0) return;  // the whole cluster leaves
  const int base = row.L - row.Sq;
  const WinPages pg = win_pages(base, base + row.Sq - 1, a.window, a.sinks);
  const float sl2 = a.scale * 1.4426950408889634f;
  float q[kWarpRows][CH], o[kWarpRows][CH] = {}, m[kWarpRows], l[kWarpRows] = {};
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) {
    m[r] = -INFINITY;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      q[r][c] = 0.f;
      if (r < rows)
        q[r][c] = pkv_to_f32<T>(((const T*)a.q)[(((int64_t)row.q0 + r / g) * a.Hq + kvh * g + r % g) * D + c0 + c]) * sl2;
    }
  }
  // A warp's step is half a page: keys 8 h .. 8 h + 7, four of them for each half warp.
  for (int w = rank * kWarps + warp; w < 2 * pg.n; w += n_cta * kWarps) {
    const int page = pg.page(w >> 1), j0 = page * 16 + (w & 1) * 8 + half * U;
    const int64_t blk = win_block(a, b, page);
    float k[U][CH], v[U][CH];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int c = 0; c < CH; ++c) k[u][c] = v[u][c] = 0.f;
      if (pg.any(j0 + u)) {
        Loader<Pool, D, CH>::load(a.k_pool, blk, (j0 + u) & 15, a.Hkv, kvh, c0, k[u]);
        Loader<Pool, D, CH>::load(a.v_pool, blk, (j0 + u) & 15, a.Hkv, kvh, c0, v[u]);
      }
    }
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      if (r >= rows) break;
      const int p = base + r / g;
      float x[U], top = -INFINITY;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) x[u] = fmaf(q[r][c], k[u][c], x[u]);
      }
#pragma unroll
      for (int d = 8; d; d >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] += __shfl_xor_sync(0xffffffffu, x[u], d);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!win_sees(p, j0 + u, a.window, a.sinks)) x[u] = -INFINITY;
        top = fmaxf(top, x[u]);
      }
      if (top > m[r]) {
        const float alpha = ptx::ex2(m[r] - top);  // 0 from -inf
        m[r] = top;
        l[r] *= alpha;
#pragma unroll
        for (int c = 0; c < CH; ++c) o[r][c] *= alpha;
      }
      const float mu = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float e = ptx::ex2(x[u] - mu);
        l[r] += e;
#pragma unroll
        for (int c = 0; c < CH; ++c) o[r][c] = fmaf(e, v[u][c], o[r][c]);
      }
    }
  }
  const int state = warp * 2 + half;
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) {
#pragma unroll
    for (int c = 0; c < CH; ++c) sm.o[state][r][c0 + c] = o[r][c];
    if ((lane & 15) == 0) sm.wm[state][r] = m[r], sm.wl[state][r] = l[r];
  }
  __syncthreads();
  for (int e = tid; e < rows * D; e += kThreads) {
    const int r = e / D, c = e % D;
    float top = -INFINITY, acc = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < S::kStates; ++w) top = fmaxf(top, sm.wm[w][r]);
#pragma unroll
    for (int w = 0; w < S::kStates; ++w) {
      const float f = sm.wm[w][r] == top ? 1.f : ptx::ex2(sm.wm[w][r] - top);
      acc += f * sm.o[w][r][c];
      sum += f * sm.wl[w][r];
    }
    sm.o[0][r][c] = acc;  // read and written by this thread alone
    if (c == 0) sm.m[r] = top, sm.l[r] = sum;
  }
  win_merge_store<T, D>(&sm.o[0][0][0], S::kStride, sm.m, sm.l, rows, 0, g, kvh, a.Hq, row.q0, (T*)a.out, tid, kThreads);
}

template <typename Kernel>
int launch(Kernel kernel, PkvKernelState& state, size_t smem, int64_t items, int64_t steps, double rate,
           double setup, const PkvWinArgs& a, cudaStream_t s) {
  const int rc = pkv_prepare_kernel((const void*)kernel, (int)smem, kThreads, 0, state);
  if (rc) return rc;
  const int ctas = pkv_plan_cluster(state, items, steps, rate, setup);
  void* args[] = {const_cast<PkvWinArgs*>(&a)};
  return pkv_launch_cluster((const void*)kernel, items, ctas, kThreads, smem, args, false, s);
}

template <typename T, typename Pool, int D>
int launch_rows(const PkvWinArgs& a, cudaStream_t s) {
  const int g = a.Hq / a.Hkv;
  const int64_t rows = (int64_t)a.max_query_len * g;
  if (rows <= kWarpRows) {
    static PkvKernelState state;
    const int64_t keys = pkv_visible_keys(a, a.max_query_len);
    return launch(attn_win_simt_few_kernel<T, Pool, D>, state, sizeof(FewSmem<D>), (int64_t)a.B * a.Hkv,
                  keys / (8 * kWarps) + 1, 0.4, 4.7, a, s);
  }
  static PkvKernelState state;
  return launch(attn_win_simt_kernel<T, Pool, D>, state, sizeof(Smem<D>), (int64_t)a.B * a.Hkv * ((rows + kRows - 1) / kRows),
                pkv_visible_keys(a, kRows / g + 1) / kKeys + 1, 0.25, 0.4, a, s);
}

template <typename T, typename Pool>
int launch_d(const PkvWinArgs& a, int D, cudaStream_t s) {
  return D == 64 ? launch_rows<T, Pool, 64>(a, s) : launch_rows<T, Pool, 128>(a, s);
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
