// Shared by the decode kernels (few query rows per kv head; attn_win_dec.cu for 16-bit pools, attn_q4_dec.cu for 4-bit
// ones): operand primitives, the softmax state of a warp, the merge of warps, clusters and splits, and the launch.
#pragma once

#include <type_traits>

#include "attn_win.cuh"
#include "tc_ptx.cuh"

namespace dec {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kRescale = 8.f;  // log2 units
// What the combine launch has to gain, in steps (one page per warp): 3 us on the GPU, and 6.5 us of the host's time (a
// workspace, a launch), which a stream of short calls waits for.
constexpr double kCombineSteps = 8.0;

template <bool BF16>
PKV_DEVINLINE void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements spread over the warp (lane 4g + t holds row g, columns 2t, 2t+1).
PKV_DEVINLINE uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

PKV_DEVINLINE uint32_t low_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
PKV_DEVINLINE uint32_t high_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

template <bool BF16>
PKV_DEVINLINE uint32_t pack(float lo, float hi) {
  return BF16 ? ptx::pack_bf16x2(lo, hi) : ptx::pack_f16x2(lo, hi);
}

// Where a CTA stands: its tile of 8 NT packed query rows, and its share of the tile's pages.
template <int NT>
struct Place {
  uint32_t item, share, rank;  // CTAs of the item, and which of them this is
  int kvh, b, qt, r0, rows, base;
  WinRow row;
  bool none;  // no rows here: the CTA (and every other of the item) leaves
};

template <int NT>
PKV_DEVINLINE Place<NT> place(const PkvWinArgs& a, int splits, int tid) {
  constexpr int ROWS = 8 * NT;
  Place<NT> p;
  const int g = a.Hq / a.Hkv;
  const int n_qt = (int)(((int64_t)a.max_query_len * g + ROWS - 1) / ROWS);
  p.share = splits > 1 ? (uint32_t)splits : cluster_size();
  p.rank = splits > 1 ? blockIdx.x % p.share : cluster_rank();
  uint32_t item = blockIdx.x / p.share;
  p.item = item;
  p.kvh = item % a.Hkv;
  item /= a.Hkv;
  p.qt = item % n_qt;
  p.b = item / n_qt;
  p.row = win_row(a, p.b, tid == 0 && p.qt == 0 && p.kvh == 0 && p.rank == 0);
  const int64_t total = (int64_t)p.row.Sq * g;
  p.none = (int64_t)p.qt * ROWS >= total;
  p.r0 = p.qt * ROWS;
  p.rows = p.none ? 0 : total - p.r0 < ROWS ? (int)(total - p.r0) : ROWS;
  p.base = p.row.L - p.row.Sq;
  return p;
}

// A warp's running softmax: per n-tile of 8 query rows, the lane's columns are rows 2t and 2t + 1.  o[nt][e] are the
// accumulators of channel tile e; m (log2 units) and l belong to the lane's rows, l holding the lane's keys only.
template <int D, int NT>
struct State {
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];

  PKV_DEVINLINE void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int e = 0; e < D / 16; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][e][c] = 0.f;
    }
  }

  // Scores s (unscaled; -inf where masked) of PG pages times f > 0 become probabilities, as P^T's B operands.
  template <bool BF16, int PG>
  PKV_DEVINLINE void update(float (&s)[PG][NT][4], const float (&f)[NT][2], uint32_t (&b0)[PG][NT],
                            uint32_t (&b1)[PG][NT]) {
    float top[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[nt][c] = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
        for (int u = 1; u < PG; ++u) top[nt][c] = ptx::max3(top[nt][c], s[u][nt][c], s[u][nt][c + 2]);
        top[nt][c] *= f[nt][c];
        grow = grow || top[nt][c] > m[nt][c] + kRescale;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) top[nt][c] = fmaxf(top[nt][c], __shfl_xor_sync(0xffffffffu, top[nt][c], k));
          if (top[nt][c] > m[nt][c]) {
            const float alpha = ptx::ex2(m[nt][c] - top[nt][c]);  // 0 from -inf
            m[nt][c] = top[nt][c];
            l[nt][c] *= alpha;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) o[nt][e][c] *= alpha, o[nt][e][c + 2] *= alpha;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mu[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) mu[c] = m[nt][c] == -INFINITY ? 0.f : -m[nt][c];
#pragma unroll
      for (int u = 0; u < PG; ++u) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[u][nt][c] = ptx::ex2(fmaf(s[u][nt][c], f[nt][c & 1], mu[c & 1]));
        l[nt][0] += s[u][nt][0] + s[u][nt][2];
        l[nt][1] += s[u][nt][1] + s[u][nt][3];
        b0[u][nt] = transpose8(pack<BF16>(s[u][nt][0], s[u][nt][1]));
        b1[u][nt] = transpose8(pack<BF16>(s[u][nt][2], s[u][nt][3]));
      }
    }
  }
};

template <int D, int NT>
struct MergeSmem {
  static constexpr int kStride = D + 2;
  float o[kWarps][8 * NT][kStride];
  float wm[kWarps][8 * NT], wl[kWarps][8 * NT];
  float m[8 * NT], l[8 * NT];
};

// Partial results of one split of an item, for the combine: [item][split] x (ROWS x D sums, ROWS maxima, ROWS sums).
template <int D, int NT>
constexpr int64_t kPartialFloats = 8 * NT * (D + 2);

// The warps' states merge in shared memory; then the cluster's CTAs write the rows, or, with splits, the CTA its
// partials.  chan(g, e, c): channel of accumulators 2c, 2c + 1 of tile e in lanes of group g.
template <typename T, int D, int NT, typename Chan>
PKV_DEVINLINE void merge(State<D, NT>& st, MergeSmem<D, NT>& sm, const PkvWinArgs& a, const Place<NT>& pl, int splits,
                         float* ws, int tid, Chan&& chan) {
  constexpr int ROWS = 8 * NT;
  const int warp = tid >> 5, lane = tid & 31, gl = lane >> 2, tl = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = st.l[nt][c];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      const int r = nt * 8 + 2 * tl + c;
      if (gl == 0) sm.wm[warp][r] = st.m[nt][c], sm.wl[warp][r] = sum;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        sm.o[warp][r][chan(gl, e, 0)] = st.o[nt][e][c];
        sm.o[warp][r][chan(gl, e, 1)] = st.o[nt][e][c + 2];
      }
    }
  __syncthreads();
  for (int e = tid; e < pl.rows * D; e += kThreads) {
    const int r = e / D, c = e % D;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.wm[w][r]);
    float acc = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sm.wm[w][r];
      const float k = mw == top ? 1.f : ptx::ex2(mw - top);
      acc += k * sm.o[w][r][c];
      sum += k * sm.wl[w][r];
    }
    if (splits > 1) {
      float* part = ws + ((int64_t)pl.item * splits + pl.rank) * kPartialFloats<D, NT>;
      part[r * D + c] = acc;
      if (c == 0) part[ROWS * D + r] = top, part[ROWS * (D + 1) + r] = sum;
      continue;
    }
    sm.o[0][r][c] = acc;  // read and written by this thread alone
    if (c == 0) sm.m[r] = top, sm.l[r] = sum;
  }
  if (splits > 1) return;
  win_merge_store<T, D>(&sm.o[0][0][0], MergeSmem<D, NT>::kStride, sm.m, sm.l, pl.rows, pl.r0, a.Hq / a.Hkv, pl.kvh, a.Hq,
                        pl.row.q0, (T*)a.out, tid, kThreads);
}

// Rows of the items that several CTAs share: one block per (item, row), its two halves each taking every other split.
// A programmatic dependent launch: its blocks may be in place before the attention's last CTAs are done.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(D) combine_kernel(const PkvWinArgs a, const int splits,
                                                             const float* __restrict__ ws) {
  constexpr int ROWS = 8 * NT, PAIRS = D / 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = a.Hq / a.Hkv;
  const int n_qt = (int)(((int64_t)a.max_query_len * g + ROWS - 1) / ROWS);
  const int r = blockIdx.x % ROWS;
  uint32_t item = blockIdx.x / ROWS;
  const float* part = ws + (int64_t)item * splits * kPartialFloats<D, NT>;
  const int kvh = item % a.Hkv;
  item /= a.Hkv;
  const int qt = item % n_qt, b = item / n_qt;
  const WinRow row = win_row(a, b, false);
  const int64_t at = (int64_t)qt * ROWS + r;
  if (at >= (int64_t)row.Sq * g) return;
  __shared__ float sm_w[kPkvMaxWinSplits];
  __shared__ float2 sm_x[PAIRS];
  __shared__ float sm_sum;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {  // the splits' weights
    float mk[2], lk[2], top = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = lane + 32 * h;
      mk[h] = k < splits ? part[k * kPartialFloats<D, NT> + ROWS * D + r] : -INFINITY;
      lk[h] = k < splits ? part[k * kPartialFloats<D, NT> + ROWS * (D + 1) + r] : 0.f;
      top = fmaxf(top, mk[h]);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float w = mk[h] == top ? 1.f : ptx::ex2(mk[h] - top);
      sm_w[lane + 32 * h] = w;
      sum += w * lk[h];
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (lane == 0) sm_sum = sum;
  }
  __syncthreads();
  const int half = tid / PAIRS, c = tid % PAIRS;
  float2 x = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int k = half; k < splits; k += 2) {
    const float2 v = *reinterpret_cast<const float2*>(part + k * kPartialFloats<D, NT> + r * D + 2 * c);
    x.x += sm_w[k] * v.x, x.y += sm_w[k] * v.y;
  }
  if (half) sm_x[c] = x;
  __syncthreads();
  if (half == 0) {
    const float sum = sm_sum, inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t tok = (int64_t)row.q0 + at / g;
    store_pair<T>((T*)a.out + (tok * a.Hq + kvh * g + at % g) * D + 2 * c, (x.x + sm_x[c].x) * inv,
                  (x.y + sm_x[c].y) * inv);
  }
}

// Plans and launches `kernel`, compiled for tiles of 8 NT rows.  ws_wanted: only say what workspace the call would use.
template <typename T, int D, int NT, typename Kernel>
int launch(Kernel kernel, PkvKernelState& state, size_t smem, double rate, double setup, const PkvWinArgs& a, void* workspace,
           size_t ws_bytes, size_t* ws_wanted, int* launches, cudaStream_t s) {
  int rc = pkv_prepare_kernel((const void*)kernel, (int)smem, kThreads, 0, state);
  if (rc) return rc;
  const int g = a.Hq / a.Hkv;
  const int64_t items = (int64_t)a.B * a.Hkv * (((int64_t)a.max_query_len * g + 8 * NT - 1) / (8 * NT));
  const int64_t steps = pkv_visible_keys(a, 8 * NT / g + 1) / (16 * kWarps) + 1;
  // Items too few for clusters of 16 to fill the GPU: more CTAs per item, and the combine launch.
  int splits = pkv_plan_splits(state, items, steps, rate, setup, kCombineSteps);
  const size_t need = splits > 1 ? (size_t)(items * splits * kPartialFloats<D, NT> * 4) : 0;
  if (ws_wanted) {
    *ws_wanted = need;
    return 0;
  }
  if (need > ws_bytes || !workspace) splits = 1;
  float* ws = splits > 1 ? (float*)workspace : nullptr;
  void* args[] = {const_cast<PkvWinArgs*>(&a), &splits, &ws};
  const int ctas = splits > 1 ? 1 : pkv_plan_cluster(state, items, steps, rate, setup);
  *launches = 1;
  rc = pkv_launch_cluster((const void*)kernel, splits > 1 ? items * splits : items, ctas, kThreads, smem, args, false, s);
  if (rc || splits == 1) return rc;
  *launches = 2;
  return pkv_launch_cluster((const void*)combine_kernel<T, D, NT>, items * 8 * NT, 1, D, 0, args, true, s);
}

}  // namespace dec
