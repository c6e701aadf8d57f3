// Shared by the window/sinks attention kernels: which keys a tile of query rows sees, and the merge of the CTAs
// that share them.
//
// Query rows are packed: row r of (sequence b, kv head) is query token r / g of head kvh * g + r % g, g = Hq / Hkv,
// so the query heads of one kv head share its keys in one tile.  The query at global position p sees key j when
// j <= p and (window == 0 or j < sinks or p - j < window).
#pragma once

#include "common.cuh"

// The 16-key pages that some row of a tile sees, numbered 0 .. n: first the sinks' pages, then the window's.
struct WinPages {
  int hi;       // keys [0, hi) end at the tile's last row
  int lo;       // first key of the tile's first row's window (0: none)
  int sinks;    // keys [0, sinks) are seen besides
  int n_sink;   // pages before the jump (0 when nothing is skipped)
  int first;    // logical page behind the jump
  int n;

  PKV_DEVINLINE int page(int v) const { return v < n_sink ? v : v - n_sink + first; }
  // Whether some row of the tile sees key j (rows are consecutive positions, so their windows leave no gap).
  PKV_DEVINLINE bool any(int j) const { return j < hi && (j >= lo || j < sinks); }
};

PKV_DEVINLINE WinPages win_pages(int p_first, int p_last, int window, int sinks) {
  WinPages w;
  w.hi = p_last + 1;
  w.lo = 0;
  if (window > 0 && p_first >= window) w.lo = p_first - (window - 1);
  w.sinks = sinks < w.hi ? sinks : w.hi;
  const int end = w.hi > 0 ? (w.hi + 15) >> 4 : 0;
  w.first = w.lo >> 4;
  w.n_sink = (w.sinks + 15) >> 4;
  if (w.first <= w.n_sink) w.n_sink = w.first = 0;
  w.n = end > 0 ? w.n_sink + end - w.first : 0;
  return w;
}

PKV_DEVINLINE bool win_sees(int p, int j, int window, int sinks) {
  return j <= p && (window == 0 || j < sinks || p - j < window);
}

// Row metadata with the checks of PKV_CHECK_BOUNDS applied.
struct WinRow {
  int q0, Sq, L;
};

PKV_DEVINLINE WinRow win_row(const PkvWinArgs& a, int b, bool flag) {
  WinRow r;
  r.q0 = a.query_start_loc[b];
  r.Sq = a.query_start_loc[b + 1] - r.q0;
  r.L = a.seq_lens[b];
  if (a.check) {
    if (r.Sq < 0 || r.Sq > a.max_query_len) {
      if (flag) pkv_raise(a.err, PKV_DEVERR_QUERY);
      r.Sq = r.Sq < 0 ? 0 : a.max_query_len;
    }
    const int most = (int64_t)a.W * 16 < a.max_seq_len ? a.W * 16 : a.max_seq_len;
    if (r.L < 0 || r.L > most) {
      if (flag) pkv_raise(a.err, PKV_DEVERR_SEQLEN);
      r.L = r.L < 0 ? 0 : most;
    }
  }
  return r;
}

// Physical block of a row's logical page; in check mode a bad id is flagged and block 0 read in its place.
PKV_DEVINLINE int win_block(const PkvWinArgs& a, int b, int page) {
  int blk = __ldg(a.block_table + (int64_t)b * a.W + page);
  if (a.check && (blk < 0 || blk >= a.num_blocks)) {
    pkv_raise(a.err, PKV_DEVERR_BLOCK);
    blk = 0;
  }
  return blk;
}

// ---------------------------------------------------------------- clusters

PKV_DEVINLINE uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
PKV_DEVINLINE uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster.
PKV_DEVINLINE void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared-memory address of `p` in the cluster's CTA `rank`.
PKV_DEVINLINE uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
PKV_DEVINLINE float cluster_ld(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
PKV_DEVINLINE float2 cluster_ld2(uint32_t addr) {
  float2 x;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
  return x;
}

template <typename T>
PKV_DEVINLINE void store_pair(T* p, float x, float y) {
  T v[2] = {pkv_from_f32<T>(x), pkv_from_f32<T>(y)};
  *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(v);
}
template <>
PKV_DEVINLINE void store_pair<float>(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}

// Each CTA holds, for every row of the tile, the sum o[row][D] of exp2(x - m[row]) v over its keys, m and l (the sum
// of the exponentials); m is in log2 units and -inf when it saw no key.  The rows are dealt out over the cluster's
// warps: a lane fetches one CTA's m and l, then D/32 channels of every CTA, so that the remote reads (some 0.2 us each)
// overlap.  Ends with a cluster barrier: no CTA leaves while another reads it.  o_stride is even.
template <typename T, int D>
PKV_DEVINLINE void win_merge_store(const float* o, int o_stride, const float* m, const float* l, int rows, int r0, int g,
                                   int kvh, int Hq, int q0, T* out, int tid, int threads) {
  constexpr int CH = D / 32;
  const uint32_t rank = cluster_rank(), n = cluster_size();
  __syncwarp();
  if (n > 1)
    cluster_sync();
  else
    __syncthreads();
  const int warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
  for (int r = rank * warps + warp; r < rows; r += n * warps) {
    float acc[CH] = {}, sum = 0.f;
    if (n == 1) {
#pragma unroll
      for (int c = 0; c < CH; ++c) acc[c] = o[r * o_stride + lane * CH + c];
      sum = l[r];
    } else {
      float mk = -INFINITY, lk = 0.f;
      if (lane < (int)n) mk = cluster_ld(cluster_addr(m + r, lane)), lk = cluster_ld(cluster_addr(l + r, lane));
      float top = mk;
#pragma unroll
      for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float w = mk == top ? 1.f : exp2f(mk - top);  // CTAs without keys hold zeros
#pragma unroll 8
      for (uint32_t k = 0; k < n; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const uint32_t src = cluster_addr(o + r * o_stride + lane * CH, k);
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          const float2 x = cluster_ld2(src + c * 4);
          acc[c] += wk * x.x, acc[c + 1] += wk * x.y;
        }
        sum += wk * __shfl_sync(0xffffffffu, lk, k);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a NaN sum stays
    const int row = r0 + r;
    const int64_t tok = (int64_t)q0 + row / g;
    T* dst = out + (tok * Hq + kvh * g + row % g) * D + lane * CH;
#pragma unroll
    for (int c = 0; c < CH; c += 2) store_pair<T>(dst + c, acc[c] * inv, acc[c + 1] * inv);
  }
  if (n > 1) {
    __syncwarp();
    cluster_sync();
  }
}
