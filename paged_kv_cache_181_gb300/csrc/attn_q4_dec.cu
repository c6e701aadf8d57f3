// Window/sinks attention for few query rows per kv head over 4-bit pools, bf16/f16 queries.  The scheme is that of
// attn_win_dec.cu (warps take pages in turn, keys as the rows of m16n8k16 products, one merge at the end); what
// differs is what bounds it: a page of one head is 2560 bytes instead of 8192, so the instructions that turn codes
// into operands weigh as much as the memory: 64 sequences of up to 16384 keys, 32/8 heads, D 128: 169 us, 74 % of the
// measured copy bandwidth (61 % of the SMs' issue and math throughput); one of 131072 keys 44 us, 56 %.
//
// A page's records (K and V, 1280 contiguous bytes each for D = 128) come by one bulk copy each into a ring of the
// warp's own, four pages deep, so no register waits for memory and the loop holds no addresses.  Codes become
// fp16(step * n + low), exactly the value the format gives them, in 13 instructions per 8 of them (q4.cuh).  Both products
// run in fp16; Q is scaled per row by a power of two into fp16's range (exact for all but values 2^-24 of the row's
// largest), and the scores scaled back in fp32.
//
// The order of a page's keys is permuted: row g of the K operand is key g / 2 + 4 (g odd) (xor 1 of the low bit for
// odd g), so that the lanes of a K read and of a V read both spread over the banks (64-byte rows).

#include "q4.cuh"
#include "win_dec.cuh"

namespace {

using namespace dec;

constexpr int kPG = 2;    // pages per step
constexpr int kRing = 2;  // steps in flight or in use per warp
constexpr uint64_t kWaitLimitNs = 1000000000ull;

PKV_DEVINLINE uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
PKV_DEVINLINE __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// Key of the page's first eight at row g of an operand.
PKV_DEVINLINE int key_of(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1; }

PKV_DEVINLINE void bulk_load(void* dst, const void* src, uint32_t n, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(src), "r"(n), "r"(ptx::smem_u32(bar))
               : "memory");
}

// K: rows g and g + 8 of the operand; a lane's 16 (D = 64: 8) bytes are channels of one group.
template <int D, typename Fn>
PKV_DEVINLINE void k_steps(const uint8_t* rec, int g, int t, Fn&& f) {
  using F = Q4<D>;
  uint32_t w[2][D / 32];
  __half2 pair[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int key = key_of(g) + 8 * r;
    const uint8_t* p = rec + key * F::kRowBytes + t * (D / 8);
    if (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[r][0] = x.x, w[r][1] = x.y, w[r][D / 32 - 2] = x.z, w[r][D / 32 - 1] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[r][0] = x.x, w[r][1] = x.y;
    }
    pair[r] = *reinterpret_cast<const __half2*>(rec + F::kPairs + (key * F::kGroups + (D == 128 ? t : t >> 1)) * 4);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    __half2 x[4], y[4];
    q4_values(w[0][i], pair[0], x);
    q4_values(w[1][i], pair[1], y);
    f(2 * i, as_u32(x[0]), as_u32(y[0]), as_u32(x[1]), as_u32(y[1]));
    f(2 * i + 1, as_u32(x[2]), as_u32(y[2]), as_u32(x[3]), as_u32(y[3]));
  }
}

// V: keys of operand columns 2t, 2t + 1, 2t + 8, 2t + 9; a lane's 8 (4) bytes of a key are 16 (8) channels of one
// group.  Keys whose bit is clear in `seen` are zeros.
template <int D, typename Fn>
PKV_DEVINLINE void v_tiles(const uint8_t* rec, int g, int t, unsigned seen, Fn&& f) {
  using F = Q4<D>;
  uint32_t w[4][D / 64], pair[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int key = key_of(2 * t + (r & 1)) + 8 * (r >> 1);
    const uint8_t* p = rec + key * F::kRowBytes + g * (D / 16);
    if (D == 128) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[r][0] = x.x, w[r][D / 64 - 1] = x.y;
    } else {
      w[r][0] = *reinterpret_cast<const uint32_t*>(p);
    }
    pair[r] = *reinterpret_cast<const uint32_t*>(rec + F::kPairs + (key * F::kGroups + (D == 128 ? g >> 1 : g >> 2)) * 4);
    if (seen != 0xffffu && !((seen >> key) & 1)) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) w[r][i] = 0;
      pair[r] = 0;
    }
  }
  __half2 step[2], low[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    step[r] = as_h2(low_halves(pair[2 * r], pair[2 * r + 1]));
    low[r] = as_h2(high_halves(pair[2 * r], pair[2 * r + 1]));
  }
  // Channels 4h .. 4h + 3 of word i for the keys 2t, 2t + 1 (r = 0) or 2t + 8, 2t + 9 (r = 1).
  auto four = [&](int r, int i, int h, __half2(&x)[4]) {
    q4_unpack(h ? high_halves(w[2 * r][i], w[2 * r + 1][i]) : low_halves(w[2 * r][i], w[2 * r + 1][i]), x);
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = __hfma2(x[c], step[r], low[r]);
  };
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
    __half2 a0[4], a1[4], a2[4], a3[4];
    if (D == 128) {
      four(0, 0, h, a0), four(0, D / 64 - 1, h, a1), four(1, 0, h, a2), four(1, D / 64 - 1, h, a3);
    } else {
      four(0, 0, 0, a0), four(0, 0, 1, a1), four(1, 0, 0, a2), four(1, 0, 1, a3);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f(4 * h + i, as_u32(a0[i]), as_u32(a1[i]), as_u32(a2[i]), as_u32(a3[i]));
  }
}

template <int D>
PKV_DEVINLINE int chan(int g, int e, int c) { return D == 128 ? 16 * g + 8 * c + e : 8 * g + 4 * c + e; }

template <int D, int NT>
struct Smem {
  union {
    uint8_t ring[kWarps][kRing][kPG][2][Q4<D>::kRecord];
    MergeSmem<D, NT> merge;
  };
  uint64_t full[kWarps][kRing];
  float rscale[8 * NT];
  uint4 q[NT > 2 ? NT : 1][NT > 2 ? D / 32 : 1][32];  // Q's B operands, when they do not fit in registers
  int abort;
};

// `splits` > 1: that many CTAs (no clusters) share an item and leave partials in `ws`.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : NT == 2 ? 3 : 2)
    attn_q4_dec_kernel(const PkvWinArgs a, const int splits, float* __restrict__ ws) {
  constexpr bool QS = NT > 2;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D, NT>& sm = *reinterpret_cast<Smem<D, NT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gl = lane >> 2, tl = lane & 3;
  const int g = a.Hq / a.Hkv;
  if (splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Place<NT> pl = place<NT>(a, splits, tid);
  if (pl.none) return;
  const int p_first = pl.base + pl.r0 / g, p_last = pl.base + (pl.r0 + pl.rows - 1) / g;
  const WinPages pg = win_pages(p_first, p_last, a.window, a.sinks);

  // This warp's pages: gw, gw + stride, ...; a lane holds the block id of one of 32, fetched ahead.
  const int gw = pl.rank * kWarps + warp, stride = pl.share * kWarps;
  const int n = pg.n > gw ? (pg.n - gw + stride - 1) / stride : 0;
  auto fetch_ids = [&](int i) -> int {
    return i + lane < n ? win_block(a, pl.b, pg.page(gw + (i + lane) * stride)) : 0;
  };
  int ids = fetch_ids(0), ids_next = fetch_ids(32);
  if (lane == 0) {
    for (int s = 0; s < kRing; ++s) ptx::mbar_init(&sm.full[warp][s], 1);
    ptx::fence_mbar_init();
  }
  if (tid == 0) sm.abort = 0;
  __syncwarp();
  // Pages i .. i + kPG - 1 into step slot (i / kPG) % kRing, a lane per record; i counts up by kPG from call to call.
  const uint8_t* const pool = (const uint8_t*)((lane & 1) ? a.v_pool : a.k_pool) + (int64_t)pl.kvh * Q4<D>::kRecord;
  auto issue = [&](int i) {
    if (i >= n) return;
    if (i && (i & 31) == 0) ids = ids_next, ids_next = fetch_ids(i + 32);
    const int blk = __shfl_sync(0xffffffffu, ids, (i + (lane >> 1)) & 31);
    const int pages = n - i < kPG ? n - i : kPG;
    const int slot = (i / kPG) % kRing;
    if (lane == 0) ptx::mbar_arrive_expect_tx(&sm.full[warp][slot], 2 * pages * Q4<D>::kRecord);
    __syncwarp();
    if (lane < 2 * pages)
      bulk_load(sm.ring[warp][slot][lane >> 1][lane & 1], pool + (int64_t)blk * (a.Hkv * Q4<D>::kRecord), Q4<D>::kRecord,
                &sm.full[warp][slot]);
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i) issue(i * kPG);

  // Q operands: n = query row gl of each group of eight, channels in the order that q4_unpack gives.
  uint4 q[QS ? 1 : NT][D / 32];
  float f[NT][2];
  int p[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + gl;
    const int64_t tok = (int64_t)pl.row.q0 + (pl.r0 + r) / g;
    const uint4* src = reinterpret_cast<const uint4*>((const T*)a.q + (tok * a.Hq + pl.kvh * g + (pl.r0 + r) % g) * D);
    uint4 x[D / 32];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      x[i] = r < pl.rows ? __ldg(src + tl * (D / 32) + i) : make_uint4(0, 0, 0, 0);
      const T* e = reinterpret_cast<const T*>(&x[i]);
#pragma unroll
      for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(pkv_to_f32<T>(e[c])));
    }
    // The row's largest magnitude goes to [2^13, 2^14) (0, infinities and NaN stay).
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e2 = top > 0.f && top <= 3.402823466e38f ? min(13 - ilogbf(top), 64) : 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const T* e = reinterpret_cast<const T*>(&x[i]);
      uint32_t w[4];  // channels (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[c] = ptx::pack_f16x2(scalbnf(pkv_to_f32<T>(e[c]), e2), scalbnf(pkv_to_f32<T>(e[c + 4]), e2));
      if (QS) {
        if (warp == 0) sm.q[nt][i][lane] = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        q[nt][i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (warp == 0 && tl == 0) sm.rscale[r] = fmaxf(scalbnf(a.scale * 1.4426950408889634f, -e2), 1e-37f);
#pragma unroll
    for (int c = 0; c < 2; ++c) p[nt][c] = pl.base + (pl.r0 + nt * 8 + 2 * tl + c) / g;
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) f[nt][c] = sm.rscale[nt * 8 + 2 * tl + c];

  State<D, NT> st;
  st.clear();
  const int key = key_of(gl);
  // Pages [v_lo, v_hi) of the list hold keys that every row sees (besides whole sink pages, which take the masked way).
  int v_lo = 0, v_hi = p_first + 1 > 0 ? (p_first + 1) >> 4 : 0;  // as logical pages
  if (a.window && p_last >= a.window) v_lo = (p_last - (a.window - 1) + 15) >> 4;
  v_lo += pg.n_sink - pg.first, v_hi += pg.n_sink - pg.first;
  if (v_lo < pg.n_sink) v_lo = pg.n_sink;
  for (int i = 0; i < n; i += kPG) {
    const int v = gw + i * stride, slot = (i / kPG) % kRing;
    const bool all = v >= v_lo && v + (kPG - 1) * stride < v_hi;  // v_hi <= pg.n: every page of the step is there
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(&sm.full[warp][slot], (i / (kPG * kRing)) & 1, &sm.abort, kWaitLimitNs))) {
      sm.abort = 1;
      if (lane == 0) pkv_raise(a.err, PKV_DEVERR_TIMEOUT);
      break;
    }
    unsigned seen[kPG];
    float s[kPG][NT][4] = {};
#pragma unroll
    for (int u = 0; u < kPG; ++u)
      k_steps<D>(sm.ring[warp][slot][u][0], gl, tl, [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 qq = QS ? sm.q[nt][k >> 1][lane] : q[QS ? 0 : nt][k >> 1];
          mma<false>(s[u][nt], a0, a1, a2, a3, (k & 1) ? qq.z : qq.x, (k & 1) ? qq.w : qq.y);
        }
      });
#pragma unroll
    for (int u = 0; u < kPG; ++u) seen[u] = 0xffffu;
    if (!all) {
#pragma unroll
      for (int u = 0; u < kPG; ++u) {
        const int j0 = i + u < n ? pg.page(v + u * stride) * 16 : 0x7fffff00;  // past every key
        seen[u] = __ballot_sync(0xffffffffu, pg.any(j0 + (lane & 15))) & 0xffffu;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s[u][nt][c] = win_sees(p[nt][c & 1], j0 + key + 8 * (c >> 1), a.window, a.sinks) ? s[u][nt][c] : -INFINITY;
      }
    }
    uint32_t b0[kPG][NT], b1[kPG][NT];
    st.template update<false>(s, f, b0, b1);
#pragma unroll
    for (int u = 0; u < kPG; ++u)
      v_tiles<D>(sm.ring[warp][slot][u][1], gl, tl, seen[u],
                 [&](int e, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                   for (int nt = 0; nt < NT; ++nt) mma<false>(st.o[nt][e], a0, a1, a2, a3, b0[u][nt], b1[u][nt]);
                 });
    __syncwarp();  // every lane has read the step's pages
    issue(i + kRing * kPG);
  }
  if (sm.abort && lane == 0) {
    // Let copies already issued land before the shared memory goes away.
    int never = 0;
    for (int s = 0; s < kRing; ++s) ptx::mbar_wait(&sm.full[warp][s], 0, &never, 1000000ull);
  }
  __syncthreads();  // the merge takes the rings' place
  merge<T>(st, sm.merge, a, pl, splits, ws, tid, [](int gg, int e, int c) { return chan<D>(gg, e, c); });
}

template <typename T, int D, int NT>
int launch_nt(const PkvWinArgs& a, void* ws, size_t bytes, size_t* wanted, int* launches, cudaStream_t s) {
  static PkvKernelState state;
  return dec::launch<T, D, NT>(attn_q4_dec_kernel<T, D, NT>, state, sizeof(Smem<D, NT>), 0.4, 7.0, a, ws, bytes, wanted,
                             launches, s);
}

template <typename T, int D>
int launch_rows(const PkvWinArgs& a, void* ws, size_t bytes, size_t* wanted, int* launches, cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_query_len * (a.Hq / a.Hkv);
  if (rows <= 8) return launch_nt<T, D, 1>(a, ws, bytes, wanted, launches, s);
  if (rows <= 16) return launch_nt<T, D, 2>(a, ws, bytes, wanted, launches, s);
  return launch_nt<T, D, 4>(a, ws, bytes, wanted, launches, s);
}

}  // namespace

int pkv_launch_q4_dec(const PkvWinArgs& a, pkv_dtype dt, int D, void* ws, size_t ws_bytes, size_t* ws_wanted,
                      int* launches, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  if (dt == PKV_BF16)
    return D == 64 ? launch_rows<__nv_bfloat16, 64>(a, ws, ws_bytes, ws_wanted, launches, s)
                   : launch_rows<__nv_bfloat16, 128>(a, ws, ws_bytes, ws_wanted, launches, s);
  if (dt == PKV_F16)
    return D == 64 ? launch_rows<__half, 64>(a, ws, ws_bytes, ws_wanted, launches, s)
                   : launch_rows<__half, 128>(a, ws, ws_bytes, ws_wanted, launches, s);
  return (int)cudaErrorInvalidValue;
}
