// Window/sinks attention for few query rows per kv head (decode, and a few tokens verified together), bf16/f16
// queries over 16-bit pools.  Bound by memory: every visible key and value is read once and meets only
// Sq * g rows, so the kernel is built around keeping loads in flight, not around the products.
//
// One cluster = 8 NT packed query rows (attn_win.cuh) of one (sequence, kv head).  All warps of its CTAs take the
// visible 16-key pages in turn, each with its own running maximum, sum and output; they merge once, at the end.
//
// Products are m16n8k16 with the keys as rows:  S^T = K Q^T  and  O^T = V^T P^T,  so that eight query rows fill the
// n side (the other way round half of each product would be padding).  No shared memory is used for keys and
// values: the sum over channels may run in any order, so a lane loads 16 contiguous bytes of a key and uses them as
// two k-steps' operands, with Q permuted to match; a V operand pairs two keys per register, which one byte
// permute per pair makes from two keys' loads.  P^T comes from S^T's registers by one 8x8 transpose per 8 keys.
// Loads of the next page are issued as soon as the registers of this page's K (then V) are used up: 12 warps of an
// SM keep 4 to 8 KB each in flight.  64 sequences x 8192-key windows (40/8 heads, D 128): 318 us, 92 % of the measured
// copy bandwidth; one sequence x 4096 keys, 8 kv heads: 11 us, latency (a page's loads, the merge, two launches).
//
// A row's maximum is raised only when a score exceeds it by 2^8 (one vote per page, no shuffles otherwise);
// probabilities stay below 2^8, exact in their 16-bit type's range.  P is rounded to the value type for the product,
// as in the prefix-mask kernel; the sum l adds the unrounded probabilities.

#include "win_dec.cuh"

namespace {

using namespace dec;

// Loads of bytes that this warp alone uses, once: past L1.
PKV_DEVINLINE uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
// ---------------------------------------------------------------- one page's operands
//
// Lane (g, t) = lane / 4, lane % 4.  K: keys g and g + 8 of the page, as A operands of the D/16 channel steps.
// V: keys 2t, 2t+1, 2t+8, 2t+9, as A operands of D/16 tiles of 16 channels.  chan() gives the channels of a tile's
// rows g and g + 8, q_vector() the vectors of Q that match K's order of channels.

template <int D>
struct Page16 {
  static constexpr int NK = D / 32, NV = D / 64;
  uint4 k[2][NK];
  uint4 v[4][NV];

  static PKV_DEVINLINE int64_t page_bytes(int Hkv) { return (int64_t)16 * Hkv * D * 2; }
  static PKV_DEVINLINE int64_t head_bytes(int kvh) { return (int64_t)kvh * D * 2; }

  // Keys whose bit is clear in `seen` (bit k: key k of the page) are not loaded and count as zeros.
  PKV_DEVINLINE void load_k(const uint8_t* head, int Hkv, int g, int t, unsigned seen) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* p = head + (int64_t)(g + 8 * r) * Hkv * D * 2 + t * 16;
      if (seen == 0xffffu || ((seen >> (g + 8 * r)) & 1)) {
#pragma unroll
        for (int i = 0; i < NK; ++i) k[r][i] = ld16(p + 64 * i);
      } else {
#pragma unroll
        for (int i = 0; i < NK; ++i) k[r][i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  PKV_DEVINLINE void load_v(const uint8_t* head, int Hkv, int g, int t, unsigned seen) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int key = 2 * t + (r & 1) + (r >> 1) * 8;
      const uint8_t* p = head + (int64_t)key * Hkv * D * 2 + g * 16;
      if (seen == 0xffffu || ((seen >> key) & 1)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[r][i] = ld16(p + 128 * i);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[r][i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  static PKV_DEVINLINE uint32_t word(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }
  template <typename F>
  PKV_DEVINLINE void k_steps(F&& f) const {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      f(2 * i, k[0][i].x, k[1][i].x, k[0][i].y, k[1][i].y);
      f(2 * i + 1, k[0][i].z, k[1][i].z, k[0][i].w, k[1][i].w);
    }
  }
  template <typename F>
  PKV_DEVINLINE void v_tiles(F&& f) const {
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
      uint32_t a[4];
#pragma unroll
      for (int r = 0; r < 2; ++r)      // keys 2t, 2t+1 / 2t+8, 2t+9
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // rows g / g + 8
          const int chunk = D == 128 ? c : 0, elem = D == 128 ? e : e + 4 * c;
          const uint32_t x = word(v[2 * r][chunk], elem >> 1), y = word(v[2 * r + 1][chunk], elem >> 1);
          a[2 * r + c] = (elem & 1) ? high_halves(x, y) : low_halves(x, y);
        }
      f(e, a[0], a[1], a[2], a[3]);
    }
  }
  static PKV_DEVINLINE int chan(int g, int e, int c) { return D == 128 ? 64 * c + 8 * g + e : 8 * g + 4 * c + e; }
  // The 8-channel vector whose four words are the B operands of steps 2i and 2i + 1.
  static PKV_DEVINLINE int q_vector(int t, int i) { return t + 4 * i; }
};

template <int D, int NT>
struct Smem {
  MergeSmem<D, NT> merge;
  uint4 q[NT > 2 ? NT : 1][NT > 2 ? D / 32 : 1][32];  // Q's B operands, when they do not fit in registers
};

// `splits` > 1: that many CTAs (no clusters) share an item and leave partials in `ws`.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
    attn_win_dec_kernel(const PkvWinArgs a, const int splits, float* __restrict__ ws) {
  constexpr bool BF16 = !std::is_same<T, __half>::value;
  constexpr bool QS = NT > 2;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D, NT>& sm = *reinterpret_cast<Smem<D, NT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gl = lane >> 2, tl = lane & 3;
  const int g = a.Hq / a.Hkv;
  if (splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Place<NT> pl = place<NT>(a, splits, tid);
  if (pl.none) return;
  const int p_first = pl.base + pl.r0 / g, p_last = pl.base + (pl.r0 + pl.rows - 1) / g;
  const WinPages pg = win_pages(p_first, p_last, a.window, a.sinks);

  // This warp's pages: gw, gw + stride, ...; their block ids are fetched 32 at a time, one per lane.
  const int gw = pl.rank * kWarps + warp, stride = pl.share * kWarps;
  const int n = pg.n > gw ? (pg.n - gw + stride - 1) / stride : 0;
  const int64_t page_bytes = (int64_t)16 * a.Hkv * D * 2, head_bytes = (int64_t)pl.kvh * D * 2;
  int ids = 0;
  Page16<D> page;
  const uint8_t* vhead = nullptr;
  int first = 0;      // first key of the page
  unsigned seen = 0;  // its keys that some row sees
  auto issue_k = [&](int i) {  // i counts up by one from call to call
    if ((i & 31) == 0) {
      const int v = gw + (i + lane) * stride;
      ids = i + lane < n ? win_block(a, pl.b, pg.page(v)) : 0;
    }
    const int64_t at = (int64_t)__shfl_sync(0xffffffffu, ids, i & 31) * page_bytes + head_bytes;
    first = pg.page(gw + i * stride) * 16;
    seen = 0xffffu;
    if (!(first + 15 < pg.hi && (first >= pg.lo || first + 15 < pg.sinks)))
      seen = __ballot_sync(0xffffffffu, pg.any(first + (lane & 15))) & 0xffffu;
    vhead = (const uint8_t*)a.v_pool + at;
    page.load_k((const uint8_t*)a.k_pool + at, a.Hkv, gl, tl, seen);
  };
  if (n > 0) {
    issue_k(0);
    page.load_v(vhead, a.Hkv, gl, tl, seen);
  }

  // Q operands: n = query row gl of each group of eight.
  const float sl2 = fmaxf(a.scale * 1.4426950408889634f, 1e-37f);
  uint4 q[QS ? 1 : NT][D / 32];
  float f[NT][2];
  int p[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + gl;
    const int64_t tok = (int64_t)pl.row.q0 + (pl.r0 + r) / g;
    const uint4* src = reinterpret_cast<const uint4*>((const T*)a.q + (tok * a.Hq + pl.kvh * g + (pl.r0 + r) % g) * D);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < pl.rows) x = __ldg(src + Page16<D>::q_vector(tl, i));
      if (QS) {
        if (warp == 0) sm.q[nt][i][lane] = x;
      } else {
        q[nt][i] = x;
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) f[nt][c] = sl2, p[nt][c] = pl.base + (pl.r0 + nt * 8 + 2 * tl + c) / g;
  }
  if (QS) __syncthreads();

  State<D, NT> st;
  st.clear();
  for (int i = 0; i < n; ++i) {
    float s[1][NT][4] = {};
    page.k_steps([&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 qq = QS ? sm.q[nt][k >> 1][lane] : q[QS ? 0 : nt][k >> 1];
        mma<BF16>(s[0][nt], a0, a1, a2, a3, (k & 1) ? qq.z : qq.x, (k & 1) ? qq.w : qq.y);
      }
    });
    const int j0 = first;
    const bool more = i + 1 < n;
    if (more) issue_k(i + 1);  // K's registers are free; V's still hold this page
    if (!(j0 + 15 <= p_first && (a.window == 0 || j0 + 15 < a.sinks || p_last - j0 < a.window))) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          s[0][nt][c] = win_sees(p[nt][c & 1], j0 + gl + 8 * (c >> 1), a.window, a.sinks) ? s[0][nt][c] : -INFINITY;
    }
    uint32_t b0[1][NT], b1[1][NT];
    st.template update<BF16>(s, f, b0, b1);
    page.v_tiles([&](int e, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma<BF16>(st.o[nt][e], a0, a1, a2, a3, b0[0][nt], b1[0][nt]);
    });
    if (more) page.load_v(vhead, a.Hkv, gl, tl, seen);
  }
  merge<T>(st, sm.merge, a, pl, splits, ws, tid, [](int gg, int e, int c) { return Page16<D>::chan(gg, e, c); });
}

template <typename T, int D, int NT>
int launch_nt(const PkvWinArgs& a, void* ws, size_t bytes, size_t* wanted, int* launches, cudaStream_t s) {
  static PkvKernelState state;
  return dec::launch<T, D, NT>(attn_win_dec_kernel<T, D, NT>, state, sizeof(Smem<D, NT>), 0.34, 5.2, a, ws, bytes, wanted,
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

int pkv_launch_win_dec(const PkvWinArgs& a, pkv_dtype dt, int D, void* ws, size_t ws_bytes, size_t* ws_wanted,
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
