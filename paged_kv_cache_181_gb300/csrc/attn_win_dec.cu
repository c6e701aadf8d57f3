// Window/sinks attention for few query rows per kv head (decode, and a few tokens verified together), bf16/f16
// queries over 16-bit or 4-bit pools.  Bound by memory: every visible key and value is read once and meets only
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
// Loads of the next step (one page; two of a 4-bit pool) are issued as soon as the registers of this step's K (then V)
// are used up.
//
// A row's maximum is raised only when a score exceeds it by 2^8 (one vote per page, no shuffles otherwise);
// probabilities stay below 2^8, exact in their 16-bit type's range.  P is rounded to the value type for the product,
// as in the prefix-mask kernel; the sum l adds the unrounded probabilities.
//
// 4-bit pools: codes become fp16 step * n + low, one rounding, exactly the value the format gives them; Q is
// scaled per row by a power of two into fp16's range (exact for all but values 2^-24 of the row's largest) and
// the scores scaled back in fp32.

#include <atomic>
#include <type_traits>

#include "attn_win.cuh"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kRescale = 8.f;  // log2 units

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

// Loads of bytes that this warp alone uses, once: past L1.
PKV_DEVINLINE uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
PKV_DEVINLINE uint2 ld8(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
PKV_DEVINLINE uint32_t ld4(const void* p) {
  uint32_t r;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

PKV_DEVINLINE uint32_t low_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
PKV_DEVINLINE uint32_t high_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
PKV_DEVINLINE uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
PKV_DEVINLINE __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// ---------------------------------------------------------------- one page's operands
//
// Lane (g, t) = lane / 4, lane % 4.  K: keys g and g + 8 of the page, as A operands of the D/16 channel steps.
// V: keys 2t, 2t+1, 2t+8, 2t+9, as A operands of D/16 tiles of 16 channels.  chan() gives the channels of a tile's
// rows g and g + 8, q_operand() the B operands of Q that match K's order of channels.

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
  static PKV_DEVINLINE uint4 q_order(const uint4& x) { return x; }
};

template <int D>
struct PageQ4 {
  using F = Q4<D>;
  uint32_t k[2][D / 32];
  uint32_t kp[2];
  uint32_t v[4][D / 64];
  uint32_t vp[4];

  static PKV_DEVINLINE int64_t page_bytes(int Hkv) { return (int64_t)Hkv * F::kRecord; }
  static PKV_DEVINLINE int64_t head_bytes(int kvh) { return (int64_t)kvh * F::kRecord; }

  PKV_DEVINLINE void load_k(const uint8_t* rec, int, int g, int t, unsigned seen) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int key = g + 8 * r;
      if (seen == 0xffffu || ((seen >> key) & 1)) {
        if (D == 128) {
          const uint4 x = ld16(rec + key * F::kRowBytes + t * 16);
          k[r][0] = x.x, k[r][1] = x.y, k[r][D / 32 - 2] = x.z, k[r][D / 32 - 1] = x.w;
        } else {
          const uint2 x = ld8(rec + key * F::kRowBytes + t * 8);
          k[r][0] = x.x, k[r][1] = x.y;
        }
        kp[r] = ld4(rec + F::kPairs + (key * F::kGroups + (D == 128 ? t : t >> 1)) * 4);
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) k[r][i] = 0;
        kp[r] = 0;
      }
    }
  }
  PKV_DEVINLINE void load_v(const uint8_t* rec, int, int g, int t, unsigned seen) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int key = 2 * t + (r & 1) + (r >> 1) * 8;
      if (seen == 0xffffu || ((seen >> key) & 1)) {
        if (D == 128) {
          const uint2 x = ld8(rec + key * F::kRowBytes + g * 8);
          v[r][0] = x.x, v[r][D / 64 - 1] = x.y;
        } else {
          v[r][0] = ld4(rec + key * F::kRowBytes + g * 4);
        }
        vp[r] = ld4(rec + F::kPairs + (key * F::kGroups + (D == 128 ? g >> 1 : g >> 2)) * 4);
      } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) v[r][i] = 0;
        vp[r] = 0;
      }
    }
  }
  template <typename Fn>
  PKV_DEVINLINE void k_steps(Fn&& f) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      __half2 x[4], y[4];
      q4_values(k[0][i], as_h2(kp[0]), x);
      q4_values(k[1][i], as_h2(kp[1]), y);
      f(2 * i, as_u32(x[0]), as_u32(y[0]), as_u32(x[1]), as_u32(y[1]));
      f(2 * i + 1, as_u32(x[2]), as_u32(y[2]), as_u32(x[3]), as_u32(y[3]));
    }
  }
  // Channels 4h .. 4h+3 of word w for keys 2t, 2t+1 (r = 0) or 2t+8, 2t+9 (r = 1): x[i] = the two keys' values.
  PKV_DEVINLINE void four(int r, int w, int h, __half2 (&x)[4]) const {
    uint32_t n = h ? high_halves(v[2 * r][w], v[2 * r + 1][w]) : low_halves(v[2 * r][w], v[2 * r + 1][w]);
    const __half2 step = as_h2(low_halves(vp[2 * r], vp[2 * r + 1])), low = as_h2(high_halves(vp[2 * r], vp[2 * r + 1]));
    q4_unpack(n, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __hfma2(x[i], step, low);
  }
  template <typename Fn>
  PKV_DEVINLINE void v_tiles(Fn&& f) const {
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {  // four tiles at a time: nibbles 4h .. 4h+3 of the word(s)
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
  static PKV_DEVINLINE int chan(int g, int e, int c) { return D == 128 ? 16 * g + 8 * c + e : 8 * g + 4 * c + e; }
  static PKV_DEVINLINE int q_vector(int t, int i) { return t * (D / 32) + i; }
  // q4_unpack gives the channel pairs (0, 4), (1, 5), (2, 6), (3, 7).
  static PKV_DEVINLINE uint4 q_order(const uint4& x) {
    return make_uint4(low_halves(x.x, x.z), high_halves(x.x, x.z), low_halves(x.y, x.w), high_halves(x.y, x.w));
  }
};

template <bool BF16>
PKV_DEVINLINE uint32_t pack(float lo, float hi) {
  return BF16 ? ptx::pack_bf16x2(lo, hi) : ptx::pack_f16x2(lo, hi);
}

template <int D, int NT>
struct DecSmem {
  static constexpr int kStride = D + 2;
  float o[kWarps][8 * NT][kStride];
  float wm[kWarps][8 * NT], wl[kWarps][8 * NT];
  float m[8 * NT], l[8 * NT];
  float rscale[8 * NT];
  uint4 q[NT > 2 ? NT : 1][NT > 2 ? D / 32 : 1][32];  // Q's B operands, when they do not fit in registers
};

// Partial results of one split of an item, for the combine: [item][split] x (ROWS x D sums, ROWS maxima, ROWS sums).
template <int D, int NT>
constexpr int64_t kPartialFloats = 8 * NT * (D + 2);

// PG pages per step.  `splits` > 1: that many CTAs (no clusters) share an item and leave partials in `ws`.
template <typename T, bool POOLQ4, int D, int NT, int PG>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
    attn_win_dec_kernel(const PkvWinArgs a, const int splits, float* __restrict__ ws) {
  constexpr bool BF16 = !POOLQ4 && sizeof(T) == 2 && !std::is_same<T, __half>::value;
  constexpr int ROWS = 8 * NT;
  constexpr bool QS = NT > 2;
  using Page = typename std::conditional<POOLQ4, PageQ4<D>, Page16<D>>::type;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  DecSmem<D, NT>& sm = *reinterpret_cast<DecSmem<D, NT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gl = lane >> 2, tl = lane & 3;
  const int g = a.Hq / a.Hkv;
  const int n_qt = (int)(((int64_t)a.max_query_len * g + ROWS - 1) / ROWS);
  if (splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t share = splits > 1 ? (uint32_t)splits : cluster_size();  // CTAs of one item
  const uint32_t rank = splits > 1 ? blockIdx.x % share : cluster_rank();
  uint32_t item = blockIdx.x / share;
  const uint32_t item_id = item;
  const int kvh = item % a.Hkv;
  item /= a.Hkv;
  const int qt = item % n_qt, b = item / n_qt;
  const WinRow row = win_row(a, b, tid == 0 && qt == 0 && kvh == 0 && rank == 0);
  const int64_t total = (int64_t)row.Sq * g;
  if ((int64_t)qt * ROWS >= total) return;  // the whole cluster leaves
  const int r0 = qt * ROWS;
  const int rows = total - r0 < ROWS ? (int)(total - r0) : ROWS;
  const int base = row.L - row.Sq;
  const int p_first = base + r0 / g, p_last = base + (r0 + rows - 1) / g;
  const WinPages pg = win_pages(p_first, p_last, a.window, a.sinks);

  // Q operands (n = query row gl of each group of eight) and the factor of each of the lane's score columns.
  const float sl2 = a.scale * 1.4426950408889634f;
  uint4 q[QS ? 1 : NT][D / 32];
  float f[NT][2];
  int p[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + gl;
    uint4 x[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const int64_t tok = (int64_t)row.q0 + (r0 + r) / g;
      const uint4* src = reinterpret_cast<const uint4*>((const T*)a.q + (tok * a.Hq + kvh * g + (r0 + r) % g) * D);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x[i] = __ldg(src + Page::q_vector(tl, i));
    }
    if (POOLQ4) {
      // fp16 operands: scale the row so that its largest magnitude lies in [2^13, 2^14) (0, infinities and NaN stay).
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const T* e = reinterpret_cast<const T*>(&x[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(pkv_to_f32<T>(e[c])));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e2 = top > 0.f && top <= 3.402823466e38f ? min(13 - ilogbf(top), 64) : 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const T* e = reinterpret_cast<const T*>(&x[i]);
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c] = ptx::pack_f16x2(scalbnf(pkv_to_f32<T>(e[2 * c]), e2), scalbnf(pkv_to_f32<T>(e[2 * c + 1]), e2));
        x[i] = Page::q_order(make_uint4(w[0], w[1], w[2], w[3]));
      }
      if (warp == 0 && tl == 0) sm.rscale[r] = scalbnf(sl2, -e2);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      if (QS) {
        if (warp == 0) sm.q[nt][i][lane] = x[i];
      } else {
        q[nt][i] = x[i];
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) p[nt][c] = base + (r0 + nt * 8 + 2 * tl + c) / g;
  }
  if (POOLQ4 || QS) __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) f[nt][c] = POOLQ4 ? sm.rscale[nt * 8 + 2 * tl + c] : sl2;

  float o[NT][D / 16][4] = {};
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;

  // This warp's pages: gw, gw + stride, ...; their block ids are fetched 32 at a time, one per lane.
  const int gw = rank * kWarps + warp, stride = share * kWarps;
  const int n = pg.n > gw ? (pg.n - gw + stride - 1) / stride : 0;
  const int64_t page_bytes = Page::page_bytes(a.Hkv), head_bytes = Page::head_bytes(kvh);
  int ids = 0;
  Page page[PG];
  const uint8_t* vhead[PG];
  int first[PG];       // first key of the page
  unsigned seen[PG];   // its keys that some row sees
  auto issue_k = [&](int i0) {  // pages i0 .. i0 + PG - 1 of the warp; i0 counts up by PG from call to call
    if ((i0 & 31) == 0) {
      const int v = gw + (i0 + lane) * stride;
      ids = i0 + lane < n ? win_block(a, b, pg.page(v)) : 0;
    }
#pragma unroll
    for (int u = 0; u < PG; ++u) {
      const int i = i0 + u;
      const int64_t at = (int64_t)__shfl_sync(0xffffffffu, ids, i & 31) * page_bytes + head_bytes;
      const int j0 = pg.page(gw + i * stride) * 16;
      unsigned bits = 0xffffu;
      if (i >= n)
        bits = 0;
      else if (!(j0 + 15 < pg.hi && (j0 >= pg.lo || j0 + 15 < pg.sinks))) {
        bits = __ballot_sync(0xffffffffu, pg.any(j0 + (lane & 15))) & 0xffffu;
      }
      seen[u] = bits;
      first[u] = i < n ? j0 : 0x3ffffff0;
      vhead[u] = (const uint8_t*)a.v_pool + at;
      page[u].load_k((const uint8_t*)a.k_pool + at, a.Hkv, gl, tl, bits);
    }
  };
  auto issue_v = [&]() {
#pragma unroll
    for (int u = 0; u < PG; ++u) page[u].load_v(vhead[u], a.Hkv, gl, tl, seen[u]);
  };
  if (n > 0) {
    issue_k(0);
    issue_v();
  }
  for (int i = 0; i < n; i += PG) {
    float x[PG][NT][4] = {};
#pragma unroll
    for (int u = 0; u < PG; ++u)
      page[u].k_steps([&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 qq = QS ? sm.q[nt][k >> 1][lane] : q[QS ? 0 : nt][k >> 1];
          mma<BF16>(x[u][nt], a0, a1, a2, a3, (k & 1) ? qq.z : qq.x, (k & 1) ? qq.w : qq.y);
        }
      });
    bool all = true;  // every row sees every key
    int j0[PG];
#pragma unroll
    for (int u = 0; u < PG; ++u) {
      j0[u] = first[u];
      all = all && j0[u] + 15 <= p_first && (a.window == 0 || j0[u] + 15 < a.sinks || p_last - j0[u] < a.window);
    }
    const bool more = i + PG < n;
    if (more) issue_k(i + PG);  // K's registers are free; V's still hold this step's
#pragma unroll
    for (int u = 0; u < PG; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[u][nt][c] *= f[nt][c & 1];
    if (!all) {
#pragma unroll
      for (int u = 0; u < PG; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            x[u][nt][c] =
                win_sees(p[nt][c & 1], j0[u] + gl + 8 * (c >> 1), a.window, a.sinks) ? x[u][nt][c] : -INFINITY;
    }
    float top[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[nt][c] = fmaxf(x[0][nt][c], x[0][nt][c + 2]);
#pragma unroll
        for (int u = 1; u < PG; ++u) top[nt][c] = ptx::max3(top[nt][c], x[u][nt][c], x[u][nt][c + 2]);
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
    uint32_t b0[PG][NT], b1[PG][NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mu[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) mu[c] = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
#pragma unroll
      for (int u = 0; u < PG; ++u) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[u][nt][c] = ptx::ex2(x[u][nt][c] - mu[c & 1]);
          l[nt][c & 1] += x[u][nt][c];
        }
        b0[u][nt] = transpose8(pack<BF16>(x[u][nt][0], x[u][nt][1]));
        b1[u][nt] = transpose8(pack<BF16>(x[u][nt][2], x[u][nt][3]));
      }
    }
#pragma unroll
    for (int u = 0; u < PG; ++u)
      page[u].v_tiles([&](int e, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma<BF16>(o[nt][e], a0, a1, a2, a3, b0[u][nt], b1[u][nt]);
      });
    if (more) issue_v();
  }

  // ---------------------------------------------------------------- merge: warps, then the cluster's CTAs
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = l[nt][c];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      const int r = nt * 8 + 2 * tl + c;
      if (gl == 0) sm.wm[warp][r] = m[nt][c], sm.wl[warp][r] = sum;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        sm.o[warp][r][Page::chan(gl, e, 0)] = o[nt][e][c];
        sm.o[warp][r][Page::chan(gl, e, 1)] = o[nt][e][c + 2];
      }
    }
  __syncthreads();
  for (int e = tid; e < rows * D; e += kThreads) {
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
      float* part = ws + ((int64_t)item_id * splits + rank) * kPartialFloats<D, NT>;
      part[r * D + c] = acc;
      if (c == 0) part[ROWS * D + r] = top, part[ROWS * (D + 1) + r] = sum;
      continue;
    }
    sm.o[0][r][c] = acc;  // read and written by this thread alone
    if (c == 0) sm.m[r] = top, sm.l[r] = sum;
  }
  if (splits > 1) return;
  win_merge_store<T, D>(&sm.o[0][0][0], DecSmem<D, NT>::kStride, sm.m, sm.l, rows, r0, g, kvh, a.Hq, row.q0, (T*)a.out,
                        tid, kThreads);
}

// Rows of the items that several CTAs share: one block per (item, row), its two halves each taking every other split.
// A programmatic dependent launch: its blocks may be in place before the attention's last CTAs are done.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(D) attn_win_combine_kernel(const PkvWinArgs a, const int splits,
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
  __shared__ float sm_w[64];
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

template <typename T, bool POOLQ4, int D, int NT>
int launch(const PkvWinArgs& a, void* workspace, size_t ws_bytes, size_t* ws_wanted, int* launches, cudaStream_t s) {
  constexpr int PG = POOLQ4 && NT <= 2 ? 2 : 1;
  auto kernel = attn_win_dec_kernel<T, POOLQ4, D, NT, PG>;
  const size_t smem = sizeof(DecSmem<D, NT>);
  static PkvKernelState state;
  int rc = pkv_prepare_kernel((const void*)kernel, (int)smem, kThreads, 0, state);
  if (rc) return rc;
  const int g = a.Hq / a.Hkv;
  const int64_t items = (int64_t)a.B * a.Hkv * (((int64_t)a.max_query_len * g + 8 * NT - 1) / (8 * NT));
  const int64_t steps = pkv_visible_keys(a, 8 * NT / g + 1) / (16 * kWarps) + 1;
  // Items too few for clusters of 16 to fill the GPU: more CTAs per item, and the combine launch.
  int splits = pkv_plan_splits(state, items, steps, 4.0, 3.0);
  const size_t need = splits > 1 ? (size_t)(items * splits * kPartialFloats<D, NT> * 4) : 0;
  if (ws_wanted) {
    *ws_wanted = need;
    return 0;
  }
  if (need > ws_bytes || !workspace) splits = 1;
  float* ws = splits > 1 ? (float*)workspace : nullptr;
  void* args[] = {const_cast<PkvWinArgs*>(&a), &splits, &ws};
  const int ctas = splits > 1 ? 1 : pkv_plan_cluster(state, items, steps, 4.0);
  *launches = 1;
  rc = pkv_launch_cluster((const void*)kernel, splits > 1 ? items * splits : items, ctas, kThreads, smem, args, false, s);
  if (rc || splits == 1) return rc;
  *launches = 2;
  return pkv_launch_cluster((const void*)attn_win_combine_kernel<T, D, NT>, items * 8 * NT, 1, D, 0, args, true, s);
}

template <typename T, bool POOLQ4, int D>
int launch_rows(const PkvWinArgs& a, void* ws, size_t bytes, size_t* wanted, int* launches, cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_query_len * (a.Hq / a.Hkv);
  if (rows <= 8) return launch<T, POOLQ4, D, 1>(a, ws, bytes, wanted, launches, s);
  if (rows <= 16) return launch<T, POOLQ4, D, 2>(a, ws, bytes, wanted, launches, s);
  return launch<T, POOLQ4, D, 4>(a, ws, bytes, wanted, launches, s);
}

template <typename T>
int launch_pool(const PkvWinArgs& a, int D, bool q4, void* ws, size_t bytes, size_t* wanted, int* launches,
                cudaStream_t s) {
  if (q4)
    return D == 64 ? launch_rows<T, true, 64>(a, ws, bytes, wanted, launches, s)
                   : launch_rows<T, true, 128>(a, ws, bytes, wanted, launches, s);
  return D == 64 ? launch_rows<T, false, 64>(a, ws, bytes, wanted, launches, s)
                 : launch_rows<T, false, 128>(a, ws, bytes, wanted, launches, s);
}

}  // namespace

int pkv_launch_win_dec(const PkvWinArgs& a, pkv_dtype dt, int D, bool q4, void* workspace, size_t ws_bytes,
                       size_t* ws_wanted, int* launches, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  if (dt == PKV_BF16) return launch_pool<__nv_bfloat16>(a, D, q4, workspace, ws_bytes, ws_wanted, launches, s);
  if (dt == PKV_F16) return launch_pool<__half>(a, D, q4, workspace, ws_bytes, ws_wanted, launches, s);
  return (int)cudaErrorInvalidValue;
}
