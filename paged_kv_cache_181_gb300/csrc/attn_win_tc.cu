// Window/sinks attention for many query rows per kv head (prompts and prompt chunks), bf16/f16 queries over 16-bit
// or 4-bit pools: tcgen05 products with TMEM accumulators, fp32 online softmax.
//
// One CTA = two 128-row tiles of packed query rows (attn_win.cuh: floor(128 / g) tokens x g heads of one kv head a
// tile), which share every key and value tile.  Packing the heads that share keys shortens the stretch of
// positions a tile spans, and with it the keys that only some of its rows see: with a window of 1024 and g = 4, 256
// rows are 64 positions and visit 1024 + 64 keys, where 256 positions of one head would visit 1024 + 256.
// The CTAs of a cluster take parts of an item's key tiles and merge through shared memory: it evens out the last
// wave and fills the GPU when there are few items.
//
// Key tiles are eight of the pages that some row sees (WinPages), so the keys between the sinks and the window are
// skipped at page granularity; what a row does not see inside a page is masked in its scores.  Values that no row
// sees are zero in shared memory (0 * NaN would not be).
//
// Warps: 1 issues the MMAs and owns TMEM; 4-7 and 8-11 are the softmax of the two tiles, one row per thread; and
//   16-bit pools: 0 loads Q and the key tiles by TMA (one box per page), 3 the value tiles;
//   4-bit pools:  0 copies whole records to shared memory, 2, 3 and 12-15 turn their codes into the fp16 numbers they
//                 stand for and store them swizzled as TMA would; Q is converted to fp16 by the softmax threads, each
//                 row scaled by a power of two.  Channels of a code word come out as (0,4), (1,5), (2,6), (3,7): Q's
//                 and the output's channels are permuted to match, which is free, instead of the codes.
// CTAs are persistent: warp 0 asks the hardware for a CTA that has not started yet, cancels its launch and takes its
// item (clusterlaunchcontrol), and the roles go on to it each at its own pace: the producers load the next item's
// keys and queries while the softmax warps finish the last one.  8192 tokens x 32 heads over 8 kv heads, D = 128, with a
// window of 64: 46 us instead of 69 with a CTA an item; window 1024: 141 instead of 163.  (Clusters keep to their item.)
//
// What bounds it: a tile's chain of hand-overs.  Its probabilities overwrite its scores in TMEM (two score and two output
// accumulators fill it at D = 128), so scores, softmax, products and the barriers between them follow one another, 3300
// cycles for 128 keys, and only the other tile's work fills the gaps: 1.19 PFLOP/s over 4000-key windows, 0.97 with 4-bit
// pools.  With work taken out: no exponentials 0 % faster, no products 11 %, no loads 5 %.
// Scores of 64 keys that go on by themselves were slower (a TMEM read is mostly latency, and there were twice as many),
// and so were two threads a row (the maxima have to be exchanged: 147 us for two prompts of up to 4096 tokens with a
// window of 1024, against 135).
// The order of MMAs, the ring of slots shared by key and value tiles, the lazy rescale and the register split between
// warpgroups are those of the prefix-mask kernel (attn_tc.cu), which says why.
// Every mbarrier wait is bounded in time (1 s, or 60 for the next item); on expiry the CTA records PKV_DEVERR_TIMEOUT
// and unwinds.

#include <cuda.h>

#include <atomic>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "attn_win.cuh"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int BM = 128;  // rows per tile; two tiles per CTA
constexpr int BN = 128;  // keys per tile
constexpr int kPages = BN / 16;
// Threads, and registers per thread: as compiled (checked at build and launch), and after the split between the
// producer/MMA warpgroups and the two softmax ones.
constexpr int kLaunchRegs = 168, kLaunchRegsQ4 = 128;
template <bool POOLQ4>
struct Roles {
  static constexpr int kThreads = POOLQ4 ? 512 : 384;
  static constexpr int kRegs = POOLQ4 ? kLaunchRegsQ4 : kLaunchRegs;
  static constexpr int kLow = POOLQ4 ? 72 : 136, kHigh = POOLQ4 ? 184 : 184;
  static_assert((kThreads - 256) * kLow + 256 * kHigh == kThreads * kRegs, "register split must add up");
};
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr uint64_t kItemLimitNs = 60 * kWaitLimitNs;  // of a role without work in an item: 2^31 keys take 30 s
constexpr float kRescale = 8.f;  // log2 units
constexpr int kDequantWarps = 6;
constexpr int kAskAhead = 4;  // key tiles an item has left to load when its CTA asks for the next one
constexpr double kFixedTiles = 4.0;  // a CTA's set-up and epilogue, in key tiles of its time (1 to 4 plan alike)

template <int D, bool POOLQ4>
struct Cfg {
  static constexpr int TILE = BN * D * 2;
  static constexpr int NSLOT = (POOLQ4 ? 4 : 5) * (128 / D);
  static constexpr int NRAW = POOLQ4 ? 3 : 0;             // 4-bit tiles in flight
  static constexpr int RAW = kPages * Q4<D>::kRecord;     // one of them
  static constexpr int GS = (D / 64) * 1024;  // stride of 8-row atoms in a key/value tile
  // The probabilities of a tile are handed over in two parts, so that the products of the first one overlap the
  // exponentials of the second (2 % over 4000-key windows); with 4-bit pools in one, where two lost 5 %.
  static constexpr int PARTS = POOLQ4 ? 1 : 2;
  static constexpr int OSTRIDE = D + 4;       // floats between rows staged for the merge
};

// An item as its CTA works on it.
struct Item {
  int n;        // key tiles of this CTA; -1: no more items
  int t_begin;  // the first of them
  int q0, Sq, kvh, b;
  int i0, n_q;  // first local query token; tiles with rows
  int base;     // position of local query 0
  WinPages pg;
};

template <int D, bool POOLQ4>
struct alignas(1024) WinSmem {
  using C = Cfg<D, POOLQ4>;
  uint8_t q[2][BM * D * 2];       // [D/64][128 rows][128 B] per tile, 128-byte swizzled
  uint8_t kv[C::NSLOT][C::TILE];  // [page][8-row group][column half][8 rows][128 B], swizzled
  uint8_t raw[POOLQ4 ? C::NRAW : 1][POOLQ4 ? C::RAW : 16];  // records of 4-bit tiles
  uint64_t full[C::NSLOT], empty[C::NSLOT];
  uint64_t raw_full[3], raw_empty[3];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2];  // p_full: [query tile][part of the keys]
  uint64_t info_full[2], info_empty[2], clc_full, tile_sync[2];
  alignas(16) uint4 clc;  // the scheduler's last answer
  Item info[2];           // the item in work, and the one to come
  uint32_t tmem_base;
  int abort, skip;
  // The merge stages 2 BM rows of OSTRIDE floats from kv on.
  static_assert(2 * BM * C::OSTRIDE * 4 <= C::NSLOT * C::TILE + C::NRAW * C::RAW, "merge rows fit");
};
static_assert(sizeof(WinSmem<128, false>) + 1024 <= 227 * 1024 && sizeof(WinSmem<128, true>) + 1024 <= 227 * 1024,
              "shared memory of a CTA");

struct WinMaps {
  CUtensorMap q, o;    // (D, g, Hkv, Tq), box = 64 columns x g heads x a tile's tokens
  CUtensorMap kb, vb;  // pools as (64, 8, D/64, slots/8, Hkv), box = one 16-row page of one head
  CUtensorMap v1;      // pool as (D, Hkv, slots), box = 64 columns of one row
};

template <int D>
__host__ __device__ constexpr int row_offset(int r, int dh) {
  return (r >> 3) * ((D / 64) * 1024) + dh * 1024 + (r & 7) * 128;
}

PKV_DEVINLINE void tma_load_4d(void* dst, const void* tmap, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(ptx::smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(ptx::smem_u32(bar))
      : "memory");
}
PKV_DEVINLINE void tma_store_4d(const void* tmap, int c0, int c1, int c2, int c3, const void* src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(tmap),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(ptx::smem_u32(src))
               : "memory");
}

// Bytes [src, src + n) of global memory to shared memory, counted on `bar`; all multiples of 16.
PKV_DEVINLINE void bulk_load(void* dst, const void* src, uint32_t n, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(src), "r"(n), "r"(ptx::smem_u32(bar))
               : "memory");
}

template <typename Smem>
PKV_DEVINLINE void note_abort(Smem& sm, unsigned int* err) {
  sm.abort = 1;
  pkv_raise(err, PKV_DEVERR_TIMEOUT);
}

PKV_DEVINLINE bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int lane,
                             uint64_t limit = kWaitLimitNs) {
  bool ok = true;
  if (lane == 0) ok = ptx::mbar_wait(bar, parity, abort, limit);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// Lane k < 8: block of page k of key tile kt.
PKV_DEVINLINE int tile_block(const PkvWinArgs& a, const WinPages& pg, int b, int kt, int lane) {
  const int v = kPages * kt + lane;
  return lane < kPages && v < pg.n ? win_block(a, b, pg.page(v)) : 0;
}

// Which keys of a page some row sees, a bit each.  (Key by key it took the value loader 2000 to 4600 cycles a tile, more
// than all that a tile needs else.)
PKV_DEVINLINE unsigned seen_keys(const WinPages& pg, int page) {
  const int j0 = page * 16;
  auto below = [&](int j) { return j <= j0 ? 0u : j - j0 >= 16 ? 0xffffu : (1u << (j - j0)) - 1u; };  // keys under j
  return below(pg.hi) & (~below(pg.lo) | below(pg.sinks)) & 0xffffu;
}

// One warp loads a 16-bit key or value tile: pages [8 kt, 8 kt + 8) of the item's list, a lane per page (block `blk`).
template <int D>
PKV_DEVINLINE void load_tile(uint8_t* dst, const WinMaps& maps, bool is_v, uint64_t* full, const PkvWinArgs& a,
                             const WinPages& pg, int blk, int kvh, int kt, int lane) {
  const int v = kPages * kt + lane;
  const bool there = lane < kPages && v < pg.n;
  const int page = there ? pg.page(v) : 0;
  unsigned seen = there ? 0xffffu : 0u;  // rows of the page that some query sees
  if (is_v && there) seen = seen_keys(pg, page);
  if (is_v && __any_sync(0xffffffffu, lane < kPages && seen != 0xffffu)) {
    // Unseen value rows are zeroed; whole 128-byte rows, so the swizzle does not matter.
    for (int k = 0; k < kPages; ++k) {
      const unsigned bits = __shfl_sync(0xffffffffu, seen, k);
      if (bits == 0xffffu) continue;
      for (int e = lane; e < 16 * (D / 64) * 8; e += 32) {
        const int c = e & 7, dh = (e >> 3) % (D / 64), r = (e >> 3) / (D / 64);
        if (!((bits >> r) & 1))
          *reinterpret_cast<uint4*>(dst + row_offset<D>(16 * k + r, dh) + c * 16) = make_uint4(0, 0, 0, 0);
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
  }
  const int rows = __reduce_add_sync(0xffffffffu, __popc(seen));
  if (lane == 0) ptx::mbar_arrive_expect_tx(full, (uint32_t)(rows * D * 2));
  __syncwarp();
  if (seen == 0xffffu) {
    ptx::tma_load_5d(dst + row_offset<D>(16 * lane, 0), is_v ? &maps.vb : &maps.kb, 0, 0, 0, blk * 2, kvh, full);
  } else if (seen) {
    for (int r = 0; r < 16; ++r)
      if ((seen >> r) & 1)
#pragma unroll
        for (int dh = 0; dh < D / 64; ++dh)
          ptx::tma_load_3d(dst + row_offset<D>(16 * lane + r, dh), &maps.v1, dh * 64, kvh, blk * 16 + r, full);
  }
}

// Ask for the launch of a CTA that has not started to be cancelled: 16 bytes of answer at `dst`, counted on `bar`.
PKV_DEVINLINE void clc_try_cancel(void* dst, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          ptx::smem_u32(dst)),
      "r"(ptx::smem_u32(bar))
      : "memory");
}
// Whether the answer holds a cancelled CTA, and its blockIdx.x.
PKV_DEVINLINE bool clc_answer(const void* src, uint32_t* cta) {
  uint32_t ok, x;
  asm volatile(
      "{\n"
      ".reg .b128 r;\n"
      ".reg .pred p;\n"
      "ld.shared.b128 r, [%2];\n"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "mov.u32 %1, 0;\n"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n"
      "}\n"
      : "=r"(ok), "=r"(x)
      : "r"(ptx::smem_u32(src))
      : "memory");
  *cta = x;
  return ok != 0;
}

// Item u of the grid for this CTA (its cluster's rank); false: no queries there.
// Items with the latest queries (the most keys) come first; the kv heads of one stretch of queries run together.
PKV_DEVINLINE bool decode_item(const PkvWinArgs& a, uint32_t u, Item& it) {
  const int g = a.Hq / a.Hkv, TM = BM / g;  // tokens per tile
  const int n_qp = (a.max_query_len + 2 * TM - 1) / (2 * TM);
  it.kvh = u % a.Hkv;
  u /= a.Hkv;
  it.b = u % a.B;
  const int qp = n_qp - 1 - (int)(u / a.B);
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  const WinRow row = win_row(a, it.b, qp == 0 && it.kvh == 0 && rank == 0);
  it.q0 = row.q0;
  it.Sq = row.Sq;
  it.i0 = qp * 2 * TM;
  if (it.i0 >= row.Sq) return false;
  it.n_q = it.i0 + TM < row.Sq ? 2 : 1;
  it.base = row.L - row.Sq;
  const int last = row.Sq < it.i0 + 2 * TM ? row.Sq : it.i0 + 2 * TM;  // one past the item's last token
  it.pg = win_pages(it.base + it.i0, it.base + last - 1, a.window, a.sinks);
  const int n_tiles = (it.pg.n + kPages - 1) / kPages;
  const int per = (n_tiles + (int)n_cta - 1) / (int)n_cta;
  it.t_begin = (int)rank * per;
  const int t_end = n_tiles < it.t_begin + per ? n_tiles : it.t_begin + per;
  it.n = t_end > it.t_begin ? t_end - it.t_begin : 0;
  return true;
}

template <int D, typename T, bool OPBF16, bool POOLQ4>
__global__ void __launch_bounds__(Roles<POOLQ4>::kThreads, 1)
    attn_win_tc_kernel(const __grid_constant__ WinMaps maps, const PkvWinArgs a, const uint32_t first_item) {
  using C = Cfg<D, POOLQ4>;
  constexpr int kThreads = Roles<POOLQ4>::kThreads;
  constexpr bool OUTBF16 = !std::is_same<T, __half>::value;
  constexpr int kReaders = POOLQ4 ? 16 : 11;  // warps that read an item (with 16-bit pools warp 2 has no work)
  extern __shared__ uint8_t smem_raw[];
  using Smem = WinSmem<D, POOLQ4>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.Hq / a.Hkv;
  const int TM = BM / g;  // tokens per tile
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  // A second launch, for the items behind whole waves, may start as soon as this one's last CTAs run.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool is_softmax = warp >= 4 && warp < 12;

  if (tid == 0) {
    for (int s = 0; s < C::NSLOT; ++s) {
      ptx::mbar_init(&sm.full[s], POOLQ4 ? kDequantWarps : 1);
      ptx::mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 3; ++s) {
      ptx::mbar_init(&sm.raw_full[s], 1);
      ptx::mbar_init(&sm.raw_empty[s], kDequantWarps);
    }
    for (int w = 0; w < 2; ++w) {
      ptx::mbar_init(&sm.q_full[w], POOLQ4 ? 128 : 1);
      ptx::mbar_init(&sm.s_full[w], 1);
      ptx::mbar_init(&sm.p_full[w][0], 128);
      ptx::mbar_init(&sm.p_full[w][1], 128);
      ptx::mbar_init(&sm.q_empty[w], 1);
      ptx::mbar_init(&sm.o_full[w], 1);
      ptx::mbar_init(&sm.info_full[w], 1);
      ptx::mbar_init(&sm.info_empty[w], kReaders);
    }
    ptx::mbar_init(&sm.clc_full, 1);
    for (int w = 0; w < 2; ++w) ptx::mbar_init(&sm.tile_sync[w], 4);
    sm.abort = 0;
    // After a pipeline timeout in an earlier launch results are invalid: do not wait for it again.
    sm.skip = (*(volatile unsigned int*)a.err & PKV_DEVERR_TIMEOUT) != 0;
    ptx::fence_mbar_init();
  }
  Item mine;
  mine.n = -1;
  bool there = false;
  if (warp == 0 && lane == 0) there = decode_item(a, first_item + blockIdx.x / n_cta, mine);
  if (!POOLQ4 && warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.q);
    ptx::prefetch_tmap(&maps.kb);
    ptx::prefetch_tmap(&maps.vb);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&sm.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();

  const uint32_t tmem = sm.tmem_base;
  const bool skip = sm.skip != 0;
  constexpr uint32_t O_COL[2] = {256, 256 + D};
  constexpr uint32_t IDESC_QK = ptx::idesc_f16(BM, BN, OPBF16 ? 1 : 0, 0);
  constexpr uint32_t IDESC_PV = ptx::idesc_f16(BM, D, OPBF16 ? 1 : 0, 1);

  // Every role walks the items: wait for the next one, work, hand its place back.  All lanes call both.
  int seq = 0;
  auto next_item = [&]() -> bool {
    const bool ok = warp_wait(&sm.info_full[seq & 1], (seq >> 1) & 1, &sm.abort, lane, kItemLimitNs);
    if (!ok) {
      if (lane == 0) note_abort(sm, a.err);
      return false;
    }
    __syncwarp();
    return sm.info[seq & 1].n >= 0;
  };
  auto done_item = [&]() {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sm.info_empty[seq & 1]);
    ++seq;
  };
  int tb = 0;  // key tiles of the items before this one: the ring goes on over them

  if (!is_softmax) {
    ptx::regs_dec<Roles<POOLQ4>::kLow>();
    // Scheduling, by one lane: publish the item in hand, then find the next one.  It is asked for when kAskAhead tiles
    // of this item are left to load: an item that is claimed earlier may wait here while another SM falls idle
    // (2048 queries over 16384 keys, 128 tiles an item: asked for at the start 674 us, so 556).
    bool have = true, pending = false;
    uint32_t answers = 0;
    int published = 0;
    auto ask = [&]() {
      if (!have || pending || n_cta > 1) return;
      ptx::mbar_arrive_expect_tx(&sm.clc_full, 16);
      clc_try_cancel(&sm.clc, &sm.clc_full);
      pending = true;
    };
    auto publish = [&]() -> bool {  // the item in hand, or that there is none
      if (!have || there) {
        const int slot = published & 1;
        if (published >= 2 && !ptx::mbar_wait(&sm.info_empty[slot], ((published >> 1) - 1) & 1, &sm.abort, kItemLimitNs))
          return false;
        if (!have)
          mine.n = -1;
        else if (skip)
          mine.n = 0;
        sm.info[slot] = mine;
        ptx::mbar_arrive(&sm.info_full[slot]);
        ++published;
      }
      return true;
    };
    auto advance = [&]() -> bool {  // the next item in hand
      if (n_cta > 1) {
        have = false;
        return true;
      }
      ask();
      if (!ptx::mbar_wait(&sm.clc_full, answers & 1, &sm.abort, kWaitLimitNs)) return false;
      ++answers;
      pending = false;
      uint32_t cta = 0;
      have = clc_answer(&sm.clc, &cta);
      ptx::fence_proxy_async_smem();  // read before the next answer is written
      if (have) there = decode_item(a, first_item + cta, mine);
      return true;
    };
    auto finish = [&]() {  // an answer under way must land before the shared memory goes away
      int never = 0;
      if (pending) ptx::mbar_wait(&sm.clc_full, answers & 1, &never, kWaitLimitNs);
    };
    // Until an item is published (the first, and each one that the last step found).
    auto schedule = [&](bool first) -> bool {
      bool ok = true;
      if (lane == 0) {
        if (!first) ok = advance();
        while (ok) {
          const int before = published;
          ok = publish();
          if (!ok || published > before) break;  // (an item without queries is passed over)
          ok = advance();
        }
        if (!ok) note_abort(sm, a.err);
      }
      return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    };
    if (!POOLQ4 && (warp == 0 || warp == 3)) {
      // ------------------------------------------------------------ producers: warp 0 Q and key tiles, warp 3 value tiles
      int loaded[2] = {0, 0};  // Q tiles
      bool go = warp == 3 || schedule(true);
      while (go && next_item()) {
        const Item& it = sm.info[seq & 1];
        const int n = it.n;
        const WinPages pg = it.pg;
        int blk = n > 0 ? tile_block(a, pg, it.b, it.t_begin, lane) : 0;  // fetched a tile ahead
        bool ok = true;
        if (warp == 0 && n > 0) {
          for (int t = 0; t < it.n_q && ok; ++t) {
            // The score MMAs of the tile's last item must be done with its place.
            if (loaded[t] > 0 && !warp_wait(&sm.q_empty[t], (loaded[t] - 1) & 1, &sm.abort, lane)) {
              if (lane == 0) note_abort(sm, a.err);
              ok = false;
              break;
            }
            if (lane == 0) {
              ptx::mbar_arrive_expect_tx(&sm.q_full[t], (uint32_t)(TM * g * D * 2));
#pragma unroll
              for (int dh = 0; dh < D / 64; ++dh)  // tokens past the last one read as zeros
                tma_load_4d(sm.q[t] + dh * (BM * 128), &maps.q, dh * 64, 0, it.kvh, it.q0 + it.i0 + t * TM, &sm.q_full[t]);
            }
            ++loaded[t];
          }
          if (!ok) break;
        }
        for (int j = 0; j < n; ++j) {
          if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort != 0)) {
            ok = false;
            break;
          }
          if (warp == 0 && lane == 0 && j + kAskAhead >= n) ask();
          const int idx = 2 * (tb + j) + (warp == 3 ? 1 : 0);
          const int pos = idx % C::NSLOT, use = idx / C::NSLOT;
          if (use > 0 && !warp_wait(&sm.empty[pos], (use - 1) & 1, &sm.abort, lane)) {
            if (lane == 0) note_abort(sm, a.err);
            ok = false;
            break;
          }
          const int ahead = j + 1 < n ? tile_block(a, pg, it.b, it.t_begin + j + 1, lane) : 0;
          load_tile<D>(sm.kv[pos], maps, warp == 3, &sm.full[pos], a, pg, blk, it.kvh, it.t_begin + j, lane);
          blk = ahead;
        }
        if (!ok) break;
        tb += n;
        done_item();
        if (warp == 0) go = schedule(false);
      }
      if (warp == 0 && lane == 0) finish();
      if (warp == 0 && *(volatile int*)&sm.abort && lane == 0) {
        int never = 0;  // let copies already issued land before the shared memory goes away
        for (int t = 0; t < 2; ++t)
          if (loaded[t]) ptx::mbar_wait(&sm.q_full[t], (loaded[t] - 1) & 1, &never, kWaitLimitNs);
      }
    } else if (POOLQ4 && warp == 0) {
      // ------------------------------------------------------------ 4-bit tiles: a lane per page copies its record
      bool go = schedule(true);
      while (go && next_item()) {
        const Item& it = sm.info[seq & 1];
        const int n = it.n;
        const WinPages pg = it.pg;
        bool ok = true;
        int ids = n > 0 ? tile_block(a, pg, it.b, it.t_begin, lane) : 0, ids_next = 0;  // fetched a tile ahead
        for (int i = 0; i < 2 * n; ++i) {
          if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort != 0)) {
            ok = false;
            break;
          }
          if (lane == 0 && i + 2 * kAskAhead >= 2 * n) ask();
          const int idx = 2 * tb + i;
          const int v = kPages * (it.t_begin + (i >> 1)) + lane;
          const bool page = lane < kPages && v < pg.n;
          if (i & 1)
            ids_next = (i >> 1) + 1 < n ? tile_block(a, pg, it.b, it.t_begin + (i >> 1) + 1, lane) : 0;
          else if (i > 0)
            ids = ids_next;
          const int pos = idx % 3, use = idx / 3;
          if (use > 0 && !warp_wait(&sm.raw_empty[pos], (use - 1) & 1, &sm.abort, lane)) {
            if (lane == 0) note_abort(sm, a.err);
            ok = false;
            break;
          }
          const int pages = __popc(__ballot_sync(0xffffffffu, page));
          if (lane == 0) ptx::mbar_arrive_expect_tx(&sm.raw_full[pos], (uint32_t)(pages * Q4<D>::kRecord));
          __syncwarp();
          if (page)
            bulk_load(sm.raw[POOLQ4 ? pos : 0] + lane * Q4<D>::kRecord,
                      (const uint8_t*)((i & 1) ? a.v_pool : a.k_pool) + ((int64_t)ids * a.Hkv + it.kvh) * Q4<D>::kRecord,
                      Q4<D>::kRecord, &sm.raw_full[pos]);
        }
        if (!ok) break;
        tb += n;
        done_item();
        go = schedule(false);
      }
      if (lane == 0) finish();
      if (*(volatile int*)&sm.abort && lane == 0) {
        // Let copies already issued land before the shared memory goes away.
        int never = 0;
        for (int s = 0; s < 3; ++s) ptx::mbar_wait(&sm.raw_full[s], 0, &never, 1000000ull);
        for (int s = 0; s < 3; ++s) ptx::mbar_wait(&sm.raw_full[s], 1, &never, 1000000ull);
      }
    } else if (POOLQ4 && warp != 1) {
      // ------------------------------------------------------------ 4-bit tiles: codes to fp16, swizzled as TMA would
      // A lane takes one group of 32 channels of one key: 16 bytes of codes in, four 16-byte chunks out.  A warp's
      // piece is 32 / (D/32) keys of all groups, so its reads are contiguous; which of the four chunks a lane stores
      // first depends on its key and group such that the eight lanes of a store phase hit different banks.  The
      // pieces of a slot are dealt out in turn, starting with another warp for each slot.
      using F = Q4<D>;
      constexpr int G = F::kGroups, KEYS = 32 / G;
      constexpr int MINE = (BN / KEYS + kDequantWarps - 1) / kDequantWarps;
      const int pw = warp < 4 ? warp - 2 : warp - 10;
      const int gi = lane % G, rk = lane / G;
      const int x = D == 128 ? (gi >> 1) | ((rk & 1) << 1) : 0;  // chunk order: 0^x, 1^x, 2^x, 3^x
      while (next_item()) {
        const Item& it = sm.info[seq & 1];
        const int n = it.n, t_begin = it.t_begin;
        const WinPages pg = it.pg;
        bool ok = true;
        for (int i = 0; i < 2 * n; ++i) {
          if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort != 0)) {
            ok = false;
            break;
          }
          const int idx = 2 * tb + i;
          const int pos = idx % C::NSLOT, use = idx / C::NSLOT, rpos = idx % 3;
          if (!warp_wait(&sm.raw_full[rpos], (idx / 3) & 1, &sm.abort, lane)) {
            if (lane == 0) note_abort(sm, a.err);
            ok = false;
            break;
          }
          // All of the warp's codes first: the reads overlap each other and the wait for the slot.
          const uint8_t* raw = sm.raw[POOLQ4 ? rpos : 0];
          const int p0 = (pw + idx) % kDequantWarps;
          uint4 code[MINE];
          uint32_t pair[MINE];
#pragma unroll
          for (int k = 0; k < MINE; ++k) {
            const int r = (p0 + k * kDequantWarps) * KEYS + rk;  // key of the tile
            const int v = kPages * (t_begin + (i >> 1)) + (r >> 4);
            code[k] = make_uint4(0, 0, 0, 0);
            pair[k] = 0;  // keys that no row sees are zeros
            if (r < BN && v < pg.n && pg.any(pg.page(v) * 16 + (r & 15))) {
              const uint8_t* rec = raw + (r >> 4) * F::kRecord;
              code[k] = *reinterpret_cast<const uint4*>(rec + (r & 15) * F::kRowBytes + gi * 16);
              pair[k] = *reinterpret_cast<const uint32_t*>(rec + F::kPairs + ((r & 15) * G + gi) * 4);
            }
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sm.raw_empty[rpos]);
          if (use > 0 && !warp_wait(&sm.empty[pos], (use - 1) & 1, &sm.abort, lane)) {
            if (lane == 0) note_abort(sm, a.err);
            ok = false;
            break;
          }
#pragma unroll
          for (int k = 0; k < MINE; ++k) {
            const int r = (p0 + k * kDequantWarps) * KEYS + rk;
            if (r >= BN) break;
            const uint32_t y0 = (x & 1) ? code[k].y : code[k].x, y1 = (x & 1) ? code[k].x : code[k].y;
            const uint32_t y2 = (x & 1) ? code[k].w : code[k].z, y3 = (x & 1) ? code[k].z : code[k].w;
            const uint32_t words[4] = {(x & 2) ? y2 : y0, (x & 2) ? y3 : y1, (x & 2) ? y0 : y2, (x & 2) ? y1 : y3};
            uint8_t* dst = sm.kv[pos] + row_offset<D>(r, gi >> 1);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              __half2 h[4];
              q4_values(words[w], *reinterpret_cast<const __half2*>(&pair[k]), h);
              *reinterpret_cast<uint4*>(dst + ((((gi & 1) * 4 + (w ^ x)) ^ (r & 7)) << 4)) =
                  make_uint4(*reinterpret_cast<uint32_t*>(&h[0]), *reinterpret_cast<uint32_t*>(&h[1]),
                             *reinterpret_cast<uint32_t*>(&h[2]), *reinterpret_cast<uint32_t*>(&h[3]));
            }
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sm.full[pos]);
        }
        if (!ok) break;
        tb += n;
        done_item();
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer (lane 0; the warp walks the items together)
      const uint32_t kv_base = ptx::smem_u32(sm.kv[0]);
      const uint64_t q_desc[2] = {ptx::smem_desc(ptx::smem_u32(sm.q[0]), 16, 1024, 2),
                                  ptx::smem_desc(ptx::smem_u32(sm.q[1]), 16, 1024, 2)};
      const uint64_t k_desc = ptx::smem_desc(kv_base, 16, C::GS, 2);
      const uint64_t v_desc = ptx::smem_desc(kv_base, 1024, C::GS, 2);
      int qc[2] = {0, 0}, pc[2] = {0, 0}, oc[2] = {0, 0};  // phases of q_full, p_full, o_full
      int kpos = 0, kphase = 0;  // ring slot of the next key tile, and the phase that fills it
      bool ok = true, primed = false;  // primed: tile 0's first scores of this item are under way
      while (next_item()) {
        const int n = sm.info[seq & 1].n, n_q = sm.info[seq & 1].n_q;
        if (lane == 0 && n > 0) {
          auto ready = [&](int pos, int phase) -> bool {
            if (!ptx::mbar_wait(&sm.full[pos], phase, &sm.abort, kWaitLimitNs)) return false;
            ptx::tc_fence_after();
            return true;
          };
          auto qk = [&](int w, uint64_t kd) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              ptx::mma_ss(tmem + 128 * w, ptx::desc_add(q_desc[w], ((ks >> 2) * (BM * 128) + (ks & 3) * 32) >> 4),
                          ptx::desc_add(kd, ((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), IDESC_QK, ks > 0);
            ptx::mma_commit(&sm.s_full[w]);
          };
          auto pv = [&](int w, int h, uint64_t vd, uint32_t more) {  // part h of the tile's keys
#pragma unroll
            for (int ks = h * (BN / 16 / C::PARTS); ks < (h + 1) * (BN / 16 / C::PARTS); ++ks)
              ptx::mma_ts(tmem + O_COL[w], tmem + 128 * w + ks * 8, ptx::desc_add(vd, (ks * 2 * C::GS) >> 4), IDESC_PV,
                          ks > 0 ? 1u : more);
          };
          // The slots of this tile's values and the next tile's keys are worked out before the probabilities are waited
          // for: from then on every instruction delays the tensor core.
          ok = ready(kpos, kphase);
          for (int w = primed ? 1 : 0; w < n_q && ok; ++w) {
            ok = ptx::mbar_wait(&sm.q_full[w], qc[w] & 1, &sm.abort, kWaitLimitNs);
            ptx::tc_fence_after();
            ++qc[w];
            if (ok) qk(w, ptx::desc_add(k_desc, (uint32_t)(kpos * C::TILE) >> 4));
          }
          primed = false;
          for (int j = 0; ok && j < n; ++j) {
            const bool next = j + 1 < n;
            int vpos = kpos + 1, vphase = kphase;
            if (vpos == C::NSLOT) vpos = 0, vphase ^= 1;
            kpos += 2;
            if (kpos >= C::NSLOT) kpos -= C::NSLOT, kphase ^= 1;  // the next key tile's, of this item or the next
            const uint64_t vd = ptx::desc_add(v_desc, (uint32_t)(vpos * C::TILE) >> 4);
            const uint64_t kd = ptx::desc_add(k_desc, (uint32_t)(kpos * C::TILE) >> 4);
            if (!ready(vpos, vphase)) {
              ok = false;
              break;
            }
            for (int w = 0; w < n_q && ok; ++w) {
#pragma unroll
              for (int h = 0; h < C::PARTS; ++h) {
                if (!ptx::mbar_wait(&sm.p_full[w][h], pc[w] & 1, &sm.abort, kWaitLimitNs)) {
                  ok = false;
                  break;
                }
                ptx::tc_fence_after();
                pv(w, h, vd, j > 0 ? 1u : 0u);
              }
              if (!ok) break;
              ++pc[w];
              if (next) {
                if (w == 0 && !ready(kpos, kphase)) {
                  ok = false;
                  break;
                }
                qk(w, kd);
                continue;
              }
              ptx::mma_commit(&sm.o_full[w]);
              ++oc[w];
              // While tile 1's softmax still works on this item, tile 0's scores of the next one, if all is in place.
              if (w == 0 && n_q == 2 && ptx::mbar_try_wait(&sm.info_full[(seq + 1) & 1], ((seq + 1) >> 1) & 1) &&
                  sm.info[(seq + 1) & 1].n > 0 && ptx::mbar_try_wait(&sm.q_full[0], qc[0] & 1) &&
                  ptx::mbar_try_wait(&sm.full[kpos], kphase)) {
                ptx::tc_fence_after();
                ++qc[0];
                qk(0, kd);
                primed = true;
              }
            }
          }
          if (!ok) {
            note_abort(sm, a.err);
            ptx::mma_commit(&sm.o_full[0]);
            ++oc[0];
          }
        }
        if (!__all_sync(0xffffffffu, ok)) break;
        tb += n;
        done_item();
      }
      if (lane == 0) {
        int never = 0;  // everything issued must finish before TMEM is released
        for (int w = 0; w < 2; ++w)
          if (oc[w] > 0) ptx::mbar_wait(&sm.o_full[w], (oc[w] - 1) & 1, &never, kWaitLimitNs);
      }
    }
  } else {
    ptx::regs_inc<Roles<POOLQ4>::kHigh>();
    // ------------------------------------------------------------ softmax: warps 4-7 rows of tile 0, warps 8-11 of tile 1
    const int grp = warp >= 8 ? 1 : 0, quarter = warp & 3;
    const int trow = quarter * 32 + lane;  // row of the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t S_COL = 128 * grp;
    int sc = 0, oc = 0;   // phases of s_full[grp], o_full[grp]
    int staged = -1;      // (row 0) the slot that the last item's output leaves through
    auto release_staged = [&]() {
      if (staged < 0) return;
      ptx::bulk_wait_read_all();
      ptx::mbar_arrive(&sm.empty[staged]);
      staged = -1;
    };
    // All warps of the tile; on an mbarrier, because a warp that gave up elsewhere does not come.
    int syncs = 0;
    auto tile_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.tile_sync[grp]);
      return __all_sync(0xffffffffu, ptx::mbar_wait(&sm.tile_sync[grp], syncs++ & 1, &sm.abort, kWaitLimitNs));
    };
    while (next_item()) {
      const Item& it = sm.info[seq & 1];
      // (The item is read from shared memory where it is used: the scores need the registers.)
      if (grp < it.n_q) {
        const int tok = it.i0 + grp * TM + trow / g;  // local query token of the row
        const bool valid = trow < TM * g && tok < it.Sq;
        const bool releases = grp == it.n_q - 1 && trow == 0;
        float sl2 = a.scale * 1.4426950408889634f;
        if (POOLQ4 && it.n > 0) {
          // The row's Q in fp16, scaled so that its largest magnitude lies in [2^13, 2^14).  (Its place is free: this
          // tile's scores of the last item were seen to be complete.)
          const int64_t at = (((int64_t)it.q0 + tok) * a.Hq + it.kvh * g + trow % g) * D;
          const uint4* src = reinterpret_cast<const uint4*>((const T*)a.q + at);
          uint4 x[D / 8];
#pragma unroll
          for (int v = 0; v < D / 8; ++v) x[v] = valid ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
          float top = 0.f;
#pragma unroll
          for (int v = 0; v < D / 8; ++v) {
            const T* e = reinterpret_cast<const T*>(&x[v]);
#pragma unroll
            for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(pkv_to_f32<T>(e[c])));
          }
          const int e2 = top > 0.f && top <= 3.402823466e38f ? min(13 - ilogbf(top), 64) : 0;
          sl2 = scalbnf(sl2, -e2);
#pragma unroll
          for (int v = 0; v < D / 8; ++v) {
            const T* e = reinterpret_cast<const T*>(&x[v]);
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              w[c] = ptx::pack_f16x2(scalbnf(pkv_to_f32<T>(e[c]), e2), scalbnf(pkv_to_f32<T>(e[c + 4]), e2));
            *reinterpret_cast<uint4*>(sm.q[grp] + (v >> 3) * (BM * 128) + trow * 128 + (((v & 7) ^ (trow & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(&sm.q_full[grp]);
        }
        const int p = valid ? it.base + tok : -1;
        // The warp's rows with queries are consecutive positions [p_lo, p_hi].
        int w_last = it.i0 + grp * TM + (quarter * 32 + 31 < TM * g ? quarter * 32 + 31 : TM * g - 1) / g;
        w_last = w_last < it.Sq ? w_last : it.Sq - 1;
        const int p_lo = it.base + it.i0 + grp * TM + (quarter * 32) / g, p_hi = it.base + w_last;
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < it.n; ++j) {
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(&sm.s_full[grp], sc & 1, &sm.abort, kWaitLimitNs))) {
            ok = false;
            break;
          }
          ++sc;
          if (trow == 0) release_staged();
          ptx::tc_fence_after();
          // The last group's scores of tile j are committed after every earlier MMA: key tile j and value tile j-1
          // are no longer read.  (The last tile's two slots stage the output.)
          if (releases) {
            const int idx = 2 * (tb + j);
            if (j < it.n - 1 || n_cta > 1) ptx::mbar_arrive(&sm.empty[idx % C::NSLOT]);
            if (j > 0) ptx::mbar_arrive(&sm.empty[(idx - 1) % C::NSLOT]);
          }
          if (!POOLQ4 && trow == 0 && j == it.n - 1) ptx::mbar_arrive(&sm.q_empty[grp]);
          float s[BN];
          {
            uint32_t r[BN / 32][32];
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) ptx::tmem_ld32(tmem + lane_base + S_COL + c * 32, r[c]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
              ptx::reg_fence32(r[c]);
#pragma unroll
              for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(r[c][e]);
            }
          }
          // Whole tile seen by all of the warp's rows?  (Pages of a tile ascend.)
          const int v0 = kPages * (it.t_begin + j);
          const int j_first = it.pg.page(v0) * 16;
          const int j_last = v0 + kPages <= it.pg.n ? it.pg.page(v0 + kPages - 1) * 16 + 15 : 0x7fffffff;
          if (!(j_last <= p_lo && (a.window == 0 || j_last < a.sinks || p_hi - j_first < a.window))) {
            uint32_t bits[BN / 32];  // seen columns
            if (v0 >= it.pg.n_sink && (a.window == 0 || j_first >= a.sinks)) {
              // Consecutive pages past the sinks: columns (p - window, p] - j_first.
              const int hi = p - j_first, lo = a.window ? hi - a.window : -1;
#pragma unroll
              for (int q = 0; q < BN / 32; ++q) {
                const int h = hi - 32 * q, w = lo - 32 * q;
                const uint32_t up = h < 0 ? 0u : h >= 31 ? 0xffffffffu : (2u << h) - 1u;
                const uint32_t down = w < 0 ? 0u : w >= 31 ? 0xffffffffu : (2u << w) - 1u;
                bits[q] = up & ~down;
              }
            } else {
              // Column c of a page is seen when c <= hi and (c < sk or c > lo); two pages a word.
#pragma unroll
              for (int q = 0; q < BN / 32; ++q) {
                bits[q] = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int v = v0 + 2 * q + k, j0 = it.pg.page(v) * 16;
                  const int hi = v < it.pg.n ? p - j0 : -1, sk = a.sinks - j0, lo = p - j0 - a.window;
                  unsigned b16 = hi < 0 ? 0u : hi >= 15 ? 0xffffu : (2u << hi) - 1u;
                  if (a.window) {
                    const unsigned head = sk <= 0 ? 0u : sk >= 16 ? 0xffffu : (1u << sk) - 1u;
                    const unsigned tail = lo < 0 ? 0xffffu : lo >= 15 ? 0u : ~((2u << lo) - 1u);
                    b16 &= head | tail;
                  }
                  bits[q] |= (b16 & 0xffffu) << (16 * k);
                }
              }
            }
#pragma unroll
            for (int c = 0; c < BN; ++c) s[c] = (bits[c >> 5] & (1u << (c & 31))) ? s[c] : -INFINITY;
          }
          float mx[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) mx[u] = fmaxf(s[2 * u], s[2 * u + 1]);
#pragma unroll
          for (int c = 16; c < BN; c += 16)
#pragma unroll
            for (int u = 0; u < 8; ++u) mx[u] = ptx::max3(mx[u], s[c + 2 * u], s[c + 2 * u + 1]);
          const float m_tile =
              fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) *
              sl2;
          const bool need = m_tile > m_ref + kRescale;
          const bool rescale = __any_sync(0xffffffffu, need);
          const float alpha = need ? ptx::ex2(m_ref - m_tile) : 1.f;  // 0 on a row's first visible tile
          if (need) {
            l *= alpha;
            m_ref = m_tile;
          }
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
          for (int c = 0; c < BN / 64; ++c) {
            uint32_t r[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float x0, x1;
              ptx::fma2(x0, x1, s[c * 64 + 2 * e], s[c * 64 + 2 * e + 1], sl2, sl2, -mu, -mu);
              const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
              if (e & 1)
                ptx::add2(l2, l3, p0, p1);
              else
                ptx::add2(l0, l1, p0, p1);
              r[e] = OPBF16 ? ptx::pack_bf16x2(p0, p1) : ptx::pack_f16x2(p0, p1);
            }
            ptx::tmem_st32(tmem + lane_base + S_COL + c * 32, r);
            if (c == 0 && rescale && j > 0) {
#pragma unroll
              for (int d = 0; d < D / 32; ++d) {
                uint32_t o[32];
                ptx::tmem_ld32(tmem + lane_base + O_COL[grp] + d * 32, o);
                ptx::tmem_wait_ld();
                ptx::reg_fence32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                ptx::tmem_st32(tmem + lane_base + O_COL[grp] + d * 32, o);
              }
            }
            if (C::PARTS == 2 || c == 1) {
              ptx::tmem_wait_st();
              ptx::tc_fence_before();
              ptx::mbar_arrive(&sm.p_full[grp][C::PARTS == 2 ? c : 0]);
            }
          }
          l += (l0 + l1) + (l2 + l3);
        }

        // ---------------------------------------------------------------- epilogue
        float o[D];
#pragma unroll
        for (int c = 0; c < D; ++c) o[c] = 0.f;
        if (ok && it.n > 0) {
          if (__all_sync(0xffffffffu, ptx::mbar_wait(&sm.o_full[grp], oc & 1, &sm.abort, kWaitLimitNs))) {
            ptx::tc_fence_after();
            uint32_t r[D / 32][32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) ptx::tmem_ld32(tmem + lane_base + O_COL[grp] + c * 32, r[c]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              ptx::reg_fence32(r[c]);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                // 4-bit values come in the order of channels (0, 4, 1, 5, 2, 6, 3, 7) of each eight
                const int ch = POOLQ4 ? (c * 32 + (e & ~7)) + ((e & 1) * 4 + ((e >> 1) & 3)) : c * 32 + e;
                o[ch] = __uint_as_float(r[c][e]);
              }
            }
            ++oc;
            ptx::tc_fence_before();  // read before the next item's first P.V
          } else {
            ok = false;
          }
        }
        if (!ok) {
          note_abort(sm, a.err);
          break;
        }
        if (n_cta > 1) {
          // Staged for the merge in the key/value ring and the Q buffer, which no copy or MMA uses any more once the
          // other tile's output is complete too (a cluster has one item).
          if (it.n > 0 && it.n_q == 2 &&
              !__all_sync(0xffffffffu, ptx::mbar_wait(&sm.o_full[grp ^ 1], 0, &sm.abort, kWaitLimitNs))) {
            note_abort(sm, a.err);
            break;
          }
          float* st = reinterpret_cast<float*>(sm.kv[0]) + (grp * BM + trow) * C::OSTRIDE;
#pragma unroll
          for (int v = 0; v < D / 4; ++v)
            *reinterpret_cast<float4*>(st + 4 * v) = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          float* ml = reinterpret_cast<float*>(sm.q[0]);  // [2 BM] maxima, [2 BM] sums
          ml[grp * BM + trow] = m_ref;
          ml[2 * BM + grp * BM + trow] = l;
        } else {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint32_t w[D / 2];
#pragma unroll
          for (int c = 0; c < D / 2; ++c) {
            const float x0 = o[2 * c] * inv, x1 = o[2 * c + 1] * inv;
            w[c] = OUTBF16 ? ptx::pack_bf16x2(x0, x1) : ptx::pack_f16x2(x0, x1);
          }
          T* const out = (T*)a.out + ((int64_t)it.q0 * a.Hq + it.kvh * g) * D;
          if (it.n > 0) {
            // Through shared memory -- the last tile's key slot (tile 0) and value slot (tile 1), which no MMA reads any
            // more -- because rows stored thread by thread take an instruction 32 lines: 7000 cycles a tile.
            const int slot = (2 * (tb + it.n) - 2 + grp) % C::NSLOT;
            uint8_t* tile = sm.kv[slot];  // [D/64][128 rows][128 B], swizzled like Q
            if (releases && grp == 0) ptx::mbar_arrive(&sm.empty[(slot + 1) % C::NSLOT]);  // nothing to stage of tile 1
#pragma unroll
            for (int v = 0; v < D / 8; ++v)
              *reinterpret_cast<uint4*>(tile + (v >> 3) * (BM * 128) + trow * 128 + (((v & 7) ^ (trow & 7)) << 4)) =
                  make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
            const int first = it.i0 + grp * TM;
            if (first + TM <= it.Sq) {  // whole tiles: one TMA store per column half
              ptx::fence_proxy_async_smem();
              ok = tile_sync();
              if (ok && trow == 0) {
#pragma unroll
                for (int dh = 0; dh < D / 64; ++dh)
                  tma_store_4d(&maps.o, dh * 64, 0, it.kvh, it.q0 + first, tile + dh * (BM * 128));
                ptx::bulk_commit();
                staged = slot;  // given back once it has been read: when the next item's first scores are there
              }
            } else {  // a sequence's last tile: the rows that are queries
              ok = tile_sync();
              const int rows = ok ? (it.Sq - first) * g : 0;
              for (int e = trow; e < rows * (D / 8); e += BM) {
                const int r = e / (D / 8), v = e % (D / 8);
                reinterpret_cast<uint4*>(out + ((int64_t)(first + r / g) * a.Hq + r % g) * D)[v] =
                    *reinterpret_cast<const uint4*>(tile + (v >> 3) * (BM * 128) + r * 128 + (((v & 7) ^ (r & 7)) << 4));
              }
              ok = ok && tile_sync();
              if (ok && trow == 0) ptx::mbar_arrive(&sm.empty[slot]);
            }
            if (!ok) {
              note_abort(sm, a.err);
              break;
            }
          } else if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(out + ((int64_t)tok * a.Hq + trow % g) * D);
#pragma unroll
            for (int v = 0; v < D / 8; ++v) dst[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
          }
        }
      }
      if (trow == 0 && (it.n == 0 || grp >= it.n_q)) release_staged();  // no first tile here to do it after
      tb += it.n;
      done_item();
    }
    if (trow == 0) release_staged();  // read before the shared memory goes away
  }

  // ---------------------------------------------------------------- teardown, and the cluster's merge
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (n_cta > 1 && sm.info[0].n >= 0) {  // the same for every CTA of the cluster
    const Item& it = sm.info[0];
    __syncwarp();
    cluster_sync();
    // Rows r of tile t in turn over the cluster's warps; a lane takes D/32 channels.
    constexpr int CH = D / 32;
    const int rows = it.n_q * BM;
    for (int e = (int)rank * (kThreads / 32) + warp; e < rows; e += (int)n_cta * (kThreads / 32)) {
      const int tr = e % BM;
      const int tk = it.i0 + (e / BM) * TM + tr / g;
      if (tr >= TM * g || tk >= it.Sq) continue;
      float mk = -INFINITY, lk = 0.f;
      if (lane < (int)n_cta) {
        const uint32_t ml = cluster_addr(reinterpret_cast<float*>(sm.q[0]) + e, lane);
        mk = cluster_ld(ml);
        lk = cluster_ld(ml + 2 * BM * 4);
      }
      float top = mk;
#pragma unroll
      for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float wk = mk == top ? 1.f : ptx::ex2(mk - top);  // CTAs without keys hold zeros
      float sum = 0.f, acc[CH] = {};
      for (int k = 0; k < (int)n_cta; ++k) {
        const float w = __shfl_sync(0xffffffffu, wk, k);
        sum += w * __shfl_sync(0xffffffffu, lk, k);
        const uint32_t src = cluster_addr(reinterpret_cast<float*>(sm.kv[0]) + e * C::OSTRIDE + lane * CH, k);
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          const float2 x = cluster_ld2(src + c * 4);
          acc[c] += w * x.x, acc[c + 1] += w * x.y;
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T* dst = (T*)a.out + (((int64_t)it.q0 + tk) * a.Hq + it.kvh * g + tr % g) * D + lane * CH;
#pragma unroll
      for (int c = 0; c < CH; c += 2) store_pair<T>(dst + c, acc[c] * inv, acc[c + 1] * inv);
    }
    __syncwarp();
    cluster_sync();
  }
  // A second launch completes after the first: what follows on the stream waits for it alone.
  if (first_item) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
  });
  return fn;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, bool bf16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, typename T, bool POOLQ4>
int launch(const PkvWinArgs& a, int64_t Tq, int* launches, cudaStream_t s) {
  constexpr bool BF16 = !std::is_same<T, __half>::value;
  auto kernel = attn_win_tc_kernel<D, T, BF16 && !POOLQ4, POOLQ4>;
  const int g = a.Hq / a.Hkv, TM = BM / g;
  WinMaps maps;
  memset(&maps, 0, sizeof(maps));
  const cuuint64_t dq[4] = {(cuuint64_t)D, (cuuint64_t)g, (cuuint64_t)a.Hkv, (cuuint64_t)Tq};
  const cuuint64_t sq[3] = {(cuuint64_t)D * 2, (cuuint64_t)g * D * 2, (cuuint64_t)a.Hq * D * 2};
  const cuuint32_t bq[4] = {64, (cuuint32_t)g, 1, (cuuint32_t)TM};
  if (!encode(&maps.o, a.out, 4, dq, sq, bq, BF16)) return (int)cudaErrorInvalidValue;
  if (!POOLQ4) {
    const cuuint64_t slots = (cuuint64_t)a.num_blocks * 16, slot = (cuuint64_t)a.Hkv * D * 2;
    const cuuint64_t d5[5] = {64, 8, (cuuint64_t)(D / 64), slots / 8, (cuuint64_t)a.Hkv};
    const cuuint64_t s5[4] = {slot, 128, 8 * slot, (cuuint64_t)D * 2};
    const cuuint32_t b5[5] = {64, 8, (cuuint32_t)(D / 64), 2, 1};
    const cuuint64_t d3[3] = {(cuuint64_t)D, (cuuint64_t)a.Hkv, slots};
    const cuuint64_t s3[2] = {(cuuint64_t)D * 2, slot};
    const cuuint32_t b1[3] = {64, 1, 1};
    if (!encode(&maps.q, a.q, 4, dq, sq, bq, BF16) || !encode(&maps.kb, a.k_pool, 5, d5, s5, b5, BF16) ||
        !encode(&maps.vb, a.v_pool, 5, d5, s5, b5, BF16) || !encode(&maps.v1, a.v_pool, 3, d3, s3, b1, BF16))
      return (int)cudaErrorInvalidValue;
  }
  const size_t smem = sizeof(WinSmem<D, POOLQ4>) + 1024;
  static PkvKernelState state;
  int rc = pkv_prepare_kernel((const void*)kernel, (int)smem, Roles<POOLQ4>::kThreads, Roles<POOLQ4>::kRegs, state);
  if (rc) return rc;
  const int64_t items = (int64_t)a.B * a.Hkv * ((a.max_query_len + 2 * TM - 1) / (2 * TM));
  const int64_t steps = pkv_visible_keys(a, 2 * TM) / BN + 1;
  const PkvClusterPlan plan = pkv_plan_cluster_tail(state, items, steps, kFixedTiles);
  uint32_t first = 0;
  void* args[] = {&maps, const_cast<PkvWinArgs*>(&a), &first};
  *launches = 0;
  if (plan.whole > 0) {
    rc = pkv_launch_cluster((const void*)kernel, plan.whole, 1, Roles<POOLQ4>::kThreads, smem, args, false, s);
    if (rc) return rc;
    ++*launches;
    first = (uint32_t)plan.whole;
  }
  if (items > plan.whole) {
    rc = pkv_launch_cluster((const void*)kernel, items - plan.whole, plan.ctas, Roles<POOLQ4>::kThreads, smem, args,
                            first != 0, s);
    if (rc) return rc;
    ++*launches;
  }
  return 0;
}

template <int D, bool POOLQ4>
int launch_t(const PkvWinArgs& a, int64_t Tq, pkv_dtype dt, int* launches, cudaStream_t s) {
  return dt == PKV_BF16 ? launch<D, __nv_bfloat16, POOLQ4>(a, Tq, launches, s)
                        : launch<D, __half, POOLQ4>(a, Tq, launches, s);
}

}  // namespace

int pkv_win_tc_heads() { return BM; }

int pkv_launch_win_tc(const PkvWinArgs& a, int64_t Tq, pkv_dtype dt, int D, bool q4, int* launches, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  if (q4) return D == 64 ? launch_t<64, true>(a, Tq, dt, launches, s) : launch_t<128, true>(a, Tq, dt, launches, s);
  return D == 64 ? launch_t<64, false>(a, Tq, dt, launches, s) : launch_t<128, false>(a, Tq, dt, launches, s);
}
