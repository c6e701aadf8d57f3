// Entry points of the serving operators: rotary append, 4-bit pools, window/sinks attention.  Argument checks,
// the choice of kernel, and the plan of how many CTAs share an item's keys.

#include <math.h>

#include "common.cuh"

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int64_t kMaxGrid = 0x7fffffff;
constexpr int kMaxKeys = 0x7fffff00;  // positions of a whole tile past them still fit an int

pkv_status check_dtype(const char* fn, pkv_dtype dt) {
  if (dt == PKV_F32 || dt == PKV_BF16 || dt == PKV_F16) return PKV_OK;
  return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
}

pkv_status append_impl(const char* fn, bool q4, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const int32_t* positions, const float* cos_sin,
                       int64_t max_position, int rot_dim, const int64_t* slots, int64_t T, int Hq, void* q_out,
                       void* key_pool, void* value_pool, int64_t num_slots, int Hkv, int D, pkv_dtype dt,
                       uint32_t flags, void* stream) {
  pkv_clear_error();
  pkv_set_launches(0);
  if (T < 0 || num_slots < 0 || max_position < 0 || Hq < 0 || Hkv <= 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: negative or zero size (T=%lld, Hq=%d, Hkv=%d)", fn, (long long)T, Hq, Hkv);
  if (D != 64 && D != 128) return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: head dim must be 64 or 128 (got %d)", fn, D);
  if (pkv_status st = check_dtype(fn, dt)) return st;
  if (rot_dim < 0 || rot_dim > D)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: rot_dim must be in [0, %d] (got %d)", fn, D, rot_dim);
  if (rot_dim % 16) return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: rot_dim must be a multiple of 16 (got %d)", fn, rot_dim);
  if (T > kMaxGrid || (int64_t)Hq + 2 * (int64_t)Hkv > 65535)
    return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: too many tokens or heads for one call (T=%lld, Hq=%d, Hkv=%d)", fn,
                    (long long)T, Hq, Hkv);
  if (T == 0) return PKV_OK;
  if ((Hq > 0 && (!q || !q_out)) || !k || !v || !slots || !key_pool || !value_pool ||
      (rot_dim && (!positions || !cos_sin)))
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  const int size = pkv_dtype_size(dt);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(key_pool) ||
      !aligned16(value_pool) || !aligned16(rot_dim ? cos_sin : nullptr) || (Hq && (q_stride * size) % 16) ||
      (k_stride * size) % 16 || (v_stride * size) % 16)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: base pointers and token strides must be 16-byte aligned", fn);
  if (Hq && q == q_out && T > 1 && q_stride != (int64_t)Hq * D)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: q_out may be q only when q is contiguous", fn);
  PkvAppendArgs a{};
  a.q = q, a.k = k, a.v = v;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.positions = positions, a.cos_sin = cos_sin, a.max_position = max_position;
  a.slots = slots, a.q_out = q_out, a.k_pool = key_pool, a.v_pool = value_pool;
  a.num_slots = num_slots, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.D = D, a.rot_dim = rot_dim;
  a.interleaved = (flags & PKV_ROPE_INTERLEAVED) ? 1 : 0;
  a.check = (flags & PKV_CHECK_BOUNDS) ? 1 : 0;
  a.err = a.check ? pkv_device_error_word() : nullptr;
  if (a.check && !a.err) return pkv_fail(PKV_ERR_CUDA, "%s: device error word unavailable", fn);
  const int rc = pkv_launch_append(a, dt, q4, stream);
  if (rc) return pkv_fail(PKV_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString((cudaError_t)rc));
  pkv_set_launches(1);
  return PKV_OK;
}

enum class WinKernel { kSimt, kTc, kDec };

// Few query rows per kv head take the memory-bound kernel, which reads each key once for all of them; more, tiles of 256
// rows on tcgen05.  Where they cross depends on how many (sequence, kv head) pairs there are, because the former spreads
// the keys of a pair further, and on the former's registers.  Measured with 1 and 6 to 100 sequences, 8 kv heads, us:
//   16-bit, D 128, 20 rows:        6 x 2000 keys 47 against 22 on tcgen05, 1 x 30000 (1 kv head) 22 against 35
//   16-bit, D 64, 20 and 40 rows:  24 x 2000 keys 52 against 51, 83 against 51; 1 x 65536 43 against 106, 74 against 106
//   4-bit, D 128, 30 and 40 rows:  24 x 2000 keys 57 against 66, 83 against 67; 1 x 65536 46 against 136, 70 against 137
WinKernel win_kernel(pkv_dtype dt, bool q4, int64_t num_blocks, int64_t pairs, int D, int64_t max_query_len, int g,
                     uint32_t flags) {
  if (dt == PKV_F32 || (flags & PKV_FORCE_SIMT)) return WinKernel::kSimt;
  const int64_t few = (q4 || D == 64 ? 32 : 16) * (pairs < 16 ? 2 : 1);
  return max_query_len * g > few && num_blocks > 0 && g <= pkv_win_tc_heads() ? WinKernel::kTc : WinKernel::kDec;
}

pkv_status win_impl(const char* fn, bool q4, const void* q, int64_t Tq, int Hq, const void* key_pool,
                    const void* value_pool, int64_t num_blocks, int block_size, int Hkv, int D, pkv_dtype dt,
                    const int32_t* block_table, int B, int W, const int32_t* query_start_loc, const int32_t* seq_lens,
                    int max_query_len, int max_seq_len, float softmax_scale, int window, int sinks, void* out,
                    void* workspace, size_t ws_bytes, uint32_t flags, void* stream) {
  pkv_clear_error();
  pkv_set_launches(0);
  if (Tq < 0 || B < 0 || W < 0 || max_query_len < 0 || max_seq_len < 0 || num_blocks < 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: negative size", fn);
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv)
    return pkv_fail(PKV_ERR_INVALID_ARG,
                    "%s: num_heads must be a positive multiple of num_kv_heads (Hq=%d, Hkv=%d)", fn, Hq, Hkv);
  if (block_size != 16) return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: block_size must be 16 (got %d)", fn, block_size);
  if (D != 64 && D != 128) return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: head dim must be 64 or 128 (got %d)", fn, D);
  if (pkv_status st = check_dtype(fn, dt)) return st;
  if (window < 0 || sinks < 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: window and sinks must not be negative (%d, %d)", fn, window, sinks);
  if (!isfinite(softmax_scale)) return pkv_fail(PKV_ERR_INVALID_ARG, "%s: softmax_scale is not finite", fn);
  if (dt != PKV_F32 && !(softmax_scale > 0.f) && !(flags & PKV_FORCE_SIMT))
    return pkv_fail(PKV_ERR_UNSUPPORTED,
                    "%s: a bf16/f16 call needs softmax_scale > 0 (got %g); pass PKV_FORCE_SIMT to run it on the "
                    "CUDA-core kernel", fn, (double)softmax_scale);
  if ((int64_t)max_seq_len > (int64_t)W * block_size)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: max_seq_len %d exceeds the table's %d x %d slots", fn, max_seq_len, W,
                    block_size);
  if (max_seq_len > kMaxKeys)
    return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: max_seq_len %d is past the %d keys of one call", fn, max_seq_len, kMaxKeys);
  if (Tq > kMaxGrid || (int64_t)max_query_len * (Hq / Hkv) > kMaxGrid - 1024)
    return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: too many queries for one call", fn);
  if (Tq == 0 || B == 0 || max_query_len == 0) return PKV_OK;
  if (!q || !key_pool || !value_pool || !block_table || !query_start_loc || !seq_lens || !out)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(key_pool) || !aligned16(value_pool) || !aligned16(out))
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: q, pools and out must be 16-byte aligned", fn);
  if (!aligned16(workspace)) return pkv_fail(PKV_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
  if (num_blocks == 0 && max_seq_len > 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: keys of up to %d positions in a pool without blocks", fn, max_seq_len);
  PkvWinArgs a{};
  a.q = q, a.k_pool = key_pool, a.v_pool = value_pool, a.out = out;
  a.block_table = block_table, a.query_start_loc = query_start_loc, a.seq_lens = seq_lens;
  a.num_blocks = num_blocks, a.B = B, a.W = W, a.Hq = Hq, a.Hkv = Hkv;
  a.max_query_len = max_query_len, a.max_seq_len = max_seq_len, a.window = window, a.sinks = sinks;
  a.check = (flags & PKV_CHECK_BOUNDS) ? 1 : 0;
  a.scale = softmax_scale;
  a.err = pkv_device_error_word();
  if (!a.err) return pkv_fail(PKV_ERR_CUDA, "%s: device error word unavailable", fn);
  int rc, launches = 1;
  switch (win_kernel(dt, q4, num_blocks, (int64_t)B * Hkv, D, max_query_len, Hq / Hkv, flags)) {
    case WinKernel::kSimt: rc = pkv_launch_win_simt(a, dt, D, q4, stream); break;
    case WinKernel::kTc: rc = pkv_launch_win_tc(a, Tq, dt, D, q4, &launches, stream); break;
    default:
      rc = (q4 ? pkv_launch_q4_dec : pkv_launch_win_dec)(a, dt, D, workspace, ws_bytes, nullptr, &launches, stream);
  }
  if (rc) return pkv_fail(PKV_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString((cudaError_t)rc));
  pkv_set_launches(launches);
  return PKV_OK;
}

}  // namespace

// ---------------------------------------------------------------- launches

int pkv_prepare_kernel(const void* kernel, int smem, int threads, int regs, PkvKernelState& state) {
  // Keyed on the context: function attributes belong to the context they were set in.  Racing first calls only
  // repeat the same settings.
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  const uint64_t ctx = pkv_context_id();
  if (ctx != 0 && state.ctx[dev].load(std::memory_order_acquire) == ctx) return 0;
  if (regs > 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return (int)e;
    if (fa.numRegs != regs) return (int)cudaErrorInvalidKernelImage;
  }
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return (int)e;
  for (int i = 0; i < 5; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1u << i);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << i;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    state.active[dev][i].store(n, std::memory_order_relaxed);
  }
  state.ctx[dev].store(ctx, std::memory_order_release);
  return 0;
}

int64_t pkv_visible_keys(const PkvWinArgs& a, int64_t tokens) {
  int64_t keys = a.max_seq_len;
  if (a.window > 0) {
    const int64_t most = (int64_t)a.window + tokens + a.sinks + 32;
    if (most < keys) keys = most;
  }
  return keys;
}

namespace {

struct Split {
  int ctas;
  double cost;
};

// A kernel of one CTA per SM runs in waves of the clusters that fit the GPU at once; each CTA takes its share of the
// steps plus the fixed cost.  The smallest estimate wins, a larger cluster only where it gains a tenth.
Split best_split(const PkvKernelState& state, int dev, int64_t items, int64_t steps, double fixed) {
  Split best{1, 1e300};
  for (int i = 0; i < 5; ++i) {
    const int c = 1 << i;
    const int64_t active = state.active[dev][i].load(std::memory_order_relaxed);
    if (active <= 0 && c > 1) break;
    if (c > 1 && (steps < 2 * c || items * c > kMaxGrid)) break;
    const int64_t at_once = active > 0 ? active : 152;
    const double cost = (double)((items + at_once - 1) / at_once) * ((double)((steps + c - 1) / c) + fixed);
    if (cost < 0.9 * best.cost) best = Split{c, cost};
  }
  return best;
}

int current_device() {
  int dev = 0;
  cudaGetDevice(&dev);
  return dev < 0 || dev >= 64 ? 0 : dev;
}

}  // namespace

// Kernels of several CTAs per SM, in steps of a CTA that has its SM to itself.  Such a CTA waits for its loads most of
// the time, so a second one costs nothing at first; `rate` is the share of the SM (its memory bandwidth or its issue
// slots) that one needs, and from 1 / rate of them on they take turns.  Each CTA costs `setup` steps more, less where
// others work meanwhile.  The SM with the most CTAs decides; past three of them the hardware deals them out as they
// finish.  A cluster costs its launch and merge.  Fitted to 681 mixes of 1 to 100 sequences, 73 to 131072 keys, 1 to 8 kv
// heads, one query to prompts, timed with every cluster size and several splits: the choice is 2 % (16-bit and fp32 tiles),
// 1 % (4-bit) and 6 % (fp32, few rows) over the best on average; a model whose CTAs share an SM at the rate of one was
// 14, 11, 3 and 13 % over it.
static double shared_cost(int64_t ctas, int64_t sms, int64_t steps, double rate, double setup) {
  const double k = (double)ctas / (double)sms;
  const double most = k <= 1.0 ? 1.0 : k <= 3.0 ? ceil(k) : k + 1.1;
  return (most * rate > 1.0 ? most * rate : 1.0) * (double)steps + setup * (1.0 + 0.31 * (most - 1.0));
}

static Split best_cluster(const PkvKernelState& state, int dev, int64_t items, int64_t steps, double rate, double setup) {
  static const double merge[5] = {0.0, 0.56, 0.55, 0.63, 1.33};  // in set-ups
  const int64_t sms = pkv_sm_count() > 0 ? pkv_sm_count() : 152;
  Split best{1, 1e300};
  for (int i = 0; i < 5; ++i) {
    const int c = 1 << i;
    if (i > 0 && (state.active[dev][i].load(std::memory_order_relaxed) <= 0 || 2 * steps < c || items * c > kMaxGrid)) break;
    const double cost = shared_cost(items * c, sms, (steps + c - 1) / c, rate, setup) + merge[i] * setup;
    if (cost < 0.99 * best.cost) best = Split{c, cost};
  }
  return best;
}

int pkv_plan_cluster(const PkvKernelState& state, int64_t items, int64_t steps, double rate, double setup) {
  return best_cluster(state, current_device(), items, steps, rate, setup).ctas;
}

int pkv_plan_splits(const PkvKernelState& state, int64_t items, int64_t steps, double rate, double setup,
                    double combine) {
  const int dev = current_device();
  const int64_t sms = pkv_sm_count() > 0 ? pkv_sm_count() : 152;
  const int64_t per_sm = state.active[dev][0].load(std::memory_order_relaxed) / sms;
  if (items * 2 > sms || steps <= 16) return 1;
  Split best = best_cluster(state, dev, items, steps, rate, setup);
  best.ctas = 1;
  for (int64_t m = 1; m <= per_sm; ++m) {  // as many CTAs on every SM
    int64_t n = m * sms / items;
    if (n > kPkvMaxWinSplits) n = kPkvMaxWinSplits;
    if (n < 2 || n > steps) continue;
    const double cost = shared_cost(items * n, sms, (steps + n - 1) / n, rate, setup) + combine;
    if (cost < 0.99 * best.cost) best = Split{(int)n, cost};
  }
  return best.ctas;
}

// Whole waves of single CTAs, and a second launch that splits the items behind them, where that is estimated a
// twentieth under one launch of equal clusters.
PkvClusterPlan pkv_plan_cluster_tail(const PkvKernelState& state, int64_t items, int64_t steps, double fixed) {
  const int dev = current_device();
  const Split one = best_split(state, dev, items, steps, fixed);
  const int64_t sms = state.active[dev][0].load(std::memory_order_relaxed);
  if (sms > 0 && items > sms && items % sms) {
    const int64_t waves = items / sms;
    const Split tail = best_split(state, dev, items % sms, steps, fixed);
    if (tail.ctas > 1 && waves * ((double)steps + fixed) + tail.cost < 0.95 * one.cost)
      return PkvClusterPlan{waves * sms, tail.ctas};
  }
  return PkvClusterPlan{0, one.ctas};
}

int pkv_launch_cluster(const void* kernel, int64_t items, int ctas, int threads, size_t smem, void** args,
                       bool overlap, void* stream) {
  if (items * ctas > kMaxGrid) return (int)cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * ctas));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  const cudaError_t last = cudaGetLastError();
  return (int)(e != cudaSuccess ? e : last);
}

// ---------------------------------------------------------------- C entries

extern "C" size_t pkv_q4_block_bytes(int D) { return D == 64 || D == 128 ? (size_t)10 * D : 0; }

extern "C" pkv_status paged_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, const int32_t* positions, const float* cos_sin,
                                      int64_t max_position, int rot_dim, const int64_t* slot_mapping, int64_t T,
                                      int Hq, void* q_out, void* key_pool, void* value_pool, int64_t num_slots,
                                      int Hkv, int D, pkv_dtype dt, uint32_t flags, void* stream) {
  return append_impl("paged_kv_append", false, q, q_stride, k, k_stride, v, v_stride, positions, cos_sin, max_position,
                     rot_dim, slot_mapping, T, Hq, q_out, key_pool, value_pool, num_slots, Hkv, D, dt, flags, stream);
}

extern "C" pkv_status paged_kv_append_q4(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                         const void* v, int64_t v_stride, const int32_t* positions,
                                         const float* cos_sin, int64_t max_position, int rot_dim,
                                         const int64_t* slot_mapping, int64_t T, int Hq, void* q_out, void* key_pool,
                                         void* value_pool, int64_t num_blocks, int Hkv, int D, pkv_dtype dt,
                                         uint32_t flags, void* stream) {
  if (num_blocks > INT64_MAX / 16) num_blocks = INT64_MAX / 16;
  return append_impl("paged_kv_append_q4", true, q, q_stride, k, k_stride, v, v_stride, positions, cos_sin,
                     max_position, rot_dim, slot_mapping, T, Hq, q_out, key_pool, value_pool, num_blocks * 16, Hkv, D,
                     dt, flags, stream);
}

extern "C" pkv_status paged_kv_gather_q4(const void* key_pool, const void* value_pool, int64_t num_blocks,
                                         const int32_t* block_table, int B, int W, int first_block, int n_blocks,
                                         void* stage_k, void* stage_v, int64_t stage_rows, int Hkv, int D,
                                         pkv_dtype dt, uint32_t flags, void* stream) {
  const char* fn = "paged_kv_gather_q4";
  pkv_clear_error();
  pkv_set_launches(0);
  if (B < 0 || W < 0 || first_block < 0 || n_blocks < 0 || num_blocks < 0 || stage_rows < 0 || Hkv <= 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: negative or zero size", fn);
  if (D != 64 && D != 128) return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: head dim must be 64 or 128 (got %d)", fn, D);
  if (pkv_status st = check_dtype(fn, dt)) return st;
  if ((int64_t)first_block + n_blocks > W)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: blocks [%d, %d) run past the table width %d", fn, first_block,
                    first_block + n_blocks, W);
  if (((int64_t)first_block + n_blocks) * 16 > stage_rows)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: %d blocks do not fit %lld staging rows", fn, first_block + n_blocks,
                    (long long)stage_rows);
  if (B == 0 || n_blocks == 0) return PKV_OK;
  if (!key_pool || !value_pool || !block_table || !stage_k || !stage_v)
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (!aligned16(key_pool) || !aligned16(value_pool) || !aligned16(stage_k) || !aligned16(stage_v))
    return pkv_fail(PKV_ERR_INVALID_ARG, "%s: base pointers must be 16-byte aligned", fn);
  const int check = (flags & PKV_CHECK_BOUNDS) ? 1 : 0;
  unsigned int* err = check ? pkv_device_error_word() : nullptr;
  if (check && !err) return pkv_fail(PKV_ERR_CUDA, "%s: device error word unavailable", fn);
  const int rc = pkv_launch_gather_q4(key_pool, value_pool, num_blocks, block_table, B, W, first_block, n_blocks,
                                      stage_k, stage_v, stage_rows, Hkv, D, dt, err, check, stream);
  if (rc) return pkv_fail(PKV_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString((cudaError_t)rc));
  pkv_set_launches(1);
  return PKV_OK;
}

extern "C" size_t paged_attn_window_workspace_size(int64_t num_blocks, int Hq, int Hkv, int D, pkv_dtype dt, int q4, int B,
                                                   int max_query_len, int max_seq_len, int window, int sinks) {
  if (num_blocks <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || B <= 0 || max_query_len <= 0 || max_seq_len < 0 ||
      max_seq_len > kMaxKeys || window < 0 || sinks < 0 || (D != 64 && D != 128) || (int64_t)max_query_len * (Hq / Hkv) > kMaxGrid - 1024 ||
      (dt != PKV_BF16 && dt != PKV_F16) ||
      win_kernel(dt, q4 != 0, num_blocks, (int64_t)B * Hkv, D, max_query_len, Hq / Hkv, 0) != WinKernel::kDec)
    return 0;
  PkvWinArgs a{};
  a.num_blocks = num_blocks, a.B = B, a.Hq = Hq, a.Hkv = Hkv;
  a.max_query_len = max_query_len, a.max_seq_len = max_seq_len, a.window = window, a.sinks = sinks;
  size_t bytes = 0;
  return (q4 ? pkv_launch_q4_dec : pkv_launch_win_dec)(a, dt, D, nullptr, 0, &bytes, nullptr, nullptr) == 0 ? bytes : 0;
}

extern "C" pkv_status paged_attn_window(const void* q, int64_t Tq, int Hq, const void* key_pool,
                                        const void* value_pool, int64_t num_blocks, int block_size, int Hkv, int D,
                                        pkv_dtype dt, const int32_t* block_table, int B, int W,
                                        const int32_t* query_start_loc, const int32_t* seq_lens, int max_query_len,
                                        int max_seq_len, float softmax_scale, int window, int sinks, void* out,
                                        void* workspace, size_t ws_bytes, uint32_t flags, void* stream) {
  return win_impl("paged_attn_window", false, q, Tq, Hq, key_pool, value_pool, num_blocks, block_size, Hkv, D, dt,
                  block_table, B, W, query_start_loc, seq_lens, max_query_len, max_seq_len, softmax_scale, window,
                  sinks, out, workspace, ws_bytes, flags, stream);
}

extern "C" pkv_status paged_attn_q4(const void* q, int64_t Tq, int Hq, const void* key_pool, const void* value_pool,
                                    int64_t num_blocks, int block_size, int Hkv, int D, pkv_dtype dt,
                                    const int32_t* block_table, int B, int W, const int32_t* query_start_loc,
                                    const int32_t* seq_lens, int max_query_len, int max_seq_len, float softmax_scale,
                                    int window, int sinks, void* out, void* workspace,
                                    size_t ws_bytes, uint32_t flags, void* stream) {
  return win_impl("paged_attn_q4", true, q, Tq, Hq, key_pool, value_pool, num_blocks, block_size, Hkv, D, dt,
                  block_table, B, W, query_start_loc, seq_lens, max_query_len, max_seq_len, softmax_scale, window,
                  sinks, out, workspace, ws_bytes, flags, stream);
}
