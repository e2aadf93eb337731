// Host side of the KV-cache calls: plans, argument checks and launches (see
// include/ss_kv.h).
#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <mutex>
#include <new>

#include "ss_kv_common.cuh"

namespace ss {
void set_last_error(const char* msg);
}

namespace {

constexpr uint32_t kSpin = 1u << 22;  // polls of a copy wait before the copy counts as lost

ss_status fail(ss_status s, const char* msg) {
  ss::set_last_error(msg);
  return s;
}
ss_status cuda_fail(cudaError_t e, const char* where) {
  char msg[256];
  std::snprintf(msg, sizeof msg, "%s: %s", where, cudaGetErrorString(e));
  ss::set_last_error(msg);
  return SS_ERR_CUDA;
}
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// The plan's device for the length of a call.
struct OnDevice {
  int prev = -1, dev;
  explicit OnDevice(int d) : dev(d) {
    cudaGetDevice(&prev);
    if (prev != dev) cudaSetDevice(dev);
  }
  ~OnDevice() {
    if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  }
};
struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled of the driver; null if it has none.
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Shared-memory limits of the plans' kernels: set once per device and kernel (and size, for kernels with several).
cudaError_t configure(int device, const ss::AttendKernel& k) {
  struct Done {
    int device;
    const void* fn;
    size_t smem;
  };
  static std::mutex mu;
  static Done done[256];  // 16 kernels with at most a few sizes each; past that they are set again each time
  static int count = 0;
  const std::lock_guard<std::mutex> lock(mu);
  bool pages = false;
  size_t most = 0;
  for (const Done* d = done; d != done + count; ++d) {
    if (d->device != device) continue;
    pages = true;
    if (d->fn == k.fn) most = std::max(most, d->smem);
  }
  cudaError_t e = pages ? cudaSuccess : ss::kv_pages_configure();
  if (e == cudaSuccess && most < k.smem) {
    e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
    if (e == cudaSuccess && count < 256) done[count++] = {device, k.fn, k.smem};
  }
  return e;
}

ss::AttendKernel attend_kernel(const ss_kv_config& c, int row_tile) {
  const bool bf16 = c.dtype == SS_BF16, low = c.cache_dtype == SS_E4M3;
  return bf16 ? (low ? ss::kv_attend_bf16_e4m3(c.head_dim, row_tile) : ss::kv_attend_bf16(c.head_dim, row_tile))
              : (low ? ss::kv_attend_f16_e4m3(c.head_dim, row_tile) : ss::kv_attend_f16(c.head_dim, row_tile));
}

// A cache as a kernel's copies see it: (part of a head, token, number of the part, head, page).  Swizzled heads come in
// parts of at most 128 bytes; a copy of 16-bit values has all parts of 64 tokens, or one part of fewer (a smaller page),
// so that in shared memory a tile is its parts of 64 tokens either way; one of 8-bit values always has all.
ss_status encode(CUtensorMap* map, const ss_kv_plan* p, const ss_kv_cache* cache, void* base, bool swizzled) {
  const ss_kv_config& c = p->c;
  const bool low = c.cache_dtype == SS_E4M3;
  const cuuint32_t el = low ? 1 : 2, tokens = std::min(c.page_size, 64);
  const cuuint32_t part = swizzled ? std::min<cuuint32_t>(c.head_dim, 128 / el) : c.head_dim, parts = c.head_dim / part;
  const cuuint64_t dims[5] = {part, (cuuint64_t)c.page_size, parts, (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)cache->token_stride * el, (cuuint64_t)part * el, (cuuint64_t)cache->head_stride * el,
                                 (cuuint64_t)cache->page_stride * el};
  const cuuint32_t box[5] = {part, tokens, low || tokens == 64 ? parts : 1, 1, 1};
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  const CUtensorMapSwizzle swizzle = !swizzled          ? CU_TENSOR_MAP_SWIZZLE_NONE
                                     : part * el == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                        : CU_TENSOR_MAP_SWIZZLE_64B;
  const CUresult r = encode_tiled()(map, low ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, base, dims, strides, box,
                                    step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SS_ERR_CUDA, "cuTensorMapEncodeTiled refused the cache's layout");
  return SS_OK;
}

// Pointers and strides of a cache; e4m3 factors only where the plan has them.
ss_status check_cache(const ss_kv_plan* p, const ss_kv_cache* cache) {
  const int64_t per16 = p->c.cache_dtype == SS_E4M3 ? 16 : 8;
  if (!cache->k || !cache->v) return fail(SS_ERR_ARG, "the cache's keys and values are required");
  if (!aligned(cache->k, 16) || !aligned(cache->v, 16)) return fail(SS_ERR_ALIGN, "cache pointers must be 16-byte aligned");
  for (const int64_t s : {cache->page_stride, cache->token_stride, cache->head_stride}) {
    if (s < 1 || s > (1ll << 36)) return fail(SS_ERR_ARG, "cache strides must be in [1, 2^36] elements");
    if (s % per16 != 0) return fail(SS_ERR_ALIGN, "cache strides must be multiples of 16 bytes");
  }
  if (p->c.cache_dtype != SS_E4M3 && (cache->k_scale || cache->v_scale))
    return fail(SS_ERR_ARG, "k_scale and v_scale belong to an SS_E4M3 cache");
  return SS_OK;
}

ss_status check_pool(const ss_kv_pool* pool) {
  if (!pool || !pool->plan) return fail(SS_ERR_ARG, "pool and plan are required");
  if (pool->B < 1 || pool->B > pool->plan->c.max_rows) return fail(SS_ERR_ARG, "B must be in [1, max_rows]");
  if (!pool->block_table || !pool->kv_len || !pool->free_pages || !pool->free_count)
    return fail(SS_ERR_ARG, "block_table, kv_len, free_pages and free_count are required");
  return SS_OK;
}

ss::PagesParams pages_params(const ss_kv_pool* pool) {
  const ss_kv_plan* p = pool->plan;
  ss::PagesParams P = {};
  P.B = pool->B;
  P.max_tokens = std::min(pool->tokens, p->c.max_tokens);
  P.max_blocks = p->c.max_blocks;
  P.num_pages = p->c.num_pages;
  P.page_shift = p->page_shift;
  P.block_table = pool->block_table;
  P.kv_len = pool->kv_len;
  P.free_pages = pool->free_pages;
  P.free_count = pool->free_count;
  return P;
}

}  // namespace

extern "C" {

ss_status ss_kv_plan_create(ss_kv_plan** out, const ss_kv_config* config) {
  if (!out) return fail(SS_ERR_ARG, "plan pointer is NULL");
  *out = nullptr;
  if (!config) return fail(SS_ERR_ARG, "config is required");
  const ss_kv_config c = *config;
  if (c.max_rows < 1 || c.max_rows > 8192) return fail(SS_ERR_UNSUPPORTED, "max_rows must be in [1, 8192]");
  if (c.max_tokens < 1 || c.max_tokens > (1 << 24)) return fail(SS_ERR_UNSUPPORTED, "max_tokens must be in [1, 2^24]");
  if (c.max_new < 1) return fail(SS_ERR_ARG, "max_new must be >= 1");
  if (c.kv_heads < 1 || c.kv_heads > 1024 || c.q_heads < 1 || c.q_heads > 65536 || c.q_heads % c.kv_heads != 0)
    return fail(SS_ERR_UNSUPPORTED, "kv_heads must be in [1, 1024] and q_heads a multiple of it, at most 65536");
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return fail(SS_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)) != 0)
    return fail(SS_ERR_UNSUPPORTED, "page_size must be a power of two in [16, 1024]");
  if (c.num_pages < 1 || (int64_t)c.num_pages * c.page_size >= (1ll << 31) || c.max_blocks < 1 ||
      (int64_t)c.max_blocks * c.page_size >= (1ll << 31))
    return fail(SS_ERR_UNSUPPORTED, "num_pages and max_blocks must be >= 1 and below 2^31 / page_size");
  const int group = c.q_heads / c.kv_heads;
  if ((int64_t)c.max_tokens * group > (1 << 30)) return fail(SS_ERR_UNSUPPORTED, "max_tokens * q_heads / kv_heads must be at most 2^30");
  if (c.dtype != SS_BF16 && c.dtype != SS_F16) return fail(SS_ERR_ARG, "dtype must be SS_BF16 or SS_F16");
  if (c.cache_dtype != c.dtype && c.cache_dtype != SS_E4M3) return fail(SS_ERR_ARG, "cache_dtype must be dtype or SS_E4M3");
  int ndev = 0;
  cudaError_t e = cudaGetDeviceCount(&ndev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDeviceCount");
  if (c.device < 0 || c.device >= ndev) return fail(SS_ERR_ARG, "device ordinal out of range");
  if (!encode_tiled()) return fail(SS_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  const OnDevice on(c.device);
  int sms = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c.device);
  // the smallest row tile that holds a row's usual query rows: larger tiles waste products on rows that do not
  // exist, smaller ones read the keys once for each of several tiles
  const int64_t rows = (int64_t)c.max_new * group;
  const int row_tile = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  const ss::AttendKernel k = attend_kernel(c, row_tile);
  if (e == cudaSuccess) e = configure(c.device, k);
  if (e != cudaSuccess) return cuda_fail(e, "kernel attributes");
  ss_kv_plan* p = new (std::nothrow) ss_kv_plan();
  if (!p) return fail(SS_ERR_ARG, "out of host memory");
  p->c = c;
  p->page_shift = __builtin_ctz((unsigned)c.page_size);
  p->sms = sms;
  p->row_tile = row_tile;
  // a CTA for every place that the GPU has, or, for a small plan, for every two tiles there can be (ss_kv_work.cuh)
  const int64_t units = std::min<int64_t>((int64_t)c.max_tokens * group, c.max_rows + (int64_t)c.max_tokens * group / row_tile) * c.kv_heads;
  const int64_t line = units * ((int64_t)c.max_blocks * c.page_size / k.tile + 1 + k.unit_cost);
  p->attend_grid = (int)std::min<int64_t>((int64_t)k.ctas * sms, std::max<int64_t>(1, (line + 1) / 2));
  p->off_part = up256((size_t)3 * p->attend_grid * 4);
  p->off_ml = p->off_part + up256((size_t)2 * p->attend_grid * row_tile * c.head_dim * 4);
  p->ws_bytes = p->off_ml + up256((size_t)2 * p->attend_grid * row_tile * 16);
  *out = p;
  return SS_OK;
}

void ss_kv_plan_destroy(ss_kv_plan* plan) { delete plan; }

size_t ss_kv_workspace_bytes(const ss_kv_plan* plan) { return plan ? plan->ws_bytes : 0; }

ss_status ss_kv_append(const ss_kv_pool* pool, const int32_t* cu_new, int32_t* slots, int32_t* positions, int32_t* seq_len,
                       uint32_t* row_status) {
  const ss_status s = check_pool(pool);
  if (s != SS_OK) return s;
  if (pool->tokens < 0) return fail(SS_ERR_ARG, "tokens must be >= 0");
  if (!cu_new || !seq_len || !row_status || (pool->tokens > 0 && (!slots || !positions)))
    return fail(SS_ERR_ARG, "cu_new, slots, positions, seq_len and row_status are required");
  ss::PagesParams P = pages_params(pool);
  P.cu_new = cu_new;
  P.slots = slots;
  P.positions = positions;
  P.seq_len = seq_len;
  P.row_status = row_status;
  const OnDevice on(pool->plan->c.device);
  const Range range("ss_kv_append");
  const cudaError_t e = ss::kv_append_launch(P, static_cast<cudaStream_t>(pool->stream));
  return e == cudaSuccess ? SS_OK : cuda_fail(e, "ss_kv_append");
}

ss_status ss_kv_commit(const ss_kv_pool* pool, const int32_t* seq_len, const int32_t* counts, int32_t plus, const int32_t* finished) {
  const ss_status s = check_pool(pool);
  if (s != SS_OK) return s;
  if (!seq_len) return fail(SS_ERR_ARG, "seq_len is required");
  ss::PagesParams P = pages_params(pool);
  P.seq_len = const_cast<int32_t*>(seq_len);
  P.counts = counts;
  P.plus = plus;
  P.finished = finished;
  const OnDevice on(pool->plan->c.device);
  const Range range("ss_kv_commit");
  const cudaError_t e = ss::kv_commit_launch(P, static_cast<cudaStream_t>(pool->stream));
  return e == cudaSuccess ? SS_OK : cuda_fail(e, "ss_kv_commit");
}

ss_status ss_rope_store(const ss_rope_batch* b, const ss_kv_cache* cache) {
  if (!b || !b->plan || !cache) return fail(SS_ERR_ARG, "batch, plan and cache are required");
  const ss_kv_plan* p = b->plan;
  const ss_kv_config& c = p->c;
  if (b->T < 0 || b->T > c.max_tokens) return fail(SS_ERR_ARG, "T must be in [0, max_tokens]");
  if (b->T == 0) return SS_OK;
  if (!b->q || !b->k || !b->v || !b->q_out || !b->positions || !b->slots)
    return fail(SS_ERR_ARG, "q, k, v, q_out, positions and slots are required");
  if (b->rot_dim < 0 || b->rot_dim > c.head_dim || b->rot_dim % 16 != 0)
    return fail(SS_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16 in [0, head_dim]");
  if (b->rot_dim > 0 && !b->inv_freq) return fail(SS_ERR_ARG, "inv_freq is required");
  if (!(b->eps >= 0.0f)) return fail(SS_ERR_ARG, "eps must be >= 0");
  if (!std::isfinite(b->rope_scale)) return fail(SS_ERR_ARG, "rope_scale must be finite");
  const int64_t wq = (int64_t)c.q_heads * c.head_dim, wk = (int64_t)c.kv_heads * c.head_dim;
  if (b->q_stride < wq || b->q_out_stride < wq || b->k_stride < wk || b->v_stride < wk)
    return fail(SS_ERR_ARG, "a token stride is smaller than its heads");
  if (b->q_stride % 8 || b->q_out_stride % 8 || b->k_stride % 8 || b->v_stride % 8)
    return fail(SS_ERR_ALIGN, "token strides must be multiples of 8 elements");
  for (const void* x : {b->q, b->k, b->v, static_cast<const void*>(b->q_out), b->q_weight, b->k_weight})
    if (!aligned(x, 16)) return fail(SS_ERR_ALIGN, "q, k, v, q_out and the weights must be 16-byte aligned");
  const ss_status s = check_cache(p, cache);
  if (s != SS_OK) return s;
  ss::RopeParams P = {};
  P.T = b->T;
  P.hq = c.q_heads;
  P.hkv = c.kv_heads;
  P.rot = b->rot_dim;
  P.interleaved = b->interleaved != 0;
  P.page_shift = p->page_shift;
  P.num_slots = (long long)c.num_pages * c.page_size;
  P.q = b->q;
  P.k = b->k;
  P.v = b->v;
  P.qw = b->q_weight;
  P.kw = b->k_weight;
  P.q_stride = b->q_stride;
  P.k_stride = b->k_stride;
  P.v_stride = b->v_stride;
  P.qo_stride = b->q_out_stride;
  P.eps = b->eps;
  P.rope_scale = b->rope_scale;
  P.inv_freq = b->inv_freq;
  P.positions = b->positions;
  P.slots = b->slots;
  P.q_out = b->q_out;
  P.k_cache = cache->k;
  P.v_cache = cache->v;
  P.page_stride = cache->page_stride;
  P.token_stride = cache->token_stride;
  P.head_stride = cache->head_stride;
  P.k_scale = cache->k_scale;
  P.v_scale = cache->v_scale;
  const OnDevice on(c.device);
  const Range range("ss_rope_store");
  const cudaError_t e =
      ss::kv_rope_launch(P, c.dtype == SS_BF16, c.cache_dtype == SS_E4M3, c.head_dim, p->sms, static_cast<cudaStream_t>(b->stream));
  return e == cudaSuccess ? SS_OK : cuda_fail(e, "ss_rope_store");
}

ss_status ss_rope_frequencies(double* inv_freq, int32_t rot_dim, double base, double factor, int32_t original_len, double low_turns,
                              double high_turns) {
  if (!inv_freq) return fail(SS_ERR_ARG, "inv_freq is required");
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 65536) return fail(SS_ERR_ARG, "rot_dim must be even, in [2, 65536]");
  if (!(base > 0.0) || !std::isfinite(base)) return fail(SS_ERR_ARG, "base must be positive and finite");
  if (!(factor >= 1.0) || !std::isfinite(factor)) return fail(SS_ERR_ARG, "factor must be at least 1 and finite");
  if (original_len < 0) return fail(SS_ERR_ARG, "original_len must be >= 0");
  if (original_len > 0 && !(low_turns >= 0.0 && high_turns > low_turns)) return fail(SS_ERR_ARG, "need 0 <= low_turns < high_turns");
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double stay = 0.0;  // share of the angle that is not stretched
    if (original_len > 0) {
      const double turns = original_len * f / (2.0 * 3.14159265358979323846);
      stay = std::min(1.0, std::max(0.0, (turns - low_turns) / (high_turns - low_turns)));
    }
    inv_freq[i] = f * stay + f / factor * (1.0 - stay);
  }
  return SS_OK;
}

ss_status ss_attend(const ss_attend_batch* b, const ss_kv_cache* cache) {
  if (!b || !b->plan || !cache) return fail(SS_ERR_ARG, "batch, plan and cache are required");
  const ss_kv_plan* p = b->plan;
  const ss_kv_config& c = p->c;
  if (b->B < 1 || b->B > c.max_rows) return fail(SS_ERR_ARG, "B must be in [1, max_rows]");
  if (b->tokens < 0) return fail(SS_ERR_ARG, "tokens must be >= 0");
  if (b->tokens == 0) return SS_OK;
  if (!b->q || !b->cu_new || !b->seq_len || !b->block_table || !b->out || !b->row_status)
    return fail(SS_ERR_ARG, "q, cu_new, seq_len, block_table, out and row_status are required");
  if (!(b->scale > 0.0f) || !std::isfinite(b->scale * 1.4426951f)) return fail(SS_ERR_ARG, "scale must be positive and finite");
  if (b->window < 0 || b->sinks < 0) return fail(SS_ERR_ARG, "window and sinks must be >= 0");
  const int64_t wq = (int64_t)c.q_heads * c.head_dim;
  if (b->q_stride < wq || b->out_stride < wq) return fail(SS_ERR_ARG, "a token stride is smaller than its heads");
  if (b->q_stride % 8 || b->out_stride % 8) return fail(SS_ERR_ALIGN, "token strides must be multiples of 8 elements");
  if (!aligned(b->q, 16) || !aligned(b->out, 16)) return fail(SS_ERR_ALIGN, "q and out must be 16-byte aligned");
  ss_status s = check_cache(p, cache);
  if (s != SS_OK) return s;
  if (!b->workspace || b->workspace_bytes < p->ws_bytes)
    return fail(SS_ERR_WORKSPACE, "workspace missing or smaller than ss_kv_workspace_bytes()");
  if (!aligned(b->workspace, 256)) return fail(SS_ERR_ALIGN, "workspace must be 256-byte aligned");
  const OnDevice on(c.device);
  CUtensorMap mk, mv;
  const ss::AttendKernel k = attend_kernel(c, p->row_tile);
  s = encode(&mk, p, cache, cache->k, k.swizzled);
  if (s == SS_OK) s = encode(&mv, p, cache, cache->v, k.swizzled);
  if (s != SS_OK) return s;
  const int32_t longest = c.max_blocks * c.page_size;
  ss::AttendParams P = {};
  P.q = b->q;
  P.out = b->out;
  P.lse = b->lse;
  P.q_stride = b->q_stride;
  P.out_stride = b->out_stride;
  P.cu_new = b->cu_new;
  P.seq_len = b->seq_len;
  P.block_table = b->block_table;
  P.row_status = b->row_status;
  P.k_scale = cache->k_scale;
  P.v_scale = cache->v_scale;
  P.scale_log2 = (float)((double)b->scale * 1.4426950408889634);
  P.B = b->B;
  P.hkv = c.kv_heads;
  P.group = c.q_heads / c.kv_heads;
  P.max_blocks = c.max_blocks;
  P.num_pages = c.num_pages;
  P.page_shift = p->page_shift;
  P.max_tokens = std::min(b->tokens, c.max_tokens);
  P.window = b->window >= longest ? 0 : b->window;  // a window that reaches every token is none
  P.sinks = P.window ? std::min(b->sinks, longest) : 0;
  char* w = static_cast<char*>(b->workspace);
  P.counters = reinterpret_cast<uint32_t*>(w);
  P.part = reinterpret_cast<float*>(w + p->off_part);
  P.ml = reinterpret_cast<float4*>(w + p->off_ml);
  P.spin_limit = kSpin;
  P.rows = p->row_tile;
  P.slots = k.slots;
  P.raw_slots = k.raw_slots;
  P.q_bufs = k.q_bufs;
  P.unit_cost = k.unit_cost;
  P.tile_shift = k.tile == 64 ? 6 : 7;
  while ((1u << P.group_shift) < (uint32_t)P.group) ++P.group_shift;
  P.group_mul = (uint32_t)(((1ull << 32) * ((1ull << P.group_shift) - P.group)) / P.group + 1);
  void* args[] = {&P, &mk, &mv};
  const Range range("ss_attend");
  const cudaError_t e = cudaLaunchKernel(k.fn, dim3(p->attend_grid), dim3(k.threads), args, k.smem, static_cast<cudaStream_t>(b->stream));
  return e == cudaSuccess ? SS_OK : cuda_fail(e, "ss_attend");
}

}  // extern "C"
