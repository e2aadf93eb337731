// Internal declarations shared by the KV-cache translation units: the plan,
// kernel parameter blocks and the launchers of each kernel.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ss_kv.h"

struct ss_kv_plan {
  ss_kv_config c;
  int page_shift;
  int sms;
  int row_tile;         // query rows per unit of ss_attend: 16, 32, 64 or (16-bit caches) 128
  int attend_grid;      // persistent CTAs of ss_attend
  size_t off_part, off_ml, ws_bytes;  // workspace: counters at 0, partial outputs, their (max, sum)
};

namespace ss {

struct PagesParams {
  int B, max_tokens, max_blocks, num_pages, page_shift;
  int32_t* block_table;
  int32_t* kv_len;
  int32_t* free_pages;
  int32_t* free_count;
  const int32_t* cu_new;
  int32_t *slots, *positions, *seq_len;
  uint32_t* row_status;
  const int32_t *counts, *finished;
  int plus;
};
cudaError_t kv_pages_configure();
cudaError_t kv_append_launch(const PagesParams& P, cudaStream_t st);
cudaError_t kv_commit_launch(const PagesParams& P, cudaStream_t st);

struct RopeParams {
  int T, hq, hkv, rot, interleaved, page_shift;
  long long num_slots;
  const void *q, *k, *v, *qw, *kw;
  long long q_stride, k_stride, v_stride, qo_stride;
  float eps, rope_scale;
  const double* inv_freq;
  const int32_t *positions, *slots;
  void *q_out, *k_cache, *v_cache;
  long long page_stride, token_stride, head_stride;
  const float *k_scale, *v_scale;
};
cudaError_t kv_rope_launch(const RopeParams& P, bool bf16, bool e4m3, int head_dim, int sms, cudaStream_t st);

struct AttendParams {
  const void* q;
  void* out;
  float* lse;
  long long q_stride, out_stride;
  const int32_t *cu_new, *seq_len, *block_table;
  uint32_t* row_status;
  const float *k_scale, *v_scale;
  float scale_log2;     // scale * log2(e)
  int B, hkv, group, max_blocks, num_pages, page_shift, max_tokens, window, sinks;
  int rows, slots, raw_slots, q_bufs;  // query rows of a unit, tiles in the rings, query buffers
  int tile_shift;           // log2 of a tile's keys
  int unit_cost;            // tiles' worth of time that starting and ending a unit takes
  uint32_t group_mul, group_shift;  // x / group = (umulhi(x, mul) + x) >> shift for x < 2^31
  uint32_t* counters;   // [3 * grid] arrivals at groups of pieces, then at units (ss_kv_join.cuh)
  float* part;          // [2 * grid][head_dim / 4][row_tile][4] outputs of pieces
  float4* ml;           // [2 * grid][row_tile] their maximum (of log2), the sum that divides and the sum of the weights
  uint32_t spin_limit;
};
// The kernel of a head size, types and row tile, its block size, ring, query buffers and shared memory.
struct AttendKernel {
  const void* fn;
  int threads, slots, raw_slots, q_bufs, ctas, tile;  // ctas: per SM; tile: keys of a tile
  size_t smem;
  int unit_cost;  // see ss_kv_work.cuh
  bool swizzled;  // how the copies lay tiles out in shared memory
};
AttendKernel kv_attend_bf16(int head_dim, int row_tile);       // bf16 activations, bf16 cache
AttendKernel kv_attend_f16(int head_dim, int row_tile);        // f16, f16
AttendKernel kv_attend_bf16_e4m3(int head_dim, int row_tile);  // bf16, e4m3
AttendKernel kv_attend_f16_e4m3(int head_dim, int row_tile);   // f16, e4m3

}  // namespace ss
