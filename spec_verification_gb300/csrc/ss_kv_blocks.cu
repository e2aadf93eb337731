// ss_kv_store_blocks and ss_kv_load_blocks: new tokens into an 8-bit cache with
// a factor for each block of tokens and key head, and held tokens back out.
//
// A run is what one call writes of one block: consecutive new tokens of a row.
// Its factor is the least power of two 2^e with max |x| <= 448 * 2^e, or the
// block's old one where that is larger and tokens before the run are kept; if
// the factor grows, the kept tokens' bytes are rounded anew.  Powers of two,
// because the kept bytes then only lose what falls below e4m3's normal range,
// however often a block grows, and because x / 2^e is exact, so that a value
// is rounded once.  A whole power of two costs no precision: e4m3 has the same
// relative step from 2^-6 to 448.
//
// Every value is read and written once (a block's kept tokens where its factor
// grows): HBM bandwidth is the bound, and latency for a step's single tokens.
// Measured, 8 heads of 128: 24 rows x 1 token 3.8 us (launch, counting the runs,
// four dependent reads); 16000 tokens of one prompt 16.6 us, 5.9 TB/s; 40000
// tokens back 40.8 us, 6.0 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "ss_kv_blocks.cuh"
#include "ss_kv_common.cuh"

namespace ss {
namespace {

constexpr int kNT = 128, kWarps = kNT / 32;
constexpr int kGroups = 256;  // of 32 rows: 8192

template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 of(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
  static __device__ __forceinline__ uint32_t to(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // the larger of each half of two pairs that have no signs; a number rather than NaN
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 of(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  // Beyond 65504 as 65504 with its sign, NaN as NaN: of f16 values those from 63488 on are held as 65536.
  static __device__ __forceinline__ float within(float x) { return fabsf(x) > 65504.0f ? copysignf(65504.0f, x) : x; }
  static __device__ __forceinline__ uint32_t to(float a, float b) {
    const __half2 h = __floats2half2_rn(within(a), within(b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
  }
};

// Two values as e4m3, rounded to nearest, what passes 448 (infinities too) as 448 with its sign, NaN as NaN.
__device__ __forceinline__ uint32_t to8(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from8(uint32_t w) {  // of the low 16 bits
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// The least e in range with x <= 448 * 2^e, 448 = 1.75 * 2^8, for finite x >= 0.
__device__ __forceinline__ int exponent_of(float x) {
  const uint32_t bits = __float_as_uint(x);
  const int e = (int)(bits >> 23) - 127;  // (numbers below 2^-126 are far below the range)
  return min(max(e - 8 + ((bits & 0x7fffffu) > 0x600000u), kLowestBlock), kHighestBlock);
}

// A row of a call; n == 0: nothing to store.
struct StoreRow {
  int q0, n, held;
  uint32_t status;
};
__device__ __forceinline__ StoreRow store_row(const StoreParams& P, int r) {
  StoreRow w;
  w.q0 = P.cu_new[r];
  const int q1 = P.cu_new[r + 1];
  w.n = q1 - w.q0;
  w.held = P.kv_len[r];
  w.status = 0;
  const int len = P.seq_len[r];
  if (w.q0 < 0 || q1 < w.q0 || q1 > P.max_tokens) {
    w.n = 0;
    w.status = SS_ST_CAPACITY;
  } else if (w.held < 0 || len < 0 || len > P.max_blocks << P.page_shift) {
    w.n = 0;
    w.status = SS_ST_BAD_PARAM;
  } else if (len < w.held || len - w.held != w.n) {
    w.n = 0;  // not served by the append
  }
  return w;
}
__device__ __forceinline__ int runs_of(const StoreParams& P, const StoreRow& w) {
  return w.n == 0 ? 0 : ((w.held + w.n - 1) >> P.block_shift) - (w.held >> P.block_shift) + 1;
}

// The group of threads that has a unit: a warp, or (large blocks) the CTA.
template <bool WIDE>
struct Group {
  static constexpr int kSize = WIDE ? kNT : 32;
  static __device__ __forceinline__ int thread() { return WIDE ? threadIdx.x : threadIdx.x & 31; }
  static __device__ __forceinline__ float max(float x, float* room) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (!WIDE) return x;
    __syncthreads();  // the last unit's maxima have been read
    if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x = fmaxf(x, room[w]);
    return x;
  }
};

// Units: (run, keys or values, head), runs in order of rows.  Every CTA counts the runs of all rows, 32 rows at a time, and
// its groups of threads take the units in turn; a group holds 32 rows, a row to a lane, until a run lies past them.  What a
// unit waits for, one after the other: its values and its page, asked for together; its old factor, where it has one.
// Count: of runs; 64 bits where they could pass 32, as rows that overlap (sums that go up and down) can.  Always 64 bits cost 2 to
// 5 % (300 rows of 8 tokens 6.2 -> 6.6 us, 8192 of one 120 -> 122).
template <class T, int D, bool WIDE, int LOADS, class Count>
__global__ void __launch_bounds__(kNT) store_kernel(const StoreParams P) {
  using G = Group<WIDE>;
  __shared__ Count first[kGroups + 1];  // runs before each 32 rows
  __shared__ float room[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = (P.B + 31) / 32;
  auto row_of = [&](int r) {
    StoreRow w = {0, 0, 0, 0};
    return r < P.B ? store_row(P, r) : w;
  };
#pragma unroll 4
  for (int g = warp; g < groups; g += kWarps) {
    const StoreRow w = row_of(32 * g + lane);
    if (w.status && blockIdx.x == 0) atomicOr(&P.row_status[32 * g + lane], w.status);
    const int sum = __reduce_add_sync(0xffffffffu, runs_of(P, w));
    if (lane == 0) first[g + 1] = sum;
  }
  __syncthreads();
  if (warp == 0) {  // eight groups to a lane
    Count n[kGroups / 32], mine = 0;
#pragma unroll
    for (int k = 0; k < kGroups / 32; ++k) {
      const int g = lane * (kGroups / 32) + k;
      n[k] = g < groups ? first[g + 1] : 0;
      mine += n[k];
    }
    Count sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Count y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += y;
    }
    sum -= mine;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kGroups / 32; ++k) {
      sum += n[k];
      first[lane * (kGroups / 32) + k + 1] = sum;
    }
    if (lane == 0) first[0] = 0;
  }
  __syncthreads();
  const int kinds = 2 * P.hkv, at = G::thread(), block = 1 << P.block_shift;
  const long long units = (long long)first[kGroups] * kinds, step = (long long)gridDim.x * (kNT / G::kSize);
  constexpr int kPer = D / 8;  // 16-byte pieces of a new token's head
  int group = -1, runs = 0;  // the 32 rows that are looked at, runs of this lane's
  Count upto = 0;            // and up to them
  StoreRow mine = {0, 0, 0, 0};
  for (long long u = (long long)blockIdx.x * (kNT / G::kSize) + (WIDE ? 0 : warp); u < units; u += step) {
    const Count run = (Count)(u / kinds);
    const int kind = (int)(u - (long long)run * kinds), h = kind % P.hkv;
    const bool values = kind >= P.hkv;
    if (group < 0 || run >= first[group + 1]) {
      group = 0;
#pragma unroll
      for (int s = kGroups / 2; s > 0; s >>= 1)
        if (first[group + s] <= run) group += s;
      mine = row_of(32 * group + lane);
      runs = upto = runs_of(P, mine);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Count y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      upto += first[group];
    }
    const int owner = __ffs(__ballot_sync(0xffffffffu, upto > run)) - 1;
    StoreRow w;
    w.q0 = __shfl_sync(0xffffffffu, mine.q0, owner);
    w.n = __shfl_sync(0xffffffffu, mine.n, owner);
    w.held = __shfl_sync(0xffffffffu, mine.held, owner);
    const int r = 32 * group + owner, left = (int)(run - __shfl_sync(0xffffffffu, upto - runs, owner));
    // tokens [p0, p1) of the row, in one block
    const int blk = (w.held >> P.block_shift) + left;
    const int p0 = max(w.held, blk << P.block_shift), p1 = min(w.held + w.n, (blk + 1) << P.block_shift);
    const int page = P.block_table[(long long)r * P.max_blocks + (p0 >> P.page_shift)];
    const int place = p0 & ((1 << P.page_shift) - 1), kept = place & (block - 1), count = (p1 - p0) * kPer;
    const long long stride = values ? P.v_stride : P.k_stride;
    const T* src = static_cast<const T*>(values ? P.v : P.k) + (w.q0 + p0 - w.held) * stride + h * D;
    auto load = [&](uint4 (&x)[LOADS], int i0) {
#pragma unroll
      for (int n = 0; n < LOADS; ++n) {
        const int i = i0 + at + n * G::kSize;
        x[n] = make_uint4(0u, 0u, 0u, 0u);
        if (i < count) x[n] = __ldg(reinterpret_cast<const uint4*>(src + i / kPer * stride + i % kPer * 8));
      }
    };
    uint4 x[LOADS];
    load(x, 0);
    if ((unsigned)page >= (unsigned)P.num_pages) {
      if (at == 0) atomicOr(&P.row_status[r], (uint32_t)SS_ST_KV_PAGE);
      continue;
    }
    unsigned char* dst = static_cast<unsigned char*>(values ? P.v_cache : P.k_cache) + page * P.page_stride + (place - kept) * P.token_stride +
                         h * P.head_stride;
    float* factor = (values ? P.v_scale : P.k_scale) + ((long long)page * P.hkv + h) * (1 << (P.page_shift - P.block_shift)) + (place >> P.block_shift);
    const float old = kept ? *factor : 0.0f;
    // the largest |x|, of pairs of 16 bits; an infinity among them has it looked for again without
    uint32_t most = 0;
    for (int i0 = 0; i0 < count; i0 += LOADS * G::kSize) {
      if (i0 > 0) load(x, i0);
#pragma unroll
      for (int n = 0; n < LOADS; ++n)
        for (const uint32_t y : {x[n].x, x[n].y, x[n].z, x[n].w}) most = Pair<T>::larger(most, y & 0x7fff7fffu);
    }
    float top = G::max(fmaxf(Pair<T>::of(most).x, Pair<T>::of(most).y), room);
    if (top == INFINITY) {
      top = 0.0f;
      for (int i0 = 0; i0 < count; i0 += LOADS * G::kSize) {
        if (count > LOADS * G::kSize) load(x, i0);
#pragma unroll
        for (int n = 0; n < LOADS; ++n) {
          for (const uint32_t y : {x[n].x, x[n].y, x[n].z, x[n].w}) {
            const float2 v = Pair<T>::of(y & 0x7fff7fffu);
            if (v.x < INFINITY) top = fmaxf(top, v.x);  // (false for NaN)
            if (v.y < INFINITY) top = fmaxf(top, v.y);
          }
        }
      }
      top = G::max(top, room);
    }
    int e = exponent_of(top);
    const int before = (int)(__float_as_uint(block_factor(old)) >> 23) - 127;
    if (kept) e = max(e, before);
    if (kept && e != before) {
      const float by = power(before - e);
      const int pieces = kept * (D / 16);
      for (int i = at; i < pieces; i += G::kSize) {
        uint4* line = reinterpret_cast<uint4*>(dst + (long long)(i / (D / 16)) * P.token_stride + i % (D / 16) * 16);
        uint4 y = *line;
        uint32_t* ys = &y.x;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float2 a = from8(ys[n]), b = from8(ys[n] >> 16);
          ys[n] = to8(a.x * by, a.y * by) | to8(b.x * by, b.y * by) << 16;
        }
        *line = y;
      }
    }
    if (at == 0) *factor = power(e);
    const float down = power(-e);
    for (int i0 = 0; i0 < count; i0 += LOADS * G::kSize) {
      if (count > LOADS * G::kSize) load(x, i0);
#pragma unroll
      for (int n = 0; n < LOADS; ++n) {
        const int i = i0 + at + n * G::kSize;
        if (i >= count) break;
        const float2 a = Pair<T>::of(x[n].x), b = Pair<T>::of(x[n].y), c = Pair<T>::of(x[n].z), d = Pair<T>::of(x[n].w);
        *reinterpret_cast<uint2*>(dst + (long long)(kept + i / kPer) * P.token_stride + i % kPer * 8) =
            make_uint2(to8(a.x * down, a.y * down) | to8(b.x * down, b.y * down) << 16, to8(c.x * down, c.y * down) | to8(d.x * down, d.y * down) << 16);
      }
    }
  }
}

// A thread: 16 values of a token and head.
template <class T, int D>
__global__ void __launch_bounds__(256) load_kernel(const LoadParams P) {
  constexpr int kPer = D / 16;
  const int per_token = P.hkv * kPer;
  const long long items = (long long)P.T * per_token;
  const bool values = blockIdx.y != 0;
  const unsigned char* cache = static_cast<const unsigned char*>(values ? P.v_cache : P.k_cache);
  const float* scale = values ? P.v_scale : P.k_scale;
  T* out = static_cast<T*>(values ? P.v_out : P.k_out);
  const long long stride = values ? P.v_stride : P.k_stride;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < items; i += (long long)gridDim.x * blockDim.x) {
    const int t = (int)(i / per_token), rest = (int)(i - (long long)t * per_token), h = rest / kPer, piece = rest % kPer;
    const int slot = P.slots[t];
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (slot >= 0 && slot < P.num_slots) {
      const int page = slot >> P.page_shift, place = slot & ((1 << P.page_shift) - 1);
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(cache + page * P.page_stride + place * P.token_stride + h * P.head_stride + piece * 16));
      const float f = block_factor(__ldg(scale + ((long long)page * P.hkv + h) * (1 << (P.page_shift - P.block_shift)) + (place >> P.block_shift)));
      auto pair = [&](uint32_t w) {
        const float2 a = from8(w);
        return Pair<T>::to(a.x * f, a.y * f);
      };
      lo = make_uint4(pair(x.x), pair(x.x >> 16), pair(x.y), pair(x.y >> 16));
      hi = make_uint4(pair(x.z), pair(x.z >> 16), pair(x.w), pair(x.w >> 16));
    }
    uint4* to = reinterpret_cast<uint4*>(out + t * stride + h * D + piece * 16);
    to[0] = lo;
    to[1] = hi;
  }
}

template <class T, int D, class Count>
cudaError_t store(const StoreParams& P, int sms, cudaStream_t st) {
  // no more CTAs than there can be units, and no more than stay on the GPU (measured, 16000 tokens of one row, 5, 6, 8 an SM:
  // 17.0, 16.6, 18.7 us)
  // a warp to a unit whose values it can hold, in 8 or 16 loads of 16 bytes a lane; else the CTA
  const int values = D << P.block_shift;
  const bool wide = values > 16 * 32 * 8;
  const long long units = 2ll * P.hkv * (2ll * P.B + ((long long)P.max_tokens >> P.block_shift));
  const int grid = (int)std::min<long long>(wide ? units : (units + kWarps - 1) / kWarps, 6ll * sms);
  if (wide) store_kernel<T, D, true, 8, Count><<<grid, kNT, 0, st>>>(P);
  else if (values > 8 * 32 * 8) store_kernel<T, D, false, 16, Count><<<grid, kNT, 0, st>>>(P);
  else store_kernel<T, D, false, 8, Count><<<grid, kNT, 0, st>>>(P);
  return cudaGetLastError();
}
template <class T, int D>
cudaError_t store(const StoreParams& P, int sms, cudaStream_t st) {
  // a row has at most max_tokens / block + 2 runs, wherever the others are
  const long long runs = P.B * (((long long)P.max_tokens >> P.block_shift) + 2);
  return runs < 1ll << 31 ? store<T, D, int>(P, sms, st) : store<T, D, long long>(P, sms, st);
}
template <class T, int D>
cudaError_t load(const LoadParams& P, int sms, cudaStream_t st) {
  const long long items = (long long)P.T * P.hkv * (D / 16);
  const int grid = (int)std::min<long long>((items + 255) / 256, 16ll * sms);
  load_kernel<T, D><<<dim3(grid, 2), 256, 0, st>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t kv_store_blocks_launch(const StoreParams& P, bool bf16, int head_dim, int sms, cudaStream_t st) {
  if (bf16)
    return head_dim == 64    ? store<__nv_bfloat16, 64>(P, sms, st)
           : head_dim == 128 ? store<__nv_bfloat16, 128>(P, sms, st)
                             : store<__nv_bfloat16, 256>(P, sms, st);
  return head_dim == 64 ? store<__half, 64>(P, sms, st) : head_dim == 128 ? store<__half, 128>(P, sms, st) : store<__half, 256>(P, sms, st);
}
cudaError_t kv_load_blocks_launch(const LoadParams& P, bool bf16, int head_dim, int sms, cudaStream_t st) {
  if (bf16)
    return head_dim == 64    ? load<__nv_bfloat16, 64>(P, sms, st)
           : head_dim == 128 ? load<__nv_bfloat16, 128>(P, sms, st)
                             : load<__nv_bfloat16, 256>(P, sms, st);
  return head_dim == 64 ? load<__half, 64>(P, sms, st) : head_dim == 128 ? load<__half, 128>(P, sms, st) : load<__half, 256>(P, sms, st);
}

}  // namespace ss
