// The factors of an 8-bit cache with one for each block of tokens and key head.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>

#include "ss_kv_common.cuh"

namespace ss {

// Exponents of the factors that ss_kv_store_blocks writes.  What a factor can reach keeps every product of a factor, a
// weight and a value inside 32 bits.
constexpr int kLowestBlock = -40, kHighestBlock = 40;

// A factor as the kernels take it: inside the range whatever the memory holds (that of a block nothing was stored in
// may be anything; NaN becomes the lowest).
__device__ __forceinline__ float block_factor(float x) { return fminf(fmaxf(x, 0x1p-40f), 0x1p40f); }

namespace kv {

// How attention takes factors.  With k8, v8 the held bytes' values and ks, vs a block's factors, a weight is
// w_t = 2^(c ks q.k8_t - m) and o = sum w_t vs v8_t / sum w_t.  The kernels keep u_t = w_t vs instead, as
// u_t = 2^(c ks q.k8_t + log2 vs - m) with m near the largest exponent of u: the product with the values is then that of
// their bytes, u fits 16 bits whatever the factors are, and sum w_t is the sum over blocks of sum u_t / vs.  A group of 16
// keys has one factor each, so that costs nothing a score.  m is a whole number, as log2 vs is where the factor is a
// power of two, so that the exponent loses no bits.
//
// Of the keys of some tiles, by groups of 16: ks, log2 vs, 1 / vs.
template <int TILES, int GROUPS>
struct Factors {
  float k[TILES][GROUPS], log[TILES][GROUPS], back[TILES][GROUPS];
};
struct NoFactors {};

__device__ __forceinline__ float log2_of(float x) {  // x normal; exact for powers of two
  const uint32_t bits = __float_as_uint(x), part = bits & 0x7fffffu;
  float y = 0.0f;
  if (part) asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(__uint_as_float(part | 0x3f800000u)));
  return y + (float)((int)(bits >> 23) - 127);
}

// The factor of a block's scores.  Held bytes times f16 queries stay below 2^33: factors this small make every score 0, and
// 0 times a hidden key's -inf, or an infinite factor times 0, must not be NaN.
__device__ __forceinline__ float factor_of(float scale, float k) { return fminf(fmaxf(scale * k, FLT_MIN), FLT_MAX); }

// A load warp's factors of one copy (of up to 64 tokens: 4 groups) of its batch.
struct CopyFactors {
  float k[4], v[4];
  // Those of the copy that starts at place `tok` of page `id`; ones where `there` is false.
  __device__ __forceinline__ void fetch(const AttendParams& P, bool there, int id, int h, int tok, int groups) {
    const long long at = ((long long)id * P.hkv + h) << (P.page_shift - P.block_shift);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      k[n] = v[n] = 1.0f;
      if (there && n < groups) {
        const int b = (tok + 16 * n) >> P.block_shift;
        k[n] = __ldg(P.k_blocks + at + b);
        v[n] = __ldg(P.v_blocks + at + b);
      }
    }
  }
  template <class F>
  __device__ __forceinline__ void write(F& f, int tile, int first, int groups) const {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if (n >= groups) continue;
      const float y = block_factor(v[n]);
      f.k[tile][first + n] = block_factor(k[n]);
      f.log[tile][first + n] = log2_of(y);
      f.back[tile][first + n] = __frcp_rn(y);
    }
  }
};

}  // namespace kv
}  // namespace ss
