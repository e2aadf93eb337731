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

// A factor as the kernels take it: a power of two inside the range whatever the memory holds (that of a block nothing was
// stored in may be anything; NaN becomes the lowest).
__device__ __forceinline__ float block_factor(float x) {
  return __uint_as_float(__float_as_uint(fminf(fmaxf(x, 0x1p-40f), 0x1p40f)) & 0x7f800000u);
}

namespace kv {

// How attention takes factors.  With k8, v8 the held bytes' values and ks, vs a block's factors, a weight is
// w_t = 2^(c ks q.k8_t - m) and o = sum w_t vs v8_t / sum w_t.  The kernels keep u_t = w_t vs instead, as
// u_t = 2^(c ks q.k8_t + log2 vs - m) with m near the largest exponent of u: the product with the values is then that of
// their bytes, u fits 16 bits whatever the factors are, and sum w_t is the sum over blocks of sum u_t / vs.  A group of 16
// keys has one factor each, so that costs nothing a score.  log2 vs - m is rounded once for a group, to half a step of 32
// bits at m, as a score of that size is.  (m is not made a whole number to spare that: the largest weight would then be no
// power of two, and its rounding to 16 bits the error of every row with one key that dominates.)
//
// Of the keys of some tiles, by groups of 16: ks and vs.
template <int TILES, int GROUPS>
struct alignas(16) Factors {
  float k[TILES][GROUPS], v[TILES][GROUPS];
};

// The factor of a block's scores.  Held bytes times f16 queries stay below 2^33: factors this small make every score 0, and
// 0 times a hidden key's -inf must not be NaN; nor may 0 times infinity, which scale_of leaves no room for.
__device__ __forceinline__ float factor_of(float scale, float k) { return fmaxf(scale * k, FLT_MIN); }
__device__ __forceinline__ float scale_of(float scale) { return fminf(scale, 0x1p80f); }
// log2 and reciprocal of a power of two
__device__ __forceinline__ float log2_of(float x) { return (float)((int)(__float_as_uint(x) >> 23) - 127); }
__device__ __forceinline__ float back_of(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

// N neighbouring factors.
template <int N>
__device__ __forceinline__ void read_factors(float (&to)[N], const float* from) {
  if constexpr (N == 4) {
    const float4 y = *reinterpret_cast<const float4*>(from);
    to[0] = y.x;
    to[1] = y.y;
    to[2] = y.z;
    to[3] = y.w;
  } else if constexpr (N == 2) {
    const float2 y = *reinterpret_cast<const float2*>(from);
    to[0] = y.x;
    to[1] = y.y;
  } else {
    to[0] = *from;
  }
}

// A load warp's factors of one copy (of up to 64 tokens: 4 groups) of its batch.
struct CopyFactors {
  float k[4], v[4];
  // Asks for those of the copy that starts at place `tok` of page `id`; ones where `there` is false.
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
    if (groups == 4) {
      *reinterpret_cast<float4*>(&f.k[tile][first]) = make_float4(block_factor(k[0]), block_factor(k[1]), block_factor(k[2]), block_factor(k[3]));
      *reinterpret_cast<float4*>(&f.v[tile][first]) = make_float4(block_factor(v[0]), block_factor(v[1]), block_factor(v[2]), block_factor(v[3]));
      return;
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (n >= groups) continue;
      f.k[tile][first + n] = block_factor(k[n]);
      f.v[tile][first + n] = block_factor(v[n]);
    }
  }
};

}  // namespace kv
}  // namespace ss
