// ss_rope_store: norms of query and key heads, rotary positions, queries out,
// keys and values into the paged cache, in one pass.
//
// Per head x: y = x * rsqrt(mean x^2 + eps) * w, then each pair (a, b) is
// turned by angle = position * inv_freq: (a cos - b sin, b cos + a sin).
// Every value is read once and written once, so HBM bandwidth is the bound;
// the work per value is a few FMAs.  The angle is what could cost more: sin
// and cos of one pair serve every head of a token, so a CTA computes them
// once per token into shared memory and its threads keep those of their own
// eight values in registers over all the heads they visit.
//
// Angles: inv_freq / (2 pi) is turned into a 64-bit fixed-point fraction of a
// turn, whose product with the position modulo 2^64 is the exact fraction of
// the position's turn (error below position * 2^-61 turns), for near and far
// positions alike; its distance to the nearest quarter turn goes through
// fp32 sin and cos of at most pi / 4.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "ss_kv_common.cuh"

namespace ss {
namespace {

constexpr int kNT = 256;

__device__ __forceinline__ void unpack(uint32_t w, float& a, float& b, __nv_bfloat16) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack(uint32_t w, float& a, float& b, __half) {
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&w));
  a = f.x;
  b = f.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (cos, sin) of position * f radians.  f = m64 * 2^(e - 63) with m64 its
// mantissa at the top of 64 bits; f / (2 pi) * 2^64 = (m64 * K >> 64) * 2^(e + 1),
// K = 2^64 / (2 pi).
__device__ __forceinline__ float2 turn_of(double f, int position) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const int be = (int)(bits >> 52) & 0x7ff;
  unsigned long long fix = 0;
  if (be != 0) {
    const unsigned long long m64 = ((bits & 0xfffffffffffffull) | 0x10000000000000ull) << 11;
    const unsigned long long hi = __umul64hi(m64, 2935890503282001226ull);
    const int up = be - 1022;
    fix = up >= 0 ? (up < 64 ? hi << up : 0ull) : (up > -64 ? hi >> -up : 0ull);
    if (bits >> 63) fix = 0ull - fix;
  }
  const unsigned long long turn = fix * (unsigned long long)(long long)position;
  const unsigned long long q = (turn + (1ull << 61)) >> 62;  // nearest quarter
  const long long rest = (long long)(turn - (q << 62));      // within an eighth of a turn
  float s, c;
  sincospif((float)rest * 0x1p-63f, &s, &c);                 // 2 * rest / 2^64 half-turns
  if (q & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (q & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c, s);
}

// x / s correctly rounded in all but rare cases: a multiplication by 1 / s
// and one correction of the remainder.
__device__ __forceinline__ float divide(float x, float s, float inv) {
  const float y = x * inv;
  return fmaf(fmaf(-y, s, x), inv, y);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// A CTA takes TB tokens (blockIdx.x) and every gridDim.y-th item (a head of q,
// k or v) of them; D / 8 lanes work on one head, eight values each.
template <class T, bool E4M3, int D, int TB>
__global__ void __launch_bounds__(kNT) rope_kernel(const RopeParams P) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kNT / kLanes / TB;  // heads of one token at a time
  constexpr int kAhead = 2;                   // heads whose loads are in flight together
  __shared__ float2 turns[TB][D / 2];
  const int tid = threadIdx.x, lane = tid % kLanes, group = tid / kLanes;
  const int tl = group % TB, g = group / TB;
  const int t0 = blockIdx.x * TB;
  const int half = P.rot >> 1;
  for (int i = tid; i < TB * half; i += kNT) {
    const int t = i / half, f = i - t * half;
    if (t0 + t < P.T) {
      const float2 cs = turn_of(P.inv_freq[f], P.positions[t0 + t]);
      turns[t][f] = make_float2(cs.x * P.rope_scale, cs.y * P.rope_scale);
    }
  }
  const int t = t0 + tl;
  const bool live = t < P.T;
  long long place = -1;
  if (live) {
    const int slot = P.slots[t];
    if (slot >= 0 && slot < P.num_slots)
      place = (long long)(slot >> P.page_shift) * P.page_stride + (long long)(slot & ((1 << P.page_shift) - 1)) * P.token_stride;
  }
  __syncthreads();

  // this thread's values: 8 * lane .. 8 * lane + 7; their partners are inside ("interleaved") or in another lane
  const int at = lane * 8;
  const bool turned = at < P.rot;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  if (turned && live) {
    if (P.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 cs = turns[tl][at / 2 + i];
        c[2 * i] = c[2 * i + 1] = cs.x;
        s[2 * i] = -cs.y;
        s[2 * i + 1] = cs.y;
      }
    } else {
      const bool low = at < half;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 cs = turns[tl][(low ? at : at - half) + i];
        c[i] = cs.x;
        s[i] = low ? -cs.y : cs.y;
      }
    }
  }
  // lane that holds this thread's partners ("half" pairs)
  const int apart = P.rot >> 4;
  const int partner = (tid & 31) - lane + (turned ? (at < half ? lane + apart : lane - apart) : lane);

  const int heads = P.hq + 2 * P.hkv;
  const int step = kGroups * gridDim.y;
  const int rounds = (heads + step - 1) / step;
  for (int r0 = 0; r0 < rounds; r0 += kAhead) {
    uint4 raw[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int h = (r0 + a) * step + blockIdx.y * kGroups + g;
      raw[a] = make_uint4(0u, 0u, 0u, 0u);
      if (live && h < heads) {
        const T* src = h < P.hq ? static_cast<const T*>(P.q) + t * P.q_stride + h * D
                       : h < P.hq + P.hkv ? static_cast<const T*>(P.k) + t * P.k_stride + (h - P.hq) * D
                                          : static_cast<const T*>(P.v) + t * P.v_stride + (h - P.hq - P.hkv) * D;
        raw[a] = *reinterpret_cast<const uint4*>(src + at);
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int h = (r0 + a) * step + blockIdx.y * kGroups + g;
      const bool is_q = h < P.hq, is_v = h >= P.hq + P.hkv;
      float x[8];
      unpack(raw[a].x, x[0], x[1], T());
      unpack(raw[a].y, x[2], x[3], T());
      unpack(raw[a].z, x[4], x[5], T());
      unpack(raw[a].w, x[6], x[7], T());
      const void* weight = is_q ? P.qw : P.kw;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (weight != nullptr && !is_v) {
        const float r = 1.0f / sqrtf(sum * (1.0f / D) + P.eps);
        const uint4 wr = *reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + at);
        float w[8];
        unpack(wr.x, w[0], w[1], T());
        unpack(wr.y, w[2], w[3], T());
        unpack(wr.z, w[4], w[5], T());
        unpack(wr.w, w[6], w[7], T());
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
      }
      float y[8];
      if (P.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i ^ 1], s[i], x[i] * c[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(__shfl_sync(0xffffffffu, x[i], partner), s[i], x[i] * c[i]);
      }
      if (!turned || is_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
      }
      if (!live || h >= heads) continue;
      if (is_q) {
        uint4 o;
        o.x = pack2(y[0], y[1], T());
        o.y = pack2(y[2], y[3], T());
        o.z = pack2(y[4], y[5], T());
        o.w = pack2(y[6], y[7], T());
        *reinterpret_cast<uint4*>(static_cast<T*>(P.q_out) + t * P.qo_stride + h * D + at) = o;
      } else if (place >= 0) {
        const int kh = is_v ? h - P.hq - P.hkv : h - P.hq;
        const long long off = place + kh * P.head_stride + at;
        void* cache = is_v ? P.v_cache : P.k_cache;
        if (E4M3) {
          const float* scales = is_v ? P.v_scale : P.k_scale;
          if (scales != nullptr) {
            const float sc = scales[kh], inv = 1.0f / sc;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = divide(y[i], sc, inv);
          }
          *reinterpret_cast<uint2*>(static_cast<unsigned char*>(cache) + off) =
              make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
        } else {
          uint4 o;
          o.x = is_v ? raw[a].x : pack2(y[0], y[1], T());
          o.y = is_v ? raw[a].y : pack2(y[2], y[3], T());
          o.z = is_v ? raw[a].z : pack2(y[4], y[5], T());
          o.w = is_v ? raw[a].w : pack2(y[6], y[7], T());
          *reinterpret_cast<uint4*>(static_cast<T*>(cache) + off) = o;
        }
      }
    }
  }
}

template <class T, bool E4M3, int D>
cudaError_t launch(const RopeParams& P, int sms, cudaStream_t st) {
  constexpr int kTokens = 4;
  const int heads = P.hq + 2 * P.hkv;
  if (P.T >= 4 * sms * kTokens) {
    rope_kernel<T, E4M3, D, kTokens><<<dim3((P.T + kTokens - 1) / kTokens, 1), kNT, 0, st>>>(P);
  } else {
    // few tokens: one a CTA, and its heads over several CTAs until the GPU has about two CTAs an SM
    const int per = kNT / (D / 8);
    const int most = (heads + per - 1) / per;
    const int split = std::min(most, std::max(1, 2 * sms / P.T));
    rope_kernel<T, E4M3, D, 1><<<dim3(P.T, split), kNT, 0, st>>>(P);
  }
  return cudaGetLastError();
}

template <class T, bool E4M3>
cudaError_t by_dim(const RopeParams& P, int d, int sms, cudaStream_t st) {
  return d == 64 ? launch<T, E4M3, 64>(P, sms, st) : d == 128 ? launch<T, E4M3, 128>(P, sms, st) : launch<T, E4M3, 256>(P, sms, st);
}

}  // namespace

cudaError_t kv_rope_launch(const RopeParams& P, bool bf16, bool e4m3, int d, int sms, cudaStream_t st) {
  if (bf16) return e4m3 ? by_dim<__nv_bfloat16, true>(P, d, sms, st) : by_dim<__nv_bfloat16, false>(P, d, sms, st);
  return e4m3 ? by_dim<__half, true>(P, d, sms, st) : by_dim<__half, false>(P, d, sms, st);
}

}  // namespace ss
