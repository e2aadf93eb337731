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
#include <type_traits>

#include "ss_kv_common.cuh"

namespace ss {
namespace {

constexpr int kNT = 128;

template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 of(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
  static __device__ __forceinline__ uint32_t to(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 of(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ uint32_t to(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// (cos, sin) of position * f radians.  f = m64 * 2^(e - 63) with m64 its
// mantissa at the top of 64 bits; f / (2 pi) * 2^64 = (m64 * K >> 64) * 2^(e + 1),
// K = 2^64 / (2 pi).
__device__ __forceinline__ float2 turn_of(double f, int position) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const int be = (int)(bits >> 52) & 0x7ff;
  if (be == 0x7ff) return make_float2(NAN, NAN);  // infinite or NaN: so are the angles
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
// and one correction of the remainder; infinities stay what they are.
__device__ __forceinline__ float divide(float x, float s, float inv) {
  const float y = x * inv;
  return fabsf(y) < INFINITY ? fmaf(fmaf(-y, s, x), inv, y) : y;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// Four values of a query or key.  Not __ldg: queries may be overwritten in place, and a read-only load is for what the
// kernel does not write.  (By way of L2, as each is read once: with plain loads the compiler holds eight registers more over
// the angles and spills, 16384 tokens 67.6 us where these take 64.7.)
__device__ __forceinline__ uint2 load_pairs(const void* p) { return __ldcg(static_cast<const uint2*>(p)); }

// Eight values of a head that one thread holds: four pairs (a, b).
struct Eight {
  float a[4], b[4];
};
// Where they are in the head: values at, at + 1, .. at + 3 and then, .., then + 3.  "half" pairs: the first four are
// a, the others b.  Otherwise (interleaved pairs, values past the rotated ones) then = at + 4, and neighbours pair.
template <class T>
__device__ __forceinline__ Eight spread(const uint2 lo, const uint2 hi, bool halves) {
  const float2 p = Pair<T>::of(lo.x), q = Pair<T>::of(lo.y), r = Pair<T>::of(hi.x), s = Pair<T>::of(hi.y);
  return halves ? Eight{{p.x, p.y, q.x, q.y}, {r.x, r.y, s.x, s.y}} : Eight{{p.x, q.x, r.x, s.x}, {p.y, q.y, r.y, s.y}};
}
__device__ __forceinline__ void gathered(const Eight& e, bool halves, float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[halves ? i : 2 * i] = e.a[i];
    y[halves ? 4 + i : 2 * i + 1] = e.b[i];
  }
}

// A CTA takes TB tokens (blockIdx.x) and every gridDim.y-th group of their heads; D / 8 lanes work on one head.  A
// thread holds both values of each of its pairs, so no lane needs another's; cos and sin of its four pairs are in
// registers, multiplied with the norm's weights, and a head costs two 8-byte loads, its sum of squares over the
// lanes, 24 multiplications and additions, and two stores.  Ten CTAs of 128 threads an SM keep enough loads in flight
// (eight: 71 us where ten take 65): 16384 tokens of 48 heads of 128, with norms, 64.7 us, 6.2 TB/s.  That was measured on
// this form; the 48 registers spill 32 bytes a thread with 8 bits (6000 tokens of 56 heads 32.8 us, 4.9 TB/s) and 64 with
// "half" pairs on part of the head (6000 of 48 heads, a quarter turned, 39 us, 3.8 TB/s).
// `Order` says what is known of the pairs at compile time: kNeighbours in every lane, kHalves in every lane (all of
// the head is rotated), or kMixed ("half" pairs in the first lanes).
enum Order { kNeighbours, kHalves, kMixed };
template <class T, bool E4M3, int D, int TB, Order kOrder>
__global__ void __launch_bounds__(kNT, 10) rope_kernel(const RopeParams P) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kNT / kLanes / TB;  // heads of one token at a time
  constexpr int kAhead = TB > 1 ? 2 : 1;      // heads to a batch; the next batch's loads are in flight over a batch
  __shared__ float2 turns[TB][D / 2];
  const int tid = threadIdx.x, lane = tid % kLanes, group = tid / kLanes;
  const int tl = group % TB;
  const int t0 = blockIdx.x * TB, t = min(t0 + tl, P.T - 1);
  const bool live = t0 + tl < P.T;
  const int half = kOrder == kHalves ? D / 2 : P.rot >> 1;
  const bool turned = kOrder == kHalves || lane * 8 < P.rot;
  const bool halves = kOrder == kHalves || (kOrder == kMixed && turned);
  const int at = halves ? lane * 4 : lane * 8, then = halves ? half + lane * 4 : at + 4;
  const int h0 = blockIdx.y * kGroups + group / TB, step = kGroups * gridDim.y;

  // batches of heads: those of q, then those of k, the same number in every lane
  const int nq = (P.hq + step * kAhead - 1) / (step * kAhead), nk = (P.hkv + step * kAhead - 1) / (step * kAhead);
  struct Raw {
    uint2 lo[kAhead], hi[kAhead];
  };
  auto load = [&](int b, Raw& r) {
    const bool is_q = b < nq;
    const T* src = is_q ? static_cast<const T*>(P.q) + t * P.q_stride : static_cast<const T*>(P.k) + t * P.k_stride;
    const int first = h0 + (is_q ? b : b - nq) * step * kAhead, last = (is_q ? P.hq : P.hkv) - 1;
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const T* p = src + min(first + n * step, last) * D;
      r.lo[n] = load_pairs(p + at);
      r.hi[n] = load_pairs(p + then);
    }
  };
  Raw raw;
  load(0, raw);

  for (int i = tid; i < TB * half; i += kNT) {
    const int n = i / half, f = i - n * half;
    if (t0 + n < P.T) {
      const float2 cs = turn_of(P.inv_freq[f], P.positions[t0 + n]);
      turns[n][f] = make_float2(cs.x * P.rope_scale, cs.y * P.rope_scale);
    }
  }
  const int slot = live ? P.slots[t] : -1;
  const long long place = (long long)(slot >> P.page_shift) * P.page_stride + (long long)(slot & ((1 << P.page_shift) - 1)) * P.token_stride;
  const bool stored = slot >= 0 && slot < P.num_slots;
  __syncthreads();

  // batches [b0, b1), the heads of one of q and k: norm, rotation, then `put`
  auto rotate = [&](int b0, int b1, int heads, const void* weight, auto put) {
    Eight w = {{1.0f, 1.0f, 1.0f, 1.0f}, {1.0f, 1.0f, 1.0f, 1.0f}};
    if (weight != nullptr) {
      const T* p = static_cast<const T*>(weight);
      w = spread<T>(*reinterpret_cast<const uint2*>(p + at), *reinterpret_cast<const uint2*>(p + then), halves);
    }
    Eight cw, sw;  // a -> a cw.a - b sw.b, b -> b cw.b + a sw.a
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 cs = turned ? turns[tl][lane * 4 + i] : make_float2(1.0f, 0.0f);
      cw.a[i] = cs.x * w.a[i];
      cw.b[i] = cs.x * w.b[i];
      sw.a[i] = cs.y * w.a[i];
      sw.b[i] = cs.y * w.b[i];
    }
    for (int b = b0; b < b1; ++b) {
      const Raw now = raw;
      if (b + 1 < nq + nk) load(b + 1, raw);
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        const int h = h0 + ((b - b0) * kAhead + n) * step;
        Eight x = spread<T>(now.lo[n], now.hi[n], halves);
        float r = 1.0f;
        if (weight != nullptr) {
          float sum = 0.0f, eps = P.eps;
          auto squares = [&]() {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = fmaf(x.a[i], x.a[i], fmaf(x.b[i], x.b[i], sum));
          };
          squares();
          if (std::is_same<T, __nv_bfloat16>::value) {
            // bf16 values whose squares come near the ends of 32 bits, or pass them: once more with the head scaled by a
            // power of two, which the norm takes out.  (Asked before the sum over the lanes, beside which the vote costs
            // least: 1 us of 65 with 16384 tokens.  Leaving such heads out for a second pass costs 1.5.)
            const bool tiny = P.eps < 0x1p-100f;  // nothing else keeps the root from the small end
            if (__any_sync(0xffffffffu, sum > 0x1p100f || (tiny && sum < 0x1p-100f))) {
#pragma unroll
              for (int d = kLanes / 2; d > 0; d >>= 1) sum = fmaxf(sum, __shfl_xor_sync(0xffffffffu, sum, d));
              const float f = sum > 0x1p100f ? 0x1p-70f : tiny && sum < 0x1p-100f ? 0x1p70f : 1.0f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x.a[i] *= f;
                x.b[i] *= f;
              }
              eps = eps * f * f;
              squares();
            }
          }
#pragma unroll
          for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          const float m = fmaf(sum, 1.0f / D, eps);
          r = rsqrtf(m);
          // a Newton step: to about a rounding (an infinite value leaves 0 of the others, as in the formula)
          if (m < INFINITY) r = fmaf(r * fmaf(-m * r, r, 1.0f), 0.5f, r);
        }
        Eight y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y.a[i] = fmaf(x.a[i], cw.a[i], -x.b[i] * sw.b[i]) * r;
          y.b[i] = fmaf(x.b[i], cw.b[i], x.a[i] * sw.a[i]) * r;
        }
        if (!turned) {  // nothing of a neighbour may reach these (sw is 0, but 0 * infinity is not)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y.a[i] = x.a[i] * cw.a[i] * r;
            y.b[i] = x.b[i] * cw.b[i] * r;
          }
        }
        if (h < heads) put(h, y);
      }
    }
  };
  auto pack = [&](const float (&y)[8], uint2& lo, uint2& hi) {
    lo = make_uint2(Pair<T>::to(y[0], y[1]), Pair<T>::to(y[2], y[3]));
    hi = make_uint2(Pair<T>::to(y[4], y[5]), Pair<T>::to(y[6], y[7]));
  };
  // y[0..3] at `at`, y[4..7] at `then` of a head of the cache, divided by the head's factor
  auto hold = [&](void* cache, const float* scales, int h, float (&y)[8]) {
    const long long off = place + h * P.head_stride;
    if (E4M3) {
      if (scales != nullptr) {
        const float sc = scales[h], inv = 1.0f / sc;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = divide(y[i], sc, inv);
      }
      unsigned char* p = static_cast<unsigned char*>(cache) + off;
      *reinterpret_cast<uint32_t*>(p + at) = e4m3x4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint32_t*>(p + then) = e4m3x4(y[4], y[5], y[6], y[7]);
    } else {
      T* p = static_cast<T*>(cache) + off;
      uint2 lo, hi;
      pack(y, lo, hi);
      *reinterpret_cast<uint2*>(p + at) = lo;
      *reinterpret_cast<uint2*>(p + then) = hi;
    }
  };

  rotate(0, nq, P.hq, P.qw, [&](int h, const Eight& e) {
    if (!live) return;
    float y[8];
    gathered(e, halves, y);
    uint2 lo, hi;
    pack(y, lo, hi);
    T* p = static_cast<T*>(P.q_out) + t * P.qo_stride + h * D;
    *reinterpret_cast<uint2*>(p + at) = lo;
    *reinterpret_cast<uint2*>(p + then) = hi;
  });
  rotate(nq, nq + nk, P.hkv, P.kw, [&](int h, const Eight& e) {
    if (!stored) return;
    float y[8];
    gathered(e, halves, y);
    hold(P.k_cache, P.k_scale, h, y);
  });
  if (!stored) return;
  const T* v = static_cast<const T*>(P.v) + t * P.v_stride + lane * 8;
  for (int h = h0; h < P.hkv; h += step) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(v + h * D));
    const long long off = place + h * P.head_stride + lane * 8;
    if (E4M3) {
      const float sc = P.v_scale ? P.v_scale[h] : 1.0f, inv = 1.0f / sc;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = Pair<T>::of(w[i]);
        y[2 * i] = divide(f.x, sc, inv);
        y[2 * i + 1] = divide(f.y, sc, inv);
      }
      *reinterpret_cast<uint2*>(static_cast<unsigned char*>(P.v_cache) + off) =
          make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
    } else {
      *reinterpret_cast<uint4*>(static_cast<T*>(P.v_cache) + off) = x;
    }
  }
}

template <class T, bool E4M3, int D, Order kOrder>
cudaError_t launch(const RopeParams& P, int sms, cudaStream_t st) {
  // Tokens of a CTA: the more, the fewer CTAs compute angles and the longer each streams; but enough CTAs to fill the
  // GPU.  Measured (us, 2 / 4 tokens): 16384 tokens of 48 heads of 128 67.8 / 64.8, 1531 tokens of 80 heads of 64 8.4 / 11.1.
  const int heads = std::max(P.hq, P.hkv);
  if (P.T >= 16 * sms) {
    rope_kernel<T, E4M3, D, 4, kOrder><<<dim3((P.T + 3) / 4, 1), kNT, 0, st>>>(P);
  } else if (P.T >= 2 * sms) {
    rope_kernel<T, E4M3, D, 2, kOrder><<<dim3((P.T + 1) / 2, 1), kNT, 0, st>>>(P);
  } else {
    // one token a CTA, and its heads over several CTAs until the GPU has about two CTAs an SM
    const int per = kNT / (D / 8);
    const int most = (heads + per - 1) / per;
    const int split = std::min(most, std::max(1, 2 * sms / P.T));
    rope_kernel<T, E4M3, D, 1, kOrder><<<dim3(P.T, split), kNT, 0, st>>>(P);
  }
  return cudaGetLastError();
}

template <class T, bool E4M3, int D>
cudaError_t by_order(const RopeParams& P, int sms, cudaStream_t st) {
  if (P.interleaved || P.rot == 0) return launch<T, E4M3, D, kNeighbours>(P, sms, st);
  return P.rot == D ? launch<T, E4M3, D, kHalves>(P, sms, st) : launch<T, E4M3, D, kMixed>(P, sms, st);
}

template <class T, bool E4M3>
cudaError_t by_dim(const RopeParams& P, int d, int sms, cudaStream_t st) {
  return d == 64 ? by_order<T, E4M3, 64>(P, sms, st) : d == 128 ? by_order<T, E4M3, 128>(P, sms, st) : by_order<T, E4M3, 256>(P, sms, st);
}

}  // namespace

cudaError_t kv_rope_launch(const RopeParams& P, bool bf16, bool e4m3, int d, int sms, cudaStream_t st) {
  if (bf16) return e4m3 ? by_dim<__nv_bfloat16, true>(P, d, sms, st) : by_dim<__nv_bfloat16, false>(P, d, sms, st);
  return e4m3 ? by_dim<__half, true>(P, d, sms, st) : by_dim<__half, false>(P, d, sms, st);
}

}  // namespace ss
