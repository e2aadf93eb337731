// How the pieces of a unit that lies in several CTAs become its output.
//
// Every CTA that has tiles of the unit writes its piece, (m, l) and O of each
// query row, to the workspace and counts itself in; the last of a group of
// neighbouring CTAs to do so joins their pieces, and the last of the groups
// joins what the groups left.  Nobody waits.  Which pieces meet is fixed by the
// split, and they are added in its order, so the result does not depend on who
// comes last.  Two levels because a unit of one long row may lie in every CTA:
// a single CTA would read all pieces alone (75 pieces of 128 rows of 64
// columns: 174 us for a call whose loads take 3).
#pragma once

#include "ss_kv_work.cuh"

namespace ss {
namespace kv {

// Pieces of a group, of n: as many as there are groups, so that the fewest are read one after the other; one group where
// that costs less than meeting twice.  Measured (us, groups of 8 / of about sqrt n): 16 query rows of 128 columns, 6
// pieces 12.4 / 13.7, about 10 75.4 / 73.5; 64 of 128, 8 pieces 57.5 / 52.4; 64 columns, 13 rows of 128 69.3 / 65.4.
__device__ __forceinline__ int group_of(int n, bool large) { return n <= (large ? 3 : 8) ? n : (int)ceilf(sqrtf((float)n)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A CTA has at most two pieces: of the unit that its range ends in (which starts in it), and of the one it begins in.
__device__ __forceinline__ int piece_of(const Segment& g, int x) { return 2 * x + (x == g.ca ? 1 : 0); }
// Piece p: of row r, (m, the sum that O is divided by, the sum of the weights); four columns of row r, from column 4 * c
// on, are at (c * rows + r).
__device__ __forceinline__ float4* piece_ml(const AttendParams& P, int p) { return P.ml + (size_t)p * P.rows; }
template <int D>
__device__ __forceinline__ float4* piece_out(const AttendParams& P, int p) {
  return reinterpret_cast<float4*>(P.part + (size_t)p * P.rows * D);
}

// Joins the pieces of CTAs first, first + step, ... (count of them) into that of `first`, or the output.  All NT
// threads; four columns of a row are an item, and a thread's items are all of one row (rows divides NT).
template <class T, class Pack, int D, int NT, class Bar>
__device__ __forceinline__ void add_pieces(const AttendParams& P, const Segment& g, int first, int step, int count, bool to_out, Bar bar) {
  constexpr int kPieces = 4, kItems = 4;  // loads in flight together
  const int tid = threadIdx.x, m = tid & (P.rows - 1), items = P.rows * (D / 4);
  const bool live = m < g.live;
  const int f = g.mt * P.rows + m, token = token_of(P, f), head = g.h * P.group + f - token * P.group;
  T* to = static_cast<T*>(P.out) + (g.q0 + token) * P.out_stride + head * D;
  float top = -INFINITY, sum = 0.0f, weights = 0.0f;
  if (live) {
    for (int e0 = tid; e0 < items; e0 += NT * kItems) {
      top = -INFINITY;
      sum = weights = 0.0f;
      float4 o[kItems];
#pragma unroll
      for (int n = 0; n < kItems; ++n) o[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int x0 = 0; x0 < count; x0 += kPieces) {
        float4 ml[kPieces];
        float4 y[kPieces][kItems];
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
          const int its = piece_of(g, first + min(x0 + x, count - 1) * step);
          ml[x] = __ldcg(piece_ml(P, its) + m);
#pragma unroll
          for (int n = 0; n < kItems; ++n) y[x][n] = __ldcg(piece_out<D>(P, its) + min(e0 + NT * n, items - P.rows + m));
        }
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
          if (x0 + x >= count) break;
          const float n = fmaxf(top, ml[x].x), zn = n == -INFINITY ? 0.0f : n, a = ex2(top - zn), b = ex2(ml[x].x - zn);
          sum = sum * a + ml[x].y * b;
          weights = weights * a + ml[x].z * b;
          top = n;
#pragma unroll
          for (int q = 0; q < kItems; ++q)
            o[q] = make_float4(o[q].x * a + y[x][q].x * b, o[q].y * a + y[x][q].y * b, o[q].z * a + y[x][q].z * b, o[q].w * a + y[x][q].w * b);
        }
      }
      const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int n = 0; n < kItems; ++n) {
        const int e = e0 + NT * n;
        if (e >= items) break;
        if (to_out)
          *reinterpret_cast<uint2*>(to + e / P.rows * 4) =
              make_uint2(Pack::pack(o[n].x * r, o[n].y * r), Pack::pack(o[n].z * r, o[n].w * r));
        else
          piece_out<D>(P, piece_of(g, first))[e] = o[n];
      }
    }
  }
  if (!to_out) bar();  // everyone has read the (m, l) of `first`
  if (live && tid < P.rows) {
    if (!to_out)
      piece_ml(P, piece_of(g, first))[m] = make_float4(top, sum, weights, 0.0f);
    else if (P.lse)
      P.lse[(size_t)(g.q0 + token) * (P.group * P.hkv) + head] = weights == 0.0f ? -INFINITY : (top + log2f(weights)) * 0.69314718055994531f;
  }
}

// After this CTA's piece of the unit is written, by the NT threads that wrote it.  `flag`: a shared word of theirs;
// `bar`: brings them together.  The output's factors (8-bit values) must be in the pieces already.
template <class T, class Pack, int D, int NT, class Bar>
__device__ __forceinline__ void join_unit(const AttendParams& P, const Segment& g, int* flag, Bar bar) {
  const int cta = blockIdx.x, size = group_of(g.cb - g.ca + 1, P.rows * D > 32 * 128), first = g.ca + (cta - g.ca) / size * size;
  const int members = min(size, g.cb - first + 1), groups = (g.cb - g.ca) / size + 1;
  // Counts in; true for the last of `of`, which leaves the counter at zero.  One thread's fences stand for all: the
  // barrier orders the others' writes before them, and their reads (from L2) after.
  auto last = [&](uint32_t* counter, int of) {
    bar();
    if (threadIdx.x == 0) {
      __threadfence();
      *flag = atomicAdd(counter, 1u) + 1 == (uint32_t)of;
      if (*flag) *counter = 0;
      __threadfence();
    }
    bar();
    return *flag != 0;
  };
  if (!last(P.counters + piece_of(g, first), members)) return;
  if (groups > 1) {
    add_pieces<T, Pack, D, NT>(P, g, first, 1, members, false, bar);
    if (!last(P.counters + 2 * gridDim.x + g.ca, groups)) return;
  }
  add_pieces<T, Pack, D, NT>(P, g, g.ca, groups > 1 ? size : 1, groups > 1 ? groups : members, true, bar);
}

}  // namespace kv
}  // namespace ss
