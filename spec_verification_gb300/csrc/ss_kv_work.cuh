// How ss_attend's work is cut up: units, their key tiles, and the ranges of
// tiles that the CTAs of its fixed grid take.
//
//  - A unit is (row, key head, tile of `rows` query rows); query row i of a
//    unit is token i / group, head i % group, so the heads that share a key
//    head share its loads.  A unit's keys are tiles of 64 or 128.
//  - The units, in order, form one line in which a unit is as long as its tiles
//    plus unit_cost (what starting and ending one costs, in tiles).  The line
//    is cut into equal parts, one per CTA: the split follows from the lengths
//    on the device, every CTA has the same work whatever the rows' lengths
//    are, and the launch never changes.  Tile i of a unit that starts at u is
//    at u + unit_cost + i and belongs to the CTA whose part that lies in; all
//    tiles of a short unit belong to the CTA that has the first.
#pragma once

#include "ss_kv_common.cuh"

namespace ss {
namespace kv {

// Least length of a part: shorter ones cost more in the join than they save, the more the larger the pieces are.
// Measured (us) with 2, 4, 8, 12: 16 query rows of 128 columns, 700 tokens 12.4, 13.8, 20.5, 20.6; 32 of 256, 2 x 2237
// 25.8, 27.6, 27.9, 34; 128 of 64, 1 x 11550 44, 37, 33, 34; 128 of 256, 13 x 9308 75.5, 75.6, 68, 74.  But not longer
// than a row's units are on average: those want a CTA each (128 query rows, 77 rows of 4 tokens, 308 units of 3: with 8
// 24.6, with 2 18.2).
__device__ __forceinline__ int least_part(const AttendParams& P, uint32_t total) {
  return P.rows == 128 ? (int)min(8u, max(2u, total / (uint32_t)(P.B * P.hkv))) : 2;
}

// Tiles of a unit that is not worth cutting: the join of its pieces would take longer.  Measured (us) with none, 2 and 4
// of 64 keys and 128 columns: 256 x 1 rows of at most 200 tokens 48.3, 47.6, 44.4; 213 x 8, window 68, 45.5, 45.9, 43.9; 64
// columns, 256 x 1, with none, 4, 8: 21.8, 20.5, 20.5.  128 keys, with none, 3, 6: one row of 300 13, 12.3, 12.2, but
// 4 x 1 rows of at most 3000 17, 17, 19.3.
__device__ __forceinline__ int longest_uncut(const AttendParams& P) {
  return P.tile_shift == 6 ? min(2 * P.unit_cost, 4) : P.unit_cost;
}

struct Row {
  int q0, n, len;
  uint32_t status;
};

__device__ __forceinline__ Row row_info(const AttendParams& P, int r) {
  Row w;
  w.q0 = P.cu_new[r];
  const int q1 = P.cu_new[r + 1];
  w.n = q1 - w.q0;
  w.len = P.seq_len[r];
  w.status = 0;
  if (w.q0 < 0 || q1 < w.q0 || q1 > P.max_tokens) {
    w.n = 0;
    w.status = SS_ST_CAPACITY;
  }
  if (w.len < 0 || w.len > P.max_blocks << P.page_shift) {
    w.len = 0;
    w.status |= SS_ST_BAD_PARAM;
  }
  return w;
}

// Token of query row x of a row of requests: x / group.
__device__ __forceinline__ int token_of(const AttendParams& P, int x) {
  return (int)((__umulhi((uint32_t)x, P.group_mul) + (uint32_t)x) >> P.group_shift);
}

// Key tiles of a unit: `sink` tiles from 0, then from `first` on.
struct Unit {
  int pos0, pos1;  // positions of its first and last token (may be negative)
  int sink, first, tiles;
};

__device__ __forceinline__ Unit unit_info(const AttendParams& P, const Row& w, int mt) {
  Unit u;
  const int j0 = token_of(P, mt * P.rows);
  const int j1 = min(w.n - 1, token_of(P, mt * P.rows + P.rows - 1));
  u.pos0 = w.len - w.n + j0;
  u.pos1 = w.len - w.n + j1;
  u.sink = 0;
  u.first = 0;
  if (P.window > 0) {
    u.first = max(0, max(0, u.pos0) - P.window + 1) >> P.tile_shift;
    u.sink = min(((P.sinks - 1) >> P.tile_shift) + 1, u.first);  // (no sum that could pass 2^31)
  }
  // a unit without a visible key still has one (masked) tile: its output is written
  u.tiles = u.pos1 < 0 ? 1 : u.sink + (u.pos1 >> P.tile_shift) - u.first + 1;
  return u;
}
__device__ __forceinline__ int tile_of(const Unit& u, int i) { return i < u.sink ? i : i - u.sink + u.first; }

__device__ __forceinline__ int row_units(const AttendParams& P, const Row& w) {  // of one key head
  return (w.n * P.group + P.rows - 1) >> (31 - __clz(P.rows));
}
__device__ __forceinline__ long long row_length(const AttendParams& P, const Row& w) {  // of one key head, on the line
  long long s = 0;
  for (int m = 0; m < row_units(P, w); ++m) s += unit_info(P, w, m).tiles + P.unit_cost;
  return s;
}

// The line cut into `ctas` parts: the first `longer` of them are base + 1 long, the others base.
struct Cut {
  long long base;
  int longer, ctas;
  __device__ __forceinline__ long long start(int c) const { return base * c + min(c, longer); }
  // the part that place t lies in
  __device__ __forceinline__ int owner(long long t) const {
    const long long edge = (base + 1) * longer;
    const bool first = t < edge;
    const long long x = first ? t : t - edge, d = first ? base + 1 : base;
    const int q = (x | d) >> 31 ? (int)(x / d) : (int)((uint32_t)x / (uint32_t)d);  // 32-bit divisions where they do
    return first ? q : longer + q;
  }
};

// A CTA's part of the line and where it starts: `skip` tiles into unit (row, h, mt), which starts at `unit`.
struct Range {
  Cut cut;
  long long unit, end;
  int row, h, mt, skip;
  Row w;  // of `row`
};

// A CTA's part of one unit.
struct Segment {
  Unit u;
  int row, h, mt, q0, n, len;
  int from, count;  // tiles [from, from + count) of the unit
  int live;         // query rows
  int ca, cb;       // first and last CTA that have tiles of the unit
};

// The next segment of the range; false at its end.
__device__ __forceinline__ bool next_segment(const AttendParams& P, Range& k, Segment& g) {
  while (k.unit < k.end) {
    while (k.mt >= row_units(P, k.w)) {  // next key head, next row with work (the line ends before the rows do)
      k.mt = 0;
      if (k.w.n == 0 || ++k.h == P.hkv) {
        k.h = 0;
        k.w = row_info(P, ++k.row);
      }
    }
    const Row& w = k.w;
    g.u = unit_info(P, w, k.mt);
    const bool uncut = g.u.tiles <= longest_uncut(P);
    const long long at = k.unit + P.unit_cost;  // of tile 0
    g.row = k.row;
    g.h = k.h;
    g.mt = k.mt;
    g.q0 = w.q0;
    g.n = w.n;
    g.len = w.len;
    g.from = k.skip;
    g.count = uncut ? (at < k.end ? g.u.tiles : 0) : (int)min((long long)g.u.tiles, k.end - at) - g.from;
    if (g.count <= 0) return false;  // the part ends inside the unit's start
    g.live = min(P.rows, w.n * P.group - k.mt * P.rows);
    g.ca = g.from != 0 ? k.cut.owner(at) : (int)blockIdx.x;
    g.cb = g.from + g.count != g.u.tiles ? k.cut.owner(at + g.u.tiles - 1) : (int)blockIdx.x;
    const bool ours = !uncut || k.skip == 0;
    k.unit = at + g.u.tiles;
    k.skip = 0;
    ++k.mt;
    if (ours) return true;
  }
  return false;
}

// This CTA's range, by all NT threads of the block: every thread sums a run of rows, but for those of warp kBusy, which
// come later than the others.  `sums` holds NT / 32 values,
// `out` gets the range; row status bits of bad rows are set.  cut.ctas == 0: nothing for this CTA.
template <int NT, int kBusy>
__device__ __forceinline__ void find_range(const AttendParams& P, long long* sums, Range* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (P.B + NT - 33) / (NT - 32), nth = warp > kBusy ? tid - 32 : tid;
  const int ra = min(P.B, nth * run), rb = warp == kBusy ? ra : min(P.B, ra + run);
  long long mine = 0, per_head = 0;  // per_head, w: of the first row, mostly the only one
  Row w = {0, 0, 0, 0};
  for (int r = rb - 1; r >= ra; --r) {
    w = row_info(P, r);
    if (w.status && blockIdx.x == 0) atomicOr(&P.row_status[r], w.status);
    per_head = row_length(P, w);
    mine += per_head * P.hkv;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  if (tid == 0) out->cut.ctas = 0;
  __syncthreads();
  long long total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const long long y = sums[w];
    if (w < warp) before += y;
    total += y;
  }
  Cut cut;
  const bool small = total < (1ll << 31);
  const int least = least_part(P, (uint32_t)total);  // (of no use to long lines)
  cut.ctas = (int)min((long long)gridDim.x, small ? (long long)(((uint32_t)total + least - 1) / least) : total);
  cut.base = cut.ctas == 0 ? 0 : small ? (long long)((uint32_t)total / (uint32_t)cut.ctas) : total / cut.ctas;
  cut.longer = (int)(total - cut.base * cut.ctas);
  const long long start = cut.start(blockIdx.x);
  if ((int)blockIdx.x < cut.ctas && start >= before && start < before + mine) {
    long long off = start - before;
    Range k;
    k.cut = cut;
    k.end = cut.start(blockIdx.x + 1);
    for (k.row = ra; off >= per_head * P.hkv;) {
      off -= per_head * P.hkv;
      w = row_info(P, ++k.row);
      per_head = row_length(P, w);
    }
    k.w = w;
    k.h = small ? (int)((uint32_t)off / (uint32_t)per_head) : (int)(off / per_head);
    off -= k.h * per_head;
    k.mt = 0;
    for (int n = unit_info(P, w, 0).tiles + P.unit_cost; off >= n; n = unit_info(P, w, k.mt).tiles + P.unit_cost) {
      off -= n;
      ++k.mt;
    }
    k.unit = start - off;
    k.skip = max(0, (int)off - P.unit_cost);
    *out = k;
  }
  __syncthreads();
}

}  // namespace kv
}  // namespace ss
