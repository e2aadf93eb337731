// ss_attend for 8-bit caches (e4m3) and at most 16 query rows to a unit.  The
// mathematics, the split of the work and the join of its pieces are those of
// ss_kv_attend.cuh.
//
// What differs: the tensor cores multiply 8-bit keys only with 8-bit queries,
// and splitting 16-bit queries and weights into several 8-bit terms costs two
// to three products for every one (above the time of the loads, whose bytes
// are halved).  Where few query rows share a key, its conversion to f16 (exact)
// is best done in registers, on the way from shared memory to 16 x 8 x 16
// warp-wide products: converting into shared memory writes and reads every key
// twice more there, which costs more than these products do.  Their operand
// layout makes it cheap: the bytes of a key may be taken in any order of
// columns as long as the queries are taken in the same one, and a register of
// transposed values holds two neighbouring columns of two keys, which one byte
// permutation each sorts into an even and an odd column.
//
// One warp runs the ring of TMA copies and publishes the CTA's segments, four
// compute.  Each has all query rows and a quarter of a tile's 128 keys, with
// its own maximum and sum, so that nothing synchronises them inside a unit; at
// its end all leave their pieces in shared memory and each adds a quarter of
// the columns, while the next segment's queries are on their way (256 rows of
// at most 1000 tokens: 106 us with a join by halves and queries read after it,
// 94 so).
// Measured: 32 rows x 4 tokens x 4 query heads over up to 32000 tokens 158 us,
// 4.7 TB/s; what bounds it is the latency of its chains (two warps to a
// scheduler, 40 % of issue slots, 24 % of the tensor pipe).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

#include "ss_kv_attend.cuh"
#include "ss_stage1.cuh"

namespace ss {
namespace kv8 {

using namespace kv;

constexpr int kTile = 128;        // keys of a tile
constexpr int kRows = 16;         // query rows of a unit
constexpr int kWarps = 4;         // computing warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr uint32_t kDrainPolls = 1u << 22;
constexpr int kMaxSlots = 16;     // tiles of keys or values in the ring
constexpr int kControl = 2048;    // bytes of the control block, at most

// ------------------------------------------------------------------ instructions
template <class T>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Pack<__half> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
__device__ __forceinline__ float2 bf16_pair(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
// both f16 halves with NaN (e4m3 has no infinities) replaced by 0
__device__ __forceinline__ uint32_t finite(uint32_t w) {
  if ((w & 0x7c00u) == 0x7c00u) w &= 0xffff0000u;
  if ((w & 0x7c000000u) == 0x7c000000u) w &= 0xffffu;
  return w;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two e4m3 values (the low 16 bits of w) as f16x2: exact.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t w) {
  uint32_t d;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ void arrive(unsigned long long* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(m)) : "memory");
}
template <int N>
__device__ __forceinline__ void bar_warps() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * N) : "memory");
}

// Brings the computing warps together; true for all if it is for any.
__device__ __forceinline__ bool any_warp(bool x) {
  uint32_t y;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(y)
               : "r"((uint32_t)x), "n"(32 * kWarps)
               : "memory");
  return y != 0;
}

// ------------------------------------------------------------------ shape of one instantiation
// (BLOCKS: a factor for each block of tokens.)
template <class T, int D, bool BLOCKS>
struct Shape {
  static constexpr bool kBlocks = BLOCKS;
  static constexpr int kFactors = BLOCKS ? 2048 : 0;         // bytes for factors
  static constexpr bool kScaleQ = std::is_same<T, __nv_bfloat16>::value;
  static_assert(D <= 128, "a head is one swizzled run");
  static constexpr int kSlot = kTile * D;                    // bytes of a key (or value) tile
  static constexpr int kCtas = 2;                            // CTAs per SM
  static constexpr int kSmem = (228 * 1024 / kCtas - 1024) & ~127;  // an SM's share of shared memory
  static constexpr int kKeys = kTile / kWarps;               // keys of a warp
  static constexpr int kKG = kKeys / 16;                     // their 16-key groups
  static constexpr int kQRow = D * 2 + 16;                   // padded: rows fall into different banks
  // ring of tiles: as many as the room beside the queries and the control block holds
  static constexpr int kFit = (kSmem - 1024 - kControl - kFactors - kRows * kQRow) / kSlot;
  static constexpr int kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
};

// ------------------------------------------------------------------ control
struct Control {
  unsigned long long full[kMaxSlots], empty[kMaxSlots];
  unsigned long long seg_full[2], seg_empty[2];  // segment published; done with by all warps
  Segment seg[2];
  int bad[kMaxSlots];   // per tile of keys: its 16-key groups that lie on pages with a bad id
  long long range_sums[kThreads / 32];
  Range range;
  int last;
  float2 ml[kWarps][16];  // of a row, the warps' maximum and sum
  float qinv[kRows];
};

static_assert(sizeof(Control) <= kControl, "control block");

// Factors of a tile's keys, by their place in the ring.
using TileFactors = Factors<kMaxSlots, kTile / 16>;
static_assert(sizeof(TileFactors) <= 2048, "room for factors");

// A place in the ring: tiles of keys and of values take turns.
struct Turn {
  int slot = 0;
  uint32_t parity = 0;
  template <int N>
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
};

template <class S>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)S::kSlots * S::kSlot + (size_t)kRows * S::kQRow + kControl + S::kFactors;
}

// ------------------------------------------------------------------ loads
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, unsigned long long* mbar, int token, int head,
                                         int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(0), "r"(token), "r"(head), "r"(page), "r"(smem_u32(mbar))
      : "memory");
}
__device__ __forceinline__ void expect(unsigned long long* mbar, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(mbar)), "r"(bytes) : "memory");
}

template <class S>
__device__ void load_warp(const AttendParams& P, const CUtensorMap* mk, const CUtensorMap* mv, unsigned char* ring, Control& c,
                          TileFactors* factors, Range k) {
  const int lane = threadIdx.x & 31;
  const int box_shift = min(P.page_shift, 6);            // tokens of one copy
  const int subs_shift = 7 - box_shift;                  // copies of a tile
  const int batch = 32 >> subs_shift;                    // tiles whose page ids one lane each holds
  const int sub = lane & ((1 << subs_shift) - 1), nth = lane >> subs_shift;
  const int page_mask = (1 << P.page_shift) - 1;
  const int groups = (1 << (1 << (box_shift - 4))) - 1;  // 16-key groups of a copy, as bits
  Turn turn;
  int asked = 0;                                         // copies in flight or landed, at most kSlots
  bool dead = false;
  Segment g;
  bool more = true;
  for (int sg = 0; more && !dead; ++sg) {
    more = next_segment(P, k, g);
    if (sg >= 2) dead = !__all_sync(0xffffffffu, mbar_wait(&c.seg_empty[sg & 1], ((sg >> 1) & 1) ^ 1, P.spin_limit, 0u));
    if (dead) break;
    if (!more) g.count = 0;  // the end of the range
    if (lane == 0) {
      c.seg[sg & 1] = g;
      arrive(&c.seg_full[sg & 1]);
    }
    __syncwarp();
    if (!more) break;
    const int32_t* table = P.block_table + (long long)g.row * P.max_blocks;
    const int used = (g.len + page_mask) >> P.page_shift;
    // Whether this lane's copy in the batch from tile i0 on is of tokens that the row holds, and its page: read a batch
    // ahead and looked at only then.  Where nothing is held the copy is from past the cache and reads zeros.
    auto block_of = [&](int i0) { return (tile_of(g.u, g.from + i0 + nth) * kTile + (sub << box_shift)) >> P.page_shift; };
    auto holds = [&](int i0) { return i0 + nth < g.count && block_of(i0) < used; };
    auto fetch = [&](int i0) { return holds(i0) ? __ldg(table + block_of(i0)) : P.num_pages; };
    int next = fetch(0);
    CopyFactors mine;   // of this lane's copy in the batch
    int keys_at = 0;    // place of the tile's keys in the ring
    const int per_copy = 1 << (box_shift - 4);
    auto place_of = [&](int i0) { return (tile_of(g.u, g.from + i0 + nth) * kTile + (sub << box_shift)) & page_mask; };
    for (int i0 = 0; i0 < g.count && !dead; i0 += batch) {
      int id = next;
      next = fetch(i0 + batch);
      const bool is_bad = holds(i0) && (unsigned)id >= (unsigned)P.num_pages;
      const uint32_t bad_lanes = __ballot_sync(0xffffffffu, is_bad);
      if (is_bad) {
        id = P.num_pages;
        atomicOr(&P.row_status[g.row], (uint32_t)SS_ST_KV_PAGE);
      }
      if (S::kBlocks && i0 == 0) mine.fetch(P, holds(0) && !is_bad, id, g.h, place_of(0), per_copy);
      const int n = min(batch, g.count - i0);
      for (int j = 0; j < n && !dead; ++j) {
        const int tok = (tile_of(g.u, g.from + i0 + j) * kTile + (sub << box_shift)) & page_mask;
#pragma unroll 1
        for (int values = 0; values < 2; ++values) {
          dead = !__all_sync(0xffffffffu, mbar_wait(&c.empty[turn.slot], turn.parity ^ 1, P.spin_limit, 0u));
          if (S::kBlocks && dead && values && lane == 0) arrive(&c.full[keys_at]);  // (its copy is waited for at the end)
          if (dead) break;
          if (lane == 0) {
            if (!values) {
              int bits = 0;
              for (int s = 0; s < 1 << subs_shift; ++s)
                if ((bad_lanes >> ((j << subs_shift) + s)) & 1) bits |= groups << (s << (box_shift - 4));
              c.bad[turn.slot] = bits;
            }
            if (S::kBlocks && !values) expect_only(&c.full[turn.slot], S::kSlot);
            else expect(&c.full[turn.slot], S::kSlot);
          }
          __syncwarp();
          if (nth == j)
            tma_load(smem_u32(ring) + turn.slot * S::kSlot + (sub << box_shift) * (S::kSlot / kTile), values ? mv : mk, &c.full[turn.slot], tok, g.h, id);
          if constexpr (S::kBlocks) {
            if (!values) {
              keys_at = turn.slot;
            } else {  // the factors come with the keys, whose barrier waits for them too
              const int tile = keys_at;
              if (nth == j) mine.write(*factors, tile, sub * per_copy, per_copy);
              __syncwarp();
              if (lane == 0) arrive(&c.full[keys_at]);
            }
          }
          turn.next<S::kSlots>();
          asked = min(asked + 1, S::kSlots);
        }
      }
      if (S::kBlocks && i0 + batch < g.count) {  // the next batch's, whose page ids have come meanwhile
        const bool there = holds(i0 + batch) && (unsigned)next < (unsigned)P.num_pages;
        mine.fetch(P, there, next, g.h, place_of(i0 + batch), per_copy);
      }
    }
  }
  // no copy may be in flight when the CTA ends (all have landed unless a wait ran out)
  for (; asked > 0; --asked) {
    if (--turn.slot < 0) {
      turn.slot = S::kSlots - 1;
      turn.parity ^= 1;
    }
    mbar_wait(&c.full[turn.slot], turn.parity, kDrainPolls, 0u);
  }
}

// ------------------------------------------------------------------ products
// Byte offset in a tile of byte b of key `key`: its 16-byte pieces are permuted by the number of its 128-byte line (a
// half line: by its half).
template <int D>
__device__ __forceinline__ uint32_t place_of(int key, int b) {
  const uint32_t off = key * D + b;
  return off ^ ((off >> 3) & (D == 128 ? 0x70 : 0x30));
}

// Weights of a warp's scores where a row's m is large (see kLarge), out of line for the same reason.
template <int N>
struct Scores {
  float s[N][4];
};
template <int N>
static __device__ __noinline__ Scores<N> large_weights(Scores<N> x, float c0, float z0, float c1, float z1) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) x.s[n][e] = ex2(__fsub_rn(__fmul_rn(x.s[n][e], e < 2 ? c0 : c1), e < 2 ? z0 : z1));
  return x;
}

// The same with factors of blocks: a pair of 8-key tiles has one.
template <int N>
struct GroupFactors {
  float k[N], log[N];
};
template <int N>
static __device__ __noinline__ Scores<N> large_weights_blocks(Scores<N> x, GroupFactors<N / 2> f, float c0, float z0, float c1, float z1) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x.s[n][e] = ex2(__fsub_rn(__fadd_rn(__fmul_rn(x.s[n][e], factor_of(e < 2 ? c0 : c1, f.k[n / 2])), f.log[n / 2]), e < 2 ? z0 : z1));
  return x;
}

template <class S, class T, int D>
__device__ void compute_warps(const AttendParams& P, unsigned char* ring, unsigned char* sq, Control& c, const TileFactors* factors) {
  constexpr int kNT = S::kKG * 2;  // 8-key tiles of a warp
  constexpr int kOT = D / 8;       // 8-column tiles of the output
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane & 3, r0 = lane >> 2;
  const uint32_t ring_u = smem_u32(ring), sq_u = smem_u32(sq);
  Turn turn;
  bool dead = false;

  // This lane's ldmatrix rows: byte `b` (a multiple of 32) of its key is at row + (b ^ x).  Keys: the two 16-byte pieces
  // vary fastest over the matrices; values: the keys do.
  const int k_key = ((lane >> 4) << 3) + (lane & 7), v_key = (((lane >> 3) & 1) << 3) + (lane & 7);
  auto permuted = [](int key, int piece) { return (uint32_t)((piece << 4) ^ (D == 128 ? (key & 7) << 4 : ((key >> 1) & 3) << 4)); };
  const uint32_t k_x = permuted(k_key, (lane >> 3) & 1), v_x = permuted(v_key, lane >> 4);
  const int in0 = warp * S::kKeys;  // this warp's keys of a tile

  // A segment's queries are read before the segment ahead of it is joined.
  constexpr int kQ = kRows * (D / 8) / (32 * kWarps);
  uint4 qx[kQ];
  auto fetch = [&](int place, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&c.seg_full[place], parity, P.spin_limit, 0u));
    const Segment& n = c.seg[place];
    if (dead || n.count == 0) return;
#pragma unroll
    for (int x = 0; x < kQ; ++x) {
      const int i = (int)threadIdx.x + 32 * kWarps * x, m = i / (D / 8), piece = i % (D / 8);
      qx[x] = make_uint4(0u, 0u, 0u, 0u);
      if (m < n.live) {
        const int f = n.mt * kRows + m, j = token_of(P, f);
        qx[x] = *reinterpret_cast<const uint4*>(static_cast<const T*>(P.q) + (n.q0 + j) * P.q_stride +
                                                (n.h * P.group + f - j * P.group) * D + piece * 8);
      }
    }
  };
  fetch(0, 0);
  bool more = true;
  for (int sg = 0; more; ++sg) {
    // the segment's fields are read from shared memory where registers are better used otherwise
    const Segment& g = c.seg[sg & 1];
    const int rows_here = dead ? 0 : g.live;

    // queries into shared memory, rows past the end zero (all warps have read the last ones: they met in the join)
#pragma unroll
    for (int n = 0; n < kQ; ++n) {
      const int i = (int)threadIdx.x + 32 * kWarps * n, m = i / (D / 8), piece = i % (D / 8);
      uint4 x = qx[n];
      if (S::kScaleQ) {
        // bf16 to f16: a row is scaled by a power of two that brings its largest value near 2^14, so every
        // value keeps its bits unless it is below 2^-28 of the largest
        const float2 a = bf16_pair(x.x), b = bf16_pair(x.y),
                     d = bf16_pair(x.z), e = bf16_pair(x.w);
        float top = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))),
                          fmaxf(fmaxf(fabsf(d.x), fabsf(d.y)), fmaxf(fabsf(e.x), fabsf(e.y))));
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = max((int)(__float_as_uint(top) >> 23), 15);                // biased exponent
        const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - ex) << 23);  // 2^(14 - exponent)
        if (piece == 0) c.qinv[m] = __uint_as_float((uint32_t)(ex - 14) << 23);
        x = make_uint4(Pack<__half>::pack(a.x * up, a.y * up), Pack<__half>::pack(b.x * up, b.y * up),
                       Pack<__half>::pack(d.x * up, d.y * up), Pack<__half>::pack(e.x * up, e.y * up));
      }
      *reinterpret_cast<uint4*>(sq + m * S::kQRow + piece * 16) = x;
    }
    dead = any_warp(dead);  // all go on, or none: they meet at barriers
    more = !dead && g.count > 0;
    if (!more) break;
    const Unit u = g.u;
    const int count = g.count, from = g.from;

    // a fragment of 16 query rows and 16 columns, the columns in the order in which the keys' bytes come
    auto q_frag = [&](uint32_t (&a)[4], int ks) {
      const unsigned char* p = sq + r0 * S::kQRow + ks * 32 + quad * 8;
      const uint2 x = *reinterpret_cast<const uint2*>(p), y = *reinterpret_cast<const uint2*>(p + 8 * S::kQRow);
      a[0] = x.x;
      a[1] = y.x;
      a[2] = x.y;
      a[3] = y.y;
    };
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) q_frag(qf[ks], ks);
    // positions of this thread's two rows; rows past the end see nothing
    const int m0 = r0, m1 = r0 + 8;
    const int p0 = m0 < rows_here ? g.len - g.n + token_of(P, g.mt * kRows + m0) : -1;
    const int p1 = m1 < rows_here ? g.len - g.n + token_of(P, g.mt * kRows + m1) : -1;
    float c0 = P.scale_log2, c1 = P.scale_log2;
    if (P.k_scale) {
      const float s = P.k_scale[g.h];
      c0 *= s;
      c1 *= s;
    }
    if (S::kScaleQ) {
      c0 *= c.qinv[m0];
      c1 *= c.qinv[m1];
    }
    c0 = fmaxf(c0, FLT_MIN);  // see softmax_warps
    c1 = fmaxf(c1, FLT_MIN);
    if (S::kBlocks) {
      c0 = scale_of(c0);
      c1 = scale_of(c1);
    }

    float o[kOT][4];
#pragma unroll
    for (int i = 0; i < kOT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float mx0 = -INFINITY, mx1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    bool large = false;  // a row of the warp has an m beyond kLarge

    Turn keys, values;
    for (int i = 0; i < count; ++i) {
      keys = values = turn;
      values.next<S::kSlots>();
      turn = values;
      turn.next<S::kSlots>();
      const bool held = i + 1 == count;  // the last tile's room serves the join below
      if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&c.full[keys.slot], keys.parity, P.spin_limit, 0u));
      const int tile = tile_of(u, from + i) * kTile, bad = c.bad[keys.slot];
      // does any live row not see all of the tile?
      const bool part = tile + kTile - 1 > u.pos0 || bad != 0 ||
                        (P.window > 0 && tile <= u.pos1 - P.window && tile > P.sinks - kTile);
      // is key `in` of the tile visible from position p?
      auto sees = [&](int in, int p) {
        const int key = tile + in;
        return key <= p && (P.window <= 0 || key > p - P.window || key < P.sinks) && !((bad >> (in >> 4)) & 1);
      };
      const uint32_t kt = ring_u + keys.slot * S::kSlot + (in0 + k_key) * D;
      const uint32_t vt = ring_u + values.slot * S::kSlot + (in0 + v_key) * D;

      // scores
      float s[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int b0 = 0; b0 < D; b0 += 32) {  // 32 columns of every key
        const int ks = b0 / 16;
#pragma unroll
        for (int gk = 0; gk < S::kKG; ++gk) {
          uint32_t b[4];
          ldsm(b, kt + gk * 16 * D + (b0 ^ k_x));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t(&a)[4] = qf[ks + h];
            mma(s[2 * gk], a, e4m3_f16(b[h]), e4m3_f16(b[h] >> 16));
            mma(s[2 * gk + 1], a, e4m3_f16(b[2 + h]), e4m3_f16(b[2 + h] >> 16));
          }
        }
      }
      // this warp's factors, before the keys' place is given back
      constexpr int kGroups = S::kBlocks ? S::kKG : 1;
      float by_k[kGroups], v_of[kGroups];
      if constexpr (S::kBlocks) {
        read_factors(by_k, &factors->k[keys.slot][warp * S::kKG]);
        read_factors(v_of, &factors->v[keys.slot][warp * S::kKG]);
      }
      __syncwarp();
      if (!held && lane == 0) arrive(&c.empty[keys.slot]);
      if (part) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int in = in0 + n * 8 + 2 * quad + e;
            if (!sees(in, p0)) s[n][e] = -INFINITY;
            if (!sees(in, p1)) s[n][2 + e] = -INFINITY;
          }
      }

      // softmax of this warp's keys; m is 7 below the largest score (weights start at 2^7) and moves only when a score
      // makes weights more than 2^8 times as large
      float t0 = s[0][0], t1 = s[0][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        t0 = fmaxf(t0, fmaxf(s[n][0], s[n][1]));
        t1 = fmaxf(t1, fmaxf(s[n][2], s[n][3]));
      }
      if constexpr (S::kBlocks) {
        t0 = t1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
          const float a = fmaxf(fmaxf(s[2 * n][0], s[2 * n][1]), fmaxf(s[2 * n + 1][0], s[2 * n + 1][1]));
          const float b = fmaxf(fmaxf(s[2 * n][2], s[2 * n][3]), fmaxf(s[2 * n + 1][2], s[2 * n + 1][3]));
          t0 = fmaxf(t0, __fadd_rn(__fmul_rn(a, factor_of(c0, by_k[n])), log2_of(v_of[n])));
          t1 = fmaxf(t1, __fadd_rn(__fmul_rn(b, factor_of(c1, by_k[n])), log2_of(v_of[n])));
        }
      } else {
        t0 *= c0;
        t1 *= c1;
      }
      constexpr float kLift = Elem<__half>::kLift;
      if (__any_sync(0xffffffffu, t0 - mx0 > 8.0f + kLift || t1 - mx1 > 8.0f + kLift)) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
        const float n0 = fmaxf(mx0, fabsf(t0) > kLarge ? t0 : t0 - kLift), n1 = fmaxf(mx1, fabsf(t1) > kLarge ? t1 : t1 - kLift);
        const float a0 = n0 == mx0 ? 1.0f : ex2(mx0 - n0), a1 = n1 == mx1 ? 1.0f : ex2(mx1 - n1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int d = 0; d < kOT; ++d) {
          o[d][0] *= a0;
          o[d][1] *= a0;
          o[d][2] *= a1;
          o[d][3] *= a1;
        }
        mx0 = n0;
        mx1 = n1;
        large = __any_sync(0xffffffffu, (mx0 != -INFINITY && fabsf(mx0) > kLarge) || (mx1 != -INFINITY && fabsf(mx1) > kLarge));
      }
      const float z0 = mx0 == -INFINITY ? 0.0f : mx0, z1 = mx1 == -INFINITY ? 0.0f : mx1;
      if (large) {
        Scores<kNT> x;
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x.s[n][e] = s[n][e];
        if constexpr (S::kBlocks) {
          GroupFactors<kNT / 2> f;
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            f.k[n] = by_k[n];
            f.log[n] = log2_of(v_of[n]);
          }
          x = large_weights_blocks(x, f, c0, z0, c1, z1);
        } else {
          x = large_weights(x, c0, z0, c1, z1);
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = x.s[n][e];
      } else if constexpr (S::kBlocks) {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const float a = factor_of(c0, by_k[n / 2]), b = factor_of(c1, by_k[n / 2]), u0 = log2_of(v_of[n / 2]) - z0, u1 = log2_of(v_of[n / 2]) - z1;
          s[n][0] = ex2(fmaf(s[n][0], a, u0));
          s[n][1] = ex2(fmaf(s[n][1], a, u0));
          s[n][2] = ex2(fmaf(s[n][2], b, u1));
          s[n][3] = ex2(fmaf(s[n][3], b, u1));
        }
      } else {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          s[n][0] = ex2(fmaf(s[n][0], c0, -z0));
          s[n][1] = ex2(fmaf(s[n][1], c0, -z0));
          s[n][2] = ex2(fmaf(s[n][2], c1, -z1));
          s[n][3] = ex2(fmaf(s[n][3], c1, -z1));
        }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if constexpr (S::kBlocks) {
          l0 = fmaf(s[n][0] + s[n][1], back_of(v_of[n / 2]), l0);
          l1 = fmaf(s[n][2] + s[n][3], back_of(v_of[n / 2]), l1);
        } else {
          l0 += s[n][0] + s[n][1];
          l1 += s[n][2] + s[n][3];
        }
      }

      // times the values
      if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&c.full[values.slot], values.parity, P.spin_limit, 0u));
      bool odd = false;  // a value of a partly visible tile is not finite
      auto clean = [&](uint32_t& x) {
        const uint32_t y = finite(x);
        odd |= y != x;
        x = y;
      };
#pragma unroll
      for (int gk = 0; gk < S::kKG; ++gk) {
        // weights are rounded to f16 for the product (half a step, 2^-12 of each, random in sign; those below 2^-14, 2^-21
        // of the largest, by up to 2^-25); their sum is not
        const uint32_t a[4] = {Pack<__half>::pack(s[2 * gk][0], s[2 * gk][1]), Pack<__half>::pack(s[2 * gk][2], s[2 * gk][3]),
                               Pack<__half>::pack(s[2 * gk + 1][0], s[2 * gk + 1][1]), Pack<__half>::pack(s[2 * gk + 1][2], s[2 * gk + 1][3])};
#pragma unroll
        for (int b0 = 0; b0 < D; b0 += 32) {
          const int d = b0 / 8;
          uint32_t b[4];
          ldsm_t(b, vt + gk * 16 * D + (b0 ^ v_x));
          // a register holds two neighbouring columns of two keys: even columns to one product, odd to the other
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t even = __byte_perm(b[2 * h], b[2 * h + 1], 0x6420), odds = __byte_perm(b[2 * h], b[2 * h + 1], 0x7531);
            uint32_t f[4] = {e4m3_f16(even), e4m3_f16(even >> 16), e4m3_f16(odds), e4m3_f16(odds >> 16)};
            if (part) {
#pragma unroll
              for (int e = 0; e < 4; ++e) clean(f[e]);
            }
            mma(o[d + 2 * h], a, f[0], f[1]);
            mma(o[d + 2 * h + 1], a, f[2], f[3]);
          }
        }
      }
      if (part && __any_sync(0xffffffffu, odd)) {
        // Some value in the tile is not finite and was left out above; rows that see its key take it here, one
        // key at a time (0 * NaN of a row that does not see it must not happen).
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
#pragma unroll 1
          for (int src = 0; src < 8; ++src) {
            const int from = (lane & ~3) + (src >> 1);
            const float e0 = __shfl_sync(0xffffffffu, s[n][0], from), e1 = __shfl_sync(0xffffffffu, s[n][1], from);
            const float e2 = __shfl_sync(0xffffffffu, s[n][2], from), e3 = __shfl_sync(0xffffffffu, s[n][3], from);
            const float w0 = src & 1 ? e1 : e0, w1 = src & 1 ? e3 : e2;
            const int in = in0 + n * 8 + src;
            const bool v0 = sees(in, p0), v1 = sees(in, p1);
#pragma unroll
            for (int d = 0; d < kOT; ++d)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int col = (d >> 1) * 16 + 4 * quad + 2 * x + (d & 1);
                const float v = __half2float(__ushort_as_half((unsigned short)e4m3_f16(ring[values.slot * S::kSlot + place_of<D>(in, col)])));
                if (!isfinite(v)) {
                  if (v0) o[d][x] = fmaf(w0, v, o[d][x]);
                  if (v1) o[d][2 + x] = fmaf(w1, v, o[d][2 + x]);
                }
              }
          }
        }
      }
      __syncwarp();
      if (!held && lane == 0) arrive(&c.empty[values.slot]);
    }
    if (dead && lane == 0) atomicOr(&P.row_status[g.row], (uint32_t)SS_ST_COPY_TIMEOUT);

    const float v_scale = P.v_scale ? P.v_scale[g.h] : 1.0f;
    fetch((sg + 1) & 1, ((sg + 1) >> 1) & 1);

    // ---- join of the warps: each leaves its piece in the room of the last tiles and adds a quarter of the columns
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    static_assert(kWarps == 4 && 2 * kOT * 32 * 16 <= S::kSlot, "room for two pieces in a tile's place");
    auto room = [&](int w) { return reinterpret_cast<float4*>(ring + (w < 2 ? keys.slot : values.slot) * S::kSlot) + (w & 1) * kOT * 32 + lane; };
    bar_warps<kWarps>();  // the tiles have been read
#pragma unroll
    for (int d = 0; d < kOT; ++d) room(warp)[d * 32] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
    if (quad == 0) {
      c.ml[warp][r0] = make_float2(mx0, l0);
      c.ml[warp][r0 + 8] = make_float2(mx1, l1);
    }
    bar_warps<kWarps>();
    const bool whole = g.ca == g.cb;
    float top[2], sum[2], by[2][kWarps];  // by row r0 and r0 + 8
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float2 ml[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ml[w] = c.ml[w][r0 + 8 * x];
      top[x] = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
      const float z = top[x] == -INFINITY ? 0.0f : top[x];
      sum[x] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        by[x][w] = ex2(ml[w].x - z);
        sum[x] = fmaf(ml[w].y, by[x][w], sum[x]);
      }
      const float f = (whole ? (sum[x] == 0.0f ? 0.0f : 1.0f / sum[x]) : 1.0f) * v_scale;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) by[x][w] *= f;
    }
    float4 y[kOT / kWarps];
#pragma unroll
    for (int d = 0; d < kOT / kWarps; ++d) {
      y[d] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 z = room(w)[(warp * (kOT / kWarps) + d) * 32];
        y[d] = make_float4(fmaf(z.x, by[0][w], y[d].x), fmaf(z.y, by[0][w], y[d].y), fmaf(z.z, by[1][w], y[d].z), fmaf(z.w, by[1][w], y[d].w));
      }
    }
    const int mine = piece_of(g, blockIdx.x);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int m = x ? m1 : m0;
      if (m >= rows_here) continue;
      const int f = g.mt * kRows + m, j = token_of(P, f), head = g.h * P.group + f - j * P.group;
      T* to = static_cast<T*>(P.out) + (g.q0 + j) * P.out_stride + head * D;
#pragma unroll
      for (int n = 0; n < kOT / kWarps; n += 2) {
        const int d = warp * (kOT / kWarps) + n;
        const float4 z = x ? make_float4(y[n].z, y[n + 1].z, y[n].w, y[n + 1].w) : make_float4(y[n].x, y[n + 1].x, y[n].y, y[n + 1].y);
        if (whole)
          *reinterpret_cast<uint2*>(to + d * 8 + quad * 4) = make_uint2(Pack<T>::pack(z.x, z.y), Pack<T>::pack(z.z, z.w));
        else
          piece_out<D>(P, mine)[(d * 2 + quad) * kRows + m] = z;
      }
      if (quad == 0 && warp == 0) {
        if (!whole) piece_ml(P, mine)[m] = make_float4(top[x], sum[x], sum[x], 0.0f);
        else if (P.lse)
          P.lse[(size_t)(g.q0 + j) * (P.group * P.hkv) + head] = sum[x] == 0.0f ? -INFINITY : (top[x] + log2f(sum[x])) * 0.69314718055994531f;
      }
    }
    // the room is given back to the loads
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      arrive(&c.empty[keys.slot]);
      arrive(&c.empty[values.slot]);
    }
    if (!whole) join_unit<T, Pack<T>, D, 32 * kWarps>(P, g, &c.last, bar_warps<kWarps>);
    __syncwarp();
    if (lane == 0) arrive(&c.seg_empty[sg & 1]);
  }
  if (dead && threadIdx.x == 0) report_range(P, &c.range);
}

// ------------------------------------------------------------------ kernel
template <class T, int D, bool BLOCKS>
__global__ void __launch_bounds__(kThreads, (Shape<T, D, BLOCKS>::kCtas))
    attend_kernel(const AttendParams P, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Shape<T, D, BLOCKS>;
  static_assert(S::kSlots >= 4, "ring length");
  extern __shared__ unsigned char raw[];
  unsigned char* ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  unsigned char* sq = ring + S::kSlots * S::kSlot;
  Control& c = *reinterpret_cast<Control*>(sq + kRows * S::kQRow);
  TileFactors* factors = BLOCKS ? reinterpret_cast<TileFactors*>(sq + kRows * S::kQRow + kControl) : nullptr;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&c.full[i]);
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&c.empty[i])), "r"(kWarps) : "memory");
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.seg_full[i]);
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&c.seg_empty[i])), "r"(kWarps) : "memory");
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps && lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &mv : &mk) : "memory");

  find_range<kThreads, kWarps>(P, c.range_sums, &c.range);
  if (c.range.cut.ctas == 0) return;
  if (warp == kWarps) load_warp<S>(P, &mk, &mv, ring, c, factors, c.range);
  else compute_warps<S, T, D>(P, ring, sq, c, factors);
}

template <class T, int D, bool BLOCKS>
AttendKernel entry() {
  using S = Shape<T, D, BLOCKS>;
  // What starting and ending a unit takes, in tiles.  Measured (us): 128 columns, 128 x 1 rows of at most 3000 tokens with
  // 2, 3, 4, 5: 96, 85.5, 88.5, 91.4; 32 x 4 rows of at most 32000: 176, 154, 152.6, 152.9; 64 columns, 200 x 1 rows of at
  // most 2000 with 1, 2, 3, 4: 38.4, 34.3, 35, 36.3.
  constexpr int kUnitCost = D == 128 ? 3 : 2;
  return {reinterpret_cast<const void*>(&attend_kernel<T, D, BLOCKS>), kThreads, S::kSlots, 0, 1, S::kCtas, kTile, smem_bytes<S>(), kUnitCost, true};
}
template <class T, bool BLOCKS = false>
AttendKernel pick(int d) {
  return d == 64 ? entry<T, 64, BLOCKS>() : entry<T, 128, BLOCKS>();
}

}  // namespace kv8
}  // namespace ss
