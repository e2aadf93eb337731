// ss_attend for 16-bit caches: attention of a step's new tokens over the paged
// key-value cache, on the 5th-generation tensor cores.
//
// Mathematics.  For a query q at position p, o = sum_t w_t v_t / sum_t w_t
// with w_t = 2^(c q.k_t - m), c = scale * log2 e and m any number near the
// largest exponent: one pass over the keys.  m is the maximum of the first
// tile that a row sees, less 7 where weights are f16; when a later tile makes
// weights 2^8 times as large as that tile's the sum and the output so far are
// scaled down and m moves (bf16 weights up to 2^8 and f16 weights up to 2^15
// lose nothing, and the output, which lives in tensor memory, is hardly ever
// touched).  The 7 are for f16's short lower end: weights below 2^-25 are held
// as 0, which the divisor does not know of; beside one dominant key that would
// be 1 % of a row of 400000 faint ones, and is 1 in 10000 at 2^-32.  Pieces (m, l, O) over disjoint keys join as
// (max m, sum l 2^(m_i - m), sum O 2^(m_i - m)), so the keys of a row can be
// split anywhere.
//
// What bounds it.  A key and its value (2 * head_dim elements) are read once
// for the n * group queries of a key head (n new tokens, group = q_heads /
// kv_heads): 4 * head_dim * n * group operations on 4 * head_dim bytes, i.e.
// 1 .. 128 operations a byte where the card's tensor rate over its HBM rate is
// about 280.  HBM bandwidth is the bound, and the kernel's one aim is to keep
// loads in flight everywhere until the end.
//
// A CTA's warps (how the work is cut up: ss_kv_work.cuh):
//  - load: walks the CTA's range, publishes its segments, gathers their query
//    rows into shared memory and runs the ring of key and value tiles: TMA
//    copies of a page (or 64 tokens of it), page ids read a batch ahead.
//  - product: one thread issues S = Q K^T (128 x 64, both from shared memory)
//    and O += P V (P from tensor memory) with tcgen05.mma; S of a tile is
//    issued before the weights of the tile before it are ready.
//  - four softmax warps: a thread owns a query row (a lane of tensor memory),
//    so maxima and sums need no exchange; it reads its 64 scores, writes its
//    weights over them and never waits for the products in between.
//  - With 64 columns a tile's loads are short and one warp's 64 exponentials a
//    row would take longer.  Where a unit has at most 64 (32) query rows they
//    are there twice (four times), in lanes 64 (32) apart, and each copy weighs
//    its half (quarter) of a tile's keys and zeros elsewhere; the copies' sums
//    and outputs are added at the end of the unit.
//  Query rows past the live ones are whatever follows in shared memory: rows
//  of a product do not mix, and nothing reads theirs.  Padding to 128 rows
//  costs tensor time only (measured with one live row in eight it stays below
//  the time of the loads), and a warp without live rows skips its part.
//  - A unit that lies in several CTAs is joined by the last of them to arrive
//    (ss_kv_join.cuh).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "ss_kv_blocks.cuh"
#include "ss_kv_join.cuh"
#include "ss_stage1.cuh"

namespace ss {
namespace kv {

constexpr int kTile = 64;                        // keys of a tile
constexpr int kSoftmaxWarps = 4;                 // warps 0 .. 3: a warp reaches the 32 lanes of its number modulo 4
constexpr int kLoadWarp = 4, kProductWarp = 5;
constexpr int kMaxSlots = 16;                    // tiles of keys or values in the ring
constexpr int kMaxRaw = 8;                       // 8-bit tiles in their ring
constexpr int kBadTiles = 16;                    // tiles whose unreadable keys are kept
constexpr int kControl = 4096;                   // bytes of the control block, at most
constexpr uint32_t kDrainPolls = 1u << 22;

// ------------------------------------------------------------------ types
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;       // of tcgen05.mma's operands
  static constexpr uint32_t kExponent = 0x7f80;
  static constexpr float kLift = 0.0f;         // of weights, in powers of two (see above)
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <>
struct Elem<__half> {
  static constexpr uint32_t kFormat = 0;
  static constexpr uint32_t kExponent = 0x7c00;
  static constexpr float kLift = 7.0f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
};

// ------------------------------------------------------------------ instructions
__device__ __forceinline__ void mbar_init_n(unsigned long long* m, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(m)), "r"(n) : "memory");
}
__device__ __forceinline__ void arrive(unsigned long long* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(m)) : "memory");
}
// One look at a barrier's phase.  Looks at two barriers overlap, where one wait after the other would take twice the
// time even if both phases are done.
__device__ __forceinline__ bool done(unsigned long long* m, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(m)), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ void expect(unsigned long long* m, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(m)), "r"(bytes) : "memory");
}
// counts bytes that are to come without arriving
__device__ __forceinline__ void expect_only(unsigned long long* m, int bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(m)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, unsigned long long* m, int token, int run, int head,
                                         int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(0), "r"(token), "r"(run), "r"(head), "r"(page), "r"(smem_u32(m))
      : "memory");
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// arrives at m when every product issued so far by this thread is done
__device__ __forceinline__ void commit(unsigned long long* m) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(m)) : "memory");
}
// D (+)= A B^T, A and B from shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a),
               "l"(b), "r"(desc), "r"((uint32_t)add)
               : "memory");
}
// D (+)= A B, A from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a),
               "l"(b), "r"(desc), "r"((uint32_t)add)
               : "memory");
}
// Tensor memory: this warp's 32 lanes, a register for each of n columns from `at` on.
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[64], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]),
        "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
        "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]),
        "=r"(r[63])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[1], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\ntcgen05.wait::ld.sync.aligned;" : "=r"(r[0]) : "r"(at) : "memory");
}
// Shared-memory operand of lines of 128 bytes, swizzled: 8 lines (1024 bytes) from one group of 8 to the next, `lead`
// bytes from one run of 64 columns to the next where a product spans several.
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t lead) {
  return (uint64_t)((at & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// ------------------------------------------------------------------ shape of one instantiation
// (BLOCKS: 8-bit values with a factor for each block of tokens.)
template <class T, int D, int KEYS, bool LOW, bool BLOCKS = false>
struct Shape {
  static_assert(LOW || !BLOCKS, "factors belong to 8-bit values");
  static constexpr bool kBlocks = BLOCKS;
  using Mul = typename std::conditional<LOW, __half, T>::type;  // what is multiplied: 8-bit values become f16
  static constexpr bool kLow = LOW;
  static constexpr bool kScaleQ = LOW && std::is_same<T, __nv_bfloat16>::value;
  static constexpr int kThreads = LOW ? 320 : 192;           // 8 bits: four warps more, which convert
  static constexpr int kRaw = kTile * D;                     // bytes of a tile of 8-bit values
  static constexpr int kCopies = kTile / KEYS;               // of the queries; a softmax thread weighs KEYS keys of a tile
  static constexpr int kLanes = 128 / kCopies;               // lanes of a copy
  static constexpr int kRuns = D / 64;                       // runs of 64 columns (128 bytes)
  static constexpr int kRun = kTile * 128;                   // bytes of a run of a tile
  static constexpr int kSlot = kRuns * kRun;                 // bytes of a tile of keys or of values
  static constexpr int kCtas = D <= 128 ? 2 : 1;             // CTAs per SM
  static constexpr uint32_t kCols = D <= 128 ? 256 : 512;    // columns of tensor memory: two tiles of scores, the output
  static constexpr uint32_t kOut = 128;
  // instruction descriptors: 32-bit sums, both operands of type T, 128 rows; S: 64 columns; O: D columns, V as it lies
  static constexpr uint32_t kCommon = 1u << 4 | Elem<Mul>::kFormat << 7 | Elem<Mul>::kFormat << 10 | (128u >> 4) << 24;
  static constexpr uint32_t kScores = kCommon | (kTile >> 3) << 17;
  static constexpr uint32_t kValues = kCommon | 1u << 16 | (uint32_t)(D >> 3) << 17;
};

struct Control {
  unsigned long long full[kMaxSlots], empty[kMaxSlots];  // ring: copies landed; products done with them
  unsigned long long seg_full[2], seg_empty[2];          // segment published with its queries; done with by all
  unsigned long long s_full[2], p_full[2], pv_done[2];   // scores there; weights there; added to the output
  unsigned long long o_free, q_free, drained;            // output read; last scores of a segment there; all products done
  Segment seg[2];
  Range range;
  long long sums[10];
  // Per tile, by its number in the CTA's range modulo kBadTiles: its 16-key groups that lie on pages with a bad id.  Not
  // by its place in the ring: that is free as soon as the scores are there, before the softmax warps have looked.
  int bad[kBadTiles];
  int slow[2];         // the tile's values were added by the softmax warps
  unsigned long long raw_full[kMaxRaw], raw_empty[kMaxRaw];  // ring of 8-bit tiles: copies landed; converted
  float q_back[2][128];  // per query row, what its f16 values were scaled by, undone
  int last;
  uint32_t tmem;
  float4 ml[128];      // of the copies of a row, as in a piece
};
static_assert(sizeof(Control) <= kControl, "control block");
// The load warp writes the word of tile t once the place of its keys is free, so with all places of the ring(s) before it
// given back; among them is that of the values of tile t - (places + 2) / 2 at the latest, which took the weights of
// every softmax warp.
static_assert((kMaxSlots + kMaxRaw + 2) / 2 <= kBadTiles && (kBadTiles & (kBadTiles - 1)) == 0, "tiles ahead of the softmax");

// Factors of the tiles' keys, kept as the words of `bad` are.
using TileFactors = Factors<kBadTiles, kTile / 16>;
static_assert(sizeof(TileFactors) <= 1024, "room for factors");

// Rows of a query buffer: where there are copies, all 128.
template <class S>
__device__ __forceinline__ uint32_t q_rows(const AttendParams& P) {
  return S::kCopies > 1 ? 128u : (uint32_t)P.rows;
}

// A place in the ring: tiles of keys and of values take turns.
struct Turn {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      parity ^= 1;
    }
  }
};

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool any_softmax(bool x) {  // over the softmax warps, which it also brings together
  uint32_t y;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(y)
               : "r"((uint32_t)x)
               : "memory");
  return y != 0;
}

// Does the diagonal or a window's edge cut tile `base` of the unit for some live row?  It follows from the segment alone,
// so that the softmax warps, which meet at a barrier in such tiles, agree on it even when one of them has lost a wait.
__device__ __forceinline__ bool partly(const AttendParams& P, const Unit& u, int base) {
  return base + kTile - 1 > u.pos0 || (P.window > 0 && base <= u.pos1 - P.window && base > P.sinks - kTile);
}
// As bits, the keys of tile `base` that are visible from position p.
__device__ __forceinline__ uint64_t visible_keys(const AttendParams& P, int base, int p, int bad) {
  auto below = [&](int key) {  // keys before `key`
    const int n = key - base;
    return n <= 0 ? 0ull : n >= kTile ? ~0ull : (1ull << n) - 1;
  };
  uint64_t seen = below(p + 1);  // (positions stay below 2^31 - 1)
  if (P.window > 0) seen &= ~below(p - P.window + 1) | below(P.sinks);
  for (int n = 0; bad != 0 && n < kTile / 16; ++n)
    if ((bad >> n) & 1) seen &= ~(0xffffull << (16 * n));
  return seen;
}

// ------------------------------------------------------------------ load warp
template <class S, class T, int D>
__device__ void load_warp(const AttendParams& P, const CUtensorMap* mk, const CUtensorMap* mv, uint32_t sq, uint32_t ring, uint32_t raw,
                          Control& c, TileFactors* factors) {
  // the ring that the copies fill
  unsigned long long* const full = S::kLow ? c.raw_full : c.full;
  unsigned long long* const empty = S::kLow ? c.raw_empty : c.empty;
  const int slots = S::kLow ? P.raw_slots : P.slots;
  const uint32_t copies = S::kLow ? raw : ring;
  constexpr int kBytes = S::kLow ? S::kRaw : S::kSlot;
  const int lane = threadIdx.x & 31;
  const int box_shift = min(P.page_shift, 6);            // tokens of one copy
  const int subs_shift = 6 - box_shift;                  // copies of a run of a tile
  const int runs = S::kLow || !subs_shift ? 1 : S::kRuns;  // a copy of 64 tokens, or of 8-bit values, has every run
  const int batch = 32 >> subs_shift;                    // tiles whose page ids one lane each holds
  const int sub = lane & ((1 << subs_shift) - 1), nth = lane >> subs_shift;
  const int page_mask = (1 << P.page_shift) - 1;
  const int groups = (1 << (1 << (box_shift - 4))) - 1;  // 16-key groups of a copy, as bits
  const uint32_t q_bytes = q_rows<S>(P) * D * 2;
  Turn turn;
  int asked = 0;                                         // copies in flight or landed, at most `slots`
  uint32_t it = 0;                                       // tiles so far
  bool dead = false;
  Range k = c.range;
  Segment g;
  int sg = 0;
  bool more = true;
  while (more && !dead) {
    more = next_segment(P, k, g);
    // the segment's place is free once segment sg - 2 is done with; so is a second query buffer, and an only one once
    // the last scores of segment sg - 1 are there, or, where its output goes by way of that buffer (copies), all of it
    if (sg >= 2) dead = !__all_sync(0xffffffffu, mbar_wait(&c.seg_empty[sg & 1], ((sg >> 1) & 1) ^ 1, P.spin_limit, 0u));
    if (sg >= 1 && P.q_bufs == 1 && !dead)
      dead = !__all_sync(0xffffffffu, S::kCopies > 1 ? mbar_wait(&c.seg_empty[(sg - 1) & 1], ((sg - 1) >> 1) & 1, P.spin_limit, 0u)
                                                     : mbar_wait(&c.q_free, (sg & 1) ^ 1, P.spin_limit, 0u));
    if (dead) break;
    if (!more) g.count = 0;  // the end of the range
    if (lane == 0) c.seg[sg & 1] = g;
    const int32_t* table = P.block_table + (long long)g.row * P.max_blocks;
    const int used = (g.len + page_mask) >> P.page_shift;
    // Whether this lane's copy in the batch from tile i0 on is of tokens that the row holds, and its page: read a batch
    // ahead and looked at only then.  Where nothing is held the copy is from past the cache and reads zeros.
    auto block_of = [&](int i0) { return (tile_of(g.u, g.from + i0 + nth) * kTile + (sub << box_shift)) >> P.page_shift; };
    auto holds = [&](int i0) { return i0 + nth < g.count && block_of(i0) < used; };
    auto fetch = [&](int i0) { return holds(i0) ? __ldg(table + block_of(i0)) : P.num_pages; };
    int next = fetch(0);
    if (more) {
      const uint32_t to = sq + (P.q_bufs == 2 && (sg & 1) ? q_bytes : 0u);
      const int pieces = g.live * (D / 8);
      auto source = [&](int i) {
        const int m = i / (D / 8), piece = i % (D / 8), f = g.mt * P.rows + m, j = token_of(P, f);
        return static_cast<const T*>(P.q) + (g.q0 + j) * P.q_stride + (g.h * P.group + f - j * P.group) * D + piece * 8;
      };
      auto place = [&](int i) {
        const int m = i / (D / 8), piece = i % (D / 8);
        return to + (piece >> 3) * (q_rows<S>(P) * 128) + m * 128 + (((piece & 7) ^ (m & 7)) << 4);
      };
      if constexpr (S::kScaleQ) {
        // bf16 to f16: a row is scaled by a power of two that brings its largest value near 2^14, so every value keeps
        // its bits unless it is below 2^-28 of the largest
        constexpr int kBatch = 8;  // loads in flight
        for (int i0 = lane; i0 - lane < pieces; i0 += 32 * kBatch) {
          uint4 x[kBatch];
#pragma unroll
          for (int n = 0; n < kBatch; ++n)
            x[n] = i0 + 32 * n < pieces ? __ldg(reinterpret_cast<const uint4*>(source(i0 + 32 * n))) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int n = 0; n < kBatch; ++n) {
            const int i = i0 + 32 * n;
            using B = Elem<__nv_bfloat16>;
            using H = Elem<__half>;
            const float2 v0 = B::unpack(x[n].x), v1 = B::unpack(x[n].y), v2 = B::unpack(x[n].z), v3 = B::unpack(x[n].w);
            float top = fmaxf(fmaxf(fmaxf(fabsf(v0.x), fabsf(v0.y)), fmaxf(fabsf(v1.x), fabsf(v1.y))),
                              fmaxf(fmaxf(fabsf(v2.x), fabsf(v2.y)), fmaxf(fabsf(v3.x), fabsf(v3.y))));
#pragma unroll
            for (int o = D / 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int ex = max((int)(__float_as_uint(top) >> 23), 15);                // biased exponent
            const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - ex) << 23);  // 2^(14 - exponent)
            if (i >= pieces) continue;
            if (i % (D / 8) == 0) c.q_back[sg & 1][i / (D / 8)] = __uint_as_float((uint32_t)(ex - 14) << 23);
            const uint32_t w0 = H::pack(v0.x * up, v0.y * up), w1 = H::pack(v1.x * up, v1.y * up), w2 = H::pack(v2.x * up, v2.y * up),
                           w3 = H::pack(v3.x * up, v3.y * up);
#pragma unroll
            for (int y = 0; y < S::kCopies; ++y)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(i) + y * S::kLanes * 128), "r"(w0), "r"(w1), "r"(w2), "r"(w3)
                           : "memory");
          }
        }
      } else {
        for (int i = lane; i < pieces; i += 32) {
#pragma unroll
          for (int n = 0; n < S::kCopies; ++n)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place(i) + n * S::kLanes * 128), "l"(source(i)) : "memory");
        }
      }
    }
    CopyFactors mine;   // of this lane's copy in the batch
    int keys_at = 0;    // place of the tile's keys in the ring
    const int per_copy = 1 << (box_shift - 4);
    auto place_of = [&](int i0) { return (tile_of(g.u, g.from + i0 + nth) * kTile + (sub << box_shift)) & page_mask; };
    bool published = false;
    auto publish = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      proxy_fence();
      __syncwarp();
      if (lane == 0) arrive(&c.seg_full[sg & 1]);
      published = true;
    };
    if (!more) publish();
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
#pragma unroll(S::kLow ? 1 : 2)
        for (int values = 0; values < 2; ++values) {
          dead = !__all_sync(0xffffffffu, mbar_wait(&empty[turn.slot], turn.parity ^ 1, P.spin_limit, 0u));
          if (S::kBlocks && dead && values && lane == 0) arrive(&full[keys_at]);  // (its copy is waited for at the end)
          if (dead) break;
          if (lane == 0) {
            if (!values) {
              int bits = 0;
              for (int s = 0; s < 1 << subs_shift; ++s)
                if ((bad_lanes >> ((j << subs_shift) + s)) & 1) bits |= groups << (s << (box_shift - 4));
              c.bad[it++ & (kBadTiles - 1)] = bits;
            }
            if (S::kBlocks && !values) expect_only(&full[turn.slot], kBytes);
            else expect(&full[turn.slot], kBytes);
          }
          __syncwarp();
          if (nth == j)
            for (int r = 0; r < runs; ++r)
              tma_load(copies + turn.slot * kBytes + r * S::kRun + (sub << box_shift) * (S::kLow ? D : 128), values ? mv : mk,
                       &full[turn.slot], tok, r, g.h, id);
          if constexpr (S::kBlocks) {
            if (!values) {
              keys_at = turn.slot;
            } else {  // the factors come with the keys, whose barrier waits for them too
              const int tile = (__shfl_sync(0xffffffffu, it, 0) - 1) & (kBadTiles - 1);
              if (nth == j) mine.write(*factors, tile, sub * per_copy, per_copy);
              __syncwarp();
              if (lane == 0) arrive(&full[keys_at]);
            }
          }
          turn.next(slots);
          asked = min(asked + 1, slots);
        }
        if (!published && !dead) publish();
      }
      if (S::kBlocks && i0 + batch < g.count) {  // the next batch's, whose page ids have come meanwhile
        const bool there = holds(i0 + batch) && (unsigned)next < (unsigned)P.num_pages;
        mine.fetch(P, there, next, g.h, place_of(i0 + batch), per_copy);
      }
    }
    if (!published) publish();
    ++sg;
  }
  // no copy may be in flight when the CTA ends (all have landed unless a wait ran out)
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (; asked > 0; --asked) {
    if (--turn.slot < 0) {
      turn.slot = slots - 1;
      turn.parity ^= 1;
    }
    mbar_wait(&full[turn.slot], turn.parity, kDrainPolls, 0u);
  }
}

// ------------------------------------------------------------------ converting warps
// Two e4m3 values (the low 16 bits of w) as f16x2: exact.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t w) {
  uint32_t d;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(d) : "r"(w));
  return d;
}

// From the ring of 8-bit tiles (a token after the other, as the copies bring them) to that of the products (runs of
// 64 columns, swizzled).  The load warp publishes segments; these warps follow their tile counts.
template <class S, int D>
__device__ void convert_warps(const AttendParams& P, const unsigned char* raw, unsigned char* ring, Control& c) {
  const int tid = threadIdx.x - 32 * (kProductWarp + 1), lane = tid & 31;
  Turn from, to;
  bool dead = false;
  auto wait = [&](unsigned long long* m, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(m, parity, P.spin_limit, 0u));
  };
  int sg = 0;
  bool more = true;
  while (more) {
    wait(&c.seg_full[sg & 1], (sg >> 1) & 1);
    const int count = dead ? 0 : c.seg[sg & 1].count;
    more = count > 0;
    for (int i = 0; i < 2 * count && !dead; ++i) {
      wait(&c.raw_full[from.slot], from.parity);
      wait(&c.empty[to.slot], to.parity ^ 1);
      if (dead) break;
      const uint4* src = reinterpret_cast<const uint4*>(raw + from.slot * S::kRaw);
      unsigned char* dst = ring + to.slot * S::kSlot;
      uint4 x[D / 32];
#pragma unroll
      for (int n = 0; n < D / 32; ++n) x[n] = src[tid + 128 * n];
#pragma unroll
      for (int n = 0; n < D / 32; ++n) {
        const int at = tid + 128 * n, token = at / (D / 16), piece = at % (D / 16);  // 16 columns
        unsigned char* line = dst + (piece >> 2) * S::kRun + token * 128;
        const uint4 lo = make_uint4(e4m3_f16(x[n].x), e4m3_f16(x[n].x >> 16), e4m3_f16(x[n].y), e4m3_f16(x[n].y >> 16));
        const uint4 hi = make_uint4(e4m3_f16(x[n].z), e4m3_f16(x[n].z >> 16), e4m3_f16(x[n].w), e4m3_f16(x[n].w >> 16));
        // every other run's second half first: neighbouring runs would meet in the same banks
        const int swap = (piece >> 2) & 1, c0 = (piece & 3) * 2 + swap, c1 = (piece & 3) * 2 + 1 - swap;
        *reinterpret_cast<uint4*>(line + ((c0 ^ (token & 7)) << 4)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(line + ((c1 ^ (token & 7)) << 4)) = swap ? lo : hi;
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) {
        arrive(&c.raw_empty[from.slot]);
        arrive(&c.full[to.slot]);
      }
      from.next(P.raw_slots);
      to.next(P.slots);
    }
    if (more && lane == 0) arrive(&c.seg_empty[sg & 1]);
    ++sg;
  }
}

// ------------------------------------------------------------------ product thread
template <class S, class T, int D>
__device__ void product_thread(const AttendParams& P, uint32_t sq, uint32_t ring, Control& c) {
  const uint32_t tmem = c.tmem, q_bytes = q_rows<S>(P) * D * 2, q_run = q_rows<S>(P) * 128;
  Turn turn;
  bool dead = false;
  auto wait = [&](unsigned long long* m, uint32_t parity) {
    if (!dead) dead = !mbar_wait(m, parity, P.spin_limit, 0u);
  };
  uint32_t it = 0;  // tiles so far
  int sg = 0;
  // adds the weights of tile `tile` times its values to the output
  auto values = [&](uint32_t tile, const Turn& at, bool first) {
    const int b = tile & 1;
    const bool there = done(&c.full[at.slot], at.parity), weighed = done(&c.p_full[b], (tile >> 1) & 1);
    if (first) wait(&c.o_free, (sg & 1) ^ 1);
    if (!there) wait(&c.full[at.slot], at.parity);
    if (!weighed) wait(&c.p_full[b], (tile >> 1) & 1);
    if (dead) return;
    fence_after();
    if (!c.slow[b]) {
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(tmem + S::kOut, tmem + b * kTile + k * 8, operand(ring + at.slot * S::kSlot + k * 2048, S::kRun), S::kValues, !first || k);
    }
    commit(&c.empty[at.slot]);
    commit(&c.pv_done[b]);
  };
  bool more = true;
  while (more && !dead) {
    wait(&c.seg_full[sg & 1], (sg >> 1) & 1);
    const int count = dead ? 0 : c.seg[sg & 1].count;
    more = count > 0;
    if (!more) break;
    const uint32_t q = sq + (P.q_bufs == 2 && (sg & 1) ? q_bytes : 0u);
    Turn before;  // the values of the tile before
    for (int i = 0; i < count && !dead; ++i, ++it) {
      const int b = it & 1;
      // the keys, and the weights of two tiles ago, which are in the same columns
      const bool there = done(&c.full[turn.slot], turn.parity), used = done(&c.pv_done[b], ((it >> 1) & 1) ^ 1);
      if (!there) wait(&c.full[turn.slot], turn.parity);
      if (!used) wait(&c.pv_done[b], ((it >> 1) & 1) ^ 1);
      if (dead) break;
      fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(tmem + b * kTile, operand(q + (k >> 2) * q_run + (k & 3) * 32, 0),
               operand(ring + turn.slot * S::kSlot + (k >> 2) * S::kRun + (k & 3) * 32, 0), S::kScores, k != 0);
      commit(&c.s_full[b]);
      commit(&c.empty[turn.slot]);
      if (i + 1 == count) commit(&c.q_free);
      turn.next(P.slots);
      if (i > 0) values(it - 1, before, i == 1);
      before = turn;
      turn.next(P.slots);
    }
    if (!dead) values(it - 1, before, count == 1);
    if (!dead) arrive(&c.seg_empty[sg & 1]);
    ++sg;
  }
  // nothing may be in flight when tensor memory is given back
  commit(&c.drained);
  mbar_wait(&c.drained, 0, kDrainPolls, 0u);
}

// ------------------------------------------------------------------ softmax warps
// A wait ran out: no row of the range is to be trusted.  (Out of line: it is not expected to run.)
static __device__ __noinline__ void report_range(const AttendParams& P, const Range* range) {
  Range k = *range;
  Segment g;
  while (next_segment(P, k, g)) atomicOr(&P.row_status[g.row], (uint32_t)SS_ST_COPY_TIMEOUT);
}

// x * scale - m is one operation, which knows more bits of the product than m has.  Where m is beyond 2^20 (a 16th of a
// power of two, the same for all keys; at 2^24 more than f16 weights can take) the product is rounded as m was, and m is
// the maximum itself: of scores that large 32 bits tell nothing below it.
constexpr float kLarge = 0x1p20f;

// A row's weights of one tile where m is large, over its scores: as in softmax_warps.  Returns their sums, that of the
// rounded ones first.  (Out of line, where it costs the other tiles nothing: as part of their code it did, 256 x 1 short
// rows 45 -> 49.5 us.)
template <class S, int KEYS>
static __device__ __noinline__ float2 large_weights(uint32_t at, int key0, float scale, float z, uint64_t seen) {
  using E = Elem<typename S::Mul>;
  float rounded = 0.0f, exact = 0.0f;
#pragma unroll 1
  for (int i = key0; i < key0 + KEYS; i += 16) {
    uint32_t x[16], w[8];
    tmem_load(x, at + i);
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
      float y[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        y[h] = (seen >> (i + n + h)) & 1 ? ex2(__fsub_rn(__fmul_rn(__uint_as_float(x[n + h]), scale), z)) : 0.0f;
      w[n / 2] = E::pack(y[0], y[1]);
      const float2 r = std::is_same<typename S::Mul, __nv_bfloat16>::value ? E::unpack(w[n / 2]) : make_float2(y[0], y[1]);
      rounded += r.x + r.y;
      exact += y[0] + y[1];
    }
    tmem_store(at + i / 2, w);
  }
  return make_float2(rounded, exact);
}

// The same with factors of blocks.
template <class S, int KEYS>
static __device__ __noinline__ float large_weights_blocks(uint32_t at, int key0, float scale, float z, uint64_t seen, const TileFactors& f, int tile) {
  using E = Elem<typename S::Mul>;
  float sum = 0.0f;
#pragma unroll 1
  for (int i = key0; i < key0 + KEYS; i += 16) {
    uint32_t x[16], w[8];
    tmem_load(x, at + i);
    const float v = f.v[tile][i >> 4], by = factor_of(scale, f.k[tile][i >> 4]), log = log2_of(v);
    float s = 0.0f;
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
      float y[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        y[h] = (seen >> (i + n + h)) & 1 ? ex2(__fsub_rn(__fadd_rn(__fmul_rn(__uint_as_float(x[n + h]), by), log), z)) : 0.0f;
      w[n / 2] = E::pack(y[0], y[1]);
      s += y[0] + y[1];
    }
    sum = fmaf(s, back_of(v), sum);
    tmem_store(at + i / 2, w);
  }
  return sum;
}

template <class S, class T, int D, int KEYS>
__device__ void softmax_warps(const AttendParams& P, unsigned char* sq, unsigned char* ring, Control& c, const TileFactors* factors) {
  using E = Elem<typename S::Mul>;
  using Out = Elem<T>;
  constexpr int kChunk = S::kLow && KEYS > 32 ? 32 : KEYS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t lanes = c.tmem + ((uint32_t)warp << 21);  // this warp's lanes of tensor memory
  const uint32_t out_at = lanes + S::kOut;
  const int copy = tid / S::kLanes, row = tid % S::kLanes, key0 = copy * KEYS;
  Turn turn;
  bool dead = false;
  auto wait = [&](unsigned long long* m, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(m, parity, P.spin_limit, 0u));
  };
  auto added = [&](uint32_t tile) {  // the output holds everything up to this tile
    wait(&c.pv_done[tile & 1], (tile >> 1) & 1);
    fence_after();
  };
  uint32_t it = 0;
  int sg = 0;
  bool more = true;
  while (more) {
    wait(&c.seg_full[sg & 1], (sg >> 1) & 1);
    dead = any_softmax(dead);  // all go on, or none: they meet at barriers
    const Segment g = c.seg[sg & 1];
    more = g.count > 0 && !dead;
    if (!more) break;
    const bool busy = warp * 32 % S::kLanes < g.live;  // the warp has live rows
    const bool live = row < g.live;
    const int f = g.mt * P.rows + row, token = token_of(P, f);
    const int p = live ? g.len - g.n + token : -1;
    float scale = P.scale_log2;
    if (S::kLow && P.k_scale) scale *= P.k_scale[g.h];
    if (S::kScaleQ && live) scale *= c.q_back[sg & 1][row];
    // A product of factors may vanish (a query of zeros comes with 2^-126), and -inf, the score of a hidden key, times 0 is
    // NaN.  Products of the held values are below 2^33, so with factors this small every score is 0 either way.
    if (S::kLow) scale = fmaxf(scale, FLT_MIN);
    if (S::kBlocks) scale = scale_of(scale);
    float mx = -INFINITY, l = 0.0f, exact = 0.0f;  // m, the sum that divides, the sum of the weights
    bool large = false;  // a row of the warp has an m beyond kLarge

    for (int i = 0; i < g.count; ++i, ++it) {
      const int b = it & 1;
      const int base = tile_of(g.u, g.from + i) * kTile;
      turn.next(P.slots);
      const Turn v_turn = turn;
      turn.next(P.slots);
      wait(&c.s_full[b], (it >> 1) & 1);
      fence_after();
      const int bad = c.bad[it & (kBadTiles - 1)];
      const bool cut = partly(P, g.u, base), part = cut || bad != 0;
      // as bits, the tile's keys that this thread's row sees
      const uint64_t seen = part ? visible_keys(P, base, p, bad) : ~0ull;
      unsigned char* values = ring + v_turn.slot * S::kSlot;
      if (busy) {
        // Where scores are read twice and have factors, hidden ones are overwritten first: with masks at every read the loops
        // below would not stay among the instructions at hand (64 query rows 113 us, so 88; 256 columns 110, so 84).
        constexpr bool kHideFirst = S::kBlocks && KEYS > kChunk;
        if (kHideFirst && part) {
#pragma unroll 1
          for (int at = 0; at < KEYS; at += 32) {
            uint32_t y[32];
            tmem_load(y, lanes + b * kTile + key0 + at);
            const uint32_t word = (uint32_t)(seen >> (key0 + at));
#pragma unroll
            for (int n = 0; n < 32; ++n)
              if (!(word >> n & 1)) y[n] = 0xff800000u;
            tmem_store(lanes + b * kTile + key0 + at, y);
          }
          store_wait();
        }
        // this thread's scores, kChunk at a time: one chunk where registers allow, else each is read once for the
        // maximum and once for its weights
        auto scores = [&](uint32_t (&x)[kChunk], int at) {
          tmem_load(x, lanes + b * kTile + key0 + at);
          if (part && !kHideFirst) {
#pragma unroll
            for (int n = 0; n < kChunk; ++n)
              if (!((uint32_t)(seen >> (key0 + at + (n & 32))) >> (n & 31) & 1)) x[n] = 0xff800000u;
          }
        };
        uint32_t x[kChunk];
        float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        // the factors of this thread's keys, by groups of 16; the loops are not unrolled for the same reason
        const int tile = it & (kBadTiles - 1), group0 = key0 >> 4;
        constexpr int kGroups = kChunk / 16;
        float top = -INFINITY;
        if constexpr (S::kBlocks) {
#pragma unroll 1
          for (int at = 0; at < KEYS; at += kChunk) {
            float by_k[kGroups], v[kGroups];
            read_factors(by_k, &factors->k[tile][group0 + (at >> 4)]);
            read_factors(v, &factors->v[tile][group0 + (at >> 4)]);
            scores(x, at);
#pragma unroll
            for (int g0 = 0; g0 < kChunk; g0 += 16) {
#pragma unroll
              for (int n = 0; n < 4; ++n)
                t[n] = fmaxf(fmaxf(__uint_as_float(x[g0 + n]), __uint_as_float(x[g0 + 4 + n])), fmaxf(__uint_as_float(x[g0 + 8 + n]), __uint_as_float(x[g0 + 12 + n])));
              top = fmaxf(top, __fadd_rn(__fmul_rn(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), factor_of(scale, by_k[g0 / 16])), log2_of(v[g0 / 16])));
            }
          }
        } else {
#pragma unroll
          for (int at = 0; at < KEYS; at += kChunk) {
            scores(x, at);
#pragma unroll
            for (int n = 0; n < kChunk; ++n) t[n & 3] = fmaxf(t[n & 3], __uint_as_float(x[n]));
          }
          top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale;
        }
        const bool grow = live && top - mx > 8.0f + E::kLift;
        if (__any_sync(0xffffffffu, grow)) {
          const float now = grow ? (fabsf(top) > kLarge ? top : top - E::kLift) : mx;
          const float by = grow ? ex2(mx - now) : 1.0f;  // 0 if nothing was seen before
          mx = now;
          large = __any_sync(0xffffffffu, mx != -INFINITY && fabsf(mx) > kLarge);
          l *= by;
          exact *= by;
          if (i > 0) {
            added(it - 1);
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              uint32_t o[32];
              tmem_load(o, out_at + d);
#pragma unroll
              for (int n = 0; n < 32; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * by);
              tmem_store(out_at + d, o);
            }
            store_wait();
          }
        }
        const float z = mx == -INFINITY ? 0.0f : mx;
        // Weights are rounded to 16 bits for the product (half a step, 2^-9 or 2^-12 of each, random in sign; f16 weights
        // below 2^-14, 2^-21 of the first tile's largest, by up to 2^-25).  To bf16 the divisor is the sum of the rounded
        // ones, so that the error of a weight that dominates its row cancels; the log-sum-exp has the sum before rounding.
        constexpr bool kTwo = std::is_same<typename S::Mul, __nv_bfloat16>::value;
        if (S::kBlocks && large) {
          const float sum = large_weights_blocks<S, KEYS>(lanes + b * kTile, key0, scale, z, seen, *factors, tile);
          l += sum;
          exact += sum;
        } else if (large) {
          const float2 sums = large_weights<S, KEYS>(lanes + b * kTile, key0, scale, z, seen);
          l += sums.x;
          exact += sums.y;
        }
        if constexpr (S::kBlocks) {
#pragma unroll 1
          for (int at = 0; at < KEYS && !large; at += kChunk) {
            float by_k[kGroups], v[kGroups];
            read_factors(by_k, &factors->k[tile][group0 + (at >> 4)]);
            read_factors(v, &factors->v[tile][group0 + (at >> 4)]);
            if (KEYS > kChunk) scores(x, at);
            uint32_t w[kChunk / 2];
#pragma unroll
            for (int g0 = 0; g0 < kChunk; g0 += 16) {
              const float by = factor_of(scale, by_k[g0 / 16]), less = log2_of(v[g0 / 16]) - z;
              float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
              for (int n = g0 / 2; n < g0 / 2 + 8; ++n) {
                const float a = ex2(fmaf(__uint_as_float(x[2 * n]), by, less)), e = ex2(fmaf(__uint_as_float(x[2 * n + 1]), by, less));
                w[n] = E::pack(a, e);
                s0 += a;
                s1 += e;
              }
              l = fmaf(s0 + s1, back_of(v[g0 / 16]), l);
            }
            tmem_store(lanes + b * kTile + (key0 + at) / 2, w);
          }
          exact = l;
        }
#pragma unroll
        for (int at = 0; at < (S::kBlocks ? 0 : KEYS) && !large; at += kChunk) {
          if (KEYS > kChunk) scores(x, at);
          uint32_t w[kChunk / 2];
          float s0 = 0.0f, s1 = 0.0f, e0 = 0.0f, e1 = 0.0f;
#pragma unroll
          for (int n = 0; n < kChunk / 2; ++n) {
            const float a = ex2(fmaf(__uint_as_float(x[2 * n]), scale, -z)), e = ex2(fmaf(__uint_as_float(x[2 * n + 1]), scale, -z));
            w[n] = E::pack(a, e);
            const float2 r = kTwo ? E::unpack(w[n]) : make_float2(a, e);
            s0 += r.x;
            s1 += r.y;
            if (kTwo) {
              e0 += a;
              e1 += e;
            }
          }
          l += s0 + s1;
          exact += kTwo ? e0 + e1 : s0 + s1;
          tmem_store(lanes + b * kTile + (key0 + at) / 2, w);
        }
        const uint32_t zeros[KEYS / 2] = {};
#pragma unroll
        for (int n = 1; n < S::kCopies; ++n) tmem_store(lanes + b * kTile + (copy + n) % S::kCopies * (KEYS / 2), zeros);
        store_wait();
      }
      bool slow = false;
      if (cut) {
        // Values of keys that no row sees must not reach the product (0 * infinity, and what was never written may be
        // anything): they become zeros, as those on unreadable pages are already (their copies read past the cache).
        // If a value that only some rows see is not finite, the tile goes the slow way.
        // (After the weights, which do not wait for the values.)
        wait(&c.full[v_turn.slot], v_turn.parity);
        const int in = tid >> 1, key = base + in;
        const bool some = key <= g.u.pos1 && (P.window <= 0 || key > max(0, g.u.pos0) - P.window || key < P.sinks);
        const bool all = key <= g.u.pos0 && (P.window <= 0 || key > g.u.pos1 - P.window || key < P.sinks);
        uint32_t wild = 0;  // bits 15 and 31: an exponent of ones, plus one, carries into the sign's place
        constexpr uint32_t kOnes = E::kExponent * 0x10001u, kOne = kOnes & ~(kOnes << 1);
#pragma unroll
        for (int r = 0; r < S::kRuns; ++r) {
          uint4* line = reinterpret_cast<uint4*>(values + r * S::kRun + in * 128) + (tid & 1) * 4;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (!some) {
              line[x] = make_uint4(0u, 0u, 0u, 0u);
            } else if (!all) {
              const uint4 y = line[x];
              for (const uint32_t w : {y.x, y.y, y.z, y.w}) wild |= (w & kOnes) + kOne;
            }
          }
        }
        proxy_fence();
        slow = any_softmax((wild & 0x80008000u) != 0);
        if (slow && busy) {
          // one key at a time, and only for the rows that see it
          if (i > 0) added(it - 1);
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t o[32];
            if (i > 0) tmem_load(o, out_at + d);
            float acc[32];
#pragma unroll
            for (int n = 0; n < 32; ++n) acc[n] = i > 0 ? __uint_as_float(o[n]) : 0.0f;
#pragma unroll 1
            for (int n = 0; n < kTile; ++n) {
              uint32_t pair[1];
              tmem_load(pair, lanes + b * kTile + (n >> 1));
              const float2 ws = E::unpack(pair[0]);
              const float wt = n & 1 ? ws.y : ws.x;
              const bool sees = (seen >> n & 1) && n / KEYS == copy;
              const unsigned char* line = values + (d >> 6) * S::kRun + n * 128;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint4 y = *reinterpret_cast<const uint4*>(line + ((((d >> 3) & 7) + q) ^ (n & 7)) * 16);
                const uint32_t ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                  const float2 v = E::unpack(ys[h]);
                  if (sees) {
                    acc[q * 8 + h * 2] = fmaf(wt, v.x, acc[q * 8 + h * 2]);
                    acc[q * 8 + h * 2 + 1] = fmaf(wt, v.y, acc[q * 8 + h * 2 + 1]);
                  }
                }
              }
            }
#pragma unroll
            for (int n = 0; n < 32; ++n) o[n] = __float_as_uint(acc[n]);
            tmem_store(out_at + d, o);
          }
          store_wait();
        }
      }
      if (tid == 0) c.slow[b] = slow;
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(&c.p_full[b]);
    }
    if (dead && lane == 0) atomicOr(&P.row_status[g.row], (uint32_t)SS_ST_COPY_TIMEOUT);

    // ---- the unit's output, or this CTA's piece of it
    added(it - 1);
    const bool whole = g.ca == g.cb;
    const float v_scale = S::kLow && P.v_scale ? P.v_scale[g.h] : 1.0f;
    const int mine = piece_of(g, blockIdx.x), head = g.h * P.group + f - token * P.group;
    auto write_sums = [&](float m, float sum, float weights) {  // of a live row
      if (!whole) piece_ml(P, mine)[row] = make_float4(m, sum, weights, 0.0f);
      else if (P.lse)
        P.lse[(size_t)(g.q0 + token) * (P.group * P.hkv) + head] = weights == 0.0f ? -INFINITY : (m + log2f(weights)) * 0.69314718055994531f;
    };
    if constexpr (S::kCopies == 1) {
      if (busy) {
        const float r = (whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f) * v_scale;
        T* to = static_cast<T*>(P.out) + (g.q0 + token) * P.out_stride + head * D;
        float4* part_to = piece_out<D>(P, mine) + row;
        constexpr int kCols = S::kLow ? 32 : 64;
#pragma unroll 1
        for (int d = 0; d < D; d += kCols) {
          uint32_t o[kCols];
          tmem_load(o, out_at + d);
          auto val = [&](int n) { return __uint_as_float(o[n]); };
          if (!live) continue;
          if (whole) {
#pragma unroll
            for (int n = 0; n < kCols; n += 8)
              *reinterpret_cast<uint4*>(to + d + n) =
                  make_uint4(Out::pack(val(n) * r, val(n + 1) * r), Out::pack(val(n + 2) * r, val(n + 3) * r),
                             Out::pack(val(n + 4) * r, val(n + 5) * r), Out::pack(val(n + 6) * r, val(n + 7) * r));
          } else {
#pragma unroll
            for (int n = 0; n < kCols; n += 4)
              part_to[(size_t)((d + n) >> 2) * P.rows] = make_float4(val(n) * r, val(n + 1) * r, val(n + 2) * r, val(n + 3) * r);
          }
        }
        if (live) write_sums(mx, l, exact);
      }
    } else {
      // the copies' outputs are added by way of the segment's query buffer, whose products are done: 32 columns of
      // 128 lanes at a time, every thread then adding four columns of a row
      static_assert(128 * D * 2 >= 128 * 32 * 4, "room for 32 columns");
      float4* room = reinterpret_cast<float4*>(sq + (P.q_bufs == 2 && (sg & 1) ? 128 * D * 2 : 0));
      c.ml[tid] = make_float4(mx, l, exact, 0.0f);
      bar_softmax();
      float top = -INFINITY, sum = 0.0f, weights = 0.0f;
#pragma unroll
      for (int n = 0; n < S::kCopies; ++n) top = fmaxf(top, c.ml[row + n * S::kLanes].x);
      const float zero = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int n = 0; n < S::kCopies; ++n) {
        const float4 its = c.ml[row + n * S::kLanes];
        const float share = ex2(its.x - zero);
        sum += its.y * share;
        weights += its.z * share;
      }
      const float by = ex2(mx - zero) * (whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f) * v_scale;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        if (busy) {
          uint32_t o[32];
          tmem_load(o, out_at + d);
          auto val = [&](int n) { return __uint_as_float(o[n]) * by; };
          if (live) {
#pragma unroll
            for (int n = 0; n < 32; n += 4) room[(n >> 2) * 128 + tid] = make_float4(val(n), val(n + 1), val(n + 2), val(n + 3));
          }
        }
        bar_softmax();
        if (live) {
          for (int n = copy; n < 8; n += S::kCopies) {
            float4 y = room[n * 128 + row];
#pragma unroll
            for (int x = 1; x < S::kCopies; ++x) {
              const float4 z = room[n * 128 + row + x * S::kLanes];
              y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
            }
            if (whole)
              *reinterpret_cast<uint2*>(static_cast<T*>(P.out) + (g.q0 + token) * P.out_stride + head * D + d + n * 4) =
                  make_uint2(Out::pack(y.x, y.y), Out::pack(y.z, y.w));
            else
              piece_out<D>(P, mine)[(size_t)((d >> 2) + n) * P.rows + row] = y;
          }
        }
        bar_softmax();
      }
      if (live && copy == 0) write_sums(top, sum, weights);
    }
    fence_before();
    __syncwarp();
    if (lane == 0) {
      arrive(&c.o_free);
      arrive(&c.seg_empty[sg & 1]);
    }
    ++sg;
    if (!whole) join_unit<T, Out, D, 32 * kSoftmaxWarps>(P, g, &c.last, bar_softmax);
  }
  if (dead && tid == 0) report_range(P, &c.range);
}

// ------------------------------------------------------------------ kernel
template <class T, int D, int KEYS, bool LOW, bool BLOCKS>
__global__ void __launch_bounds__((Shape<T, D, KEYS, LOW, BLOCKS>::kThreads), (Shape<T, D, KEYS, LOW, BLOCKS>::kCtas))
    attend_kernel(const AttendParams P, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = Shape<T, D, KEYS, LOW, BLOCKS>;
  extern __shared__ unsigned char raw[];
  __shared__ Control c;
  TileFactors* factors = nullptr;
  if constexpr (BLOCKS) {
    __shared__ TileFactors f;
    factors = &f;
  }
  // query buffers first: products read 128 rows from each of their runs, into the ring where fewer are live
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  unsigned char* ring = base + P.q_bufs * q_rows<S>(P) * D * 2;
  unsigned char* raw_ring = ring + P.slots * S::kSlot;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    if (LOW) {
      for (int i = 0; i < P.raw_slots; ++i) {
        mbar_init_n(&c.raw_full[i], 1);
        mbar_init_n(&c.raw_empty[i], 4);
      }
    }
    for (int i = 0; i < P.slots; ++i) {
      mbar_init_n(&c.full[i], LOW ? 4 : 1);
      mbar_init_n(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_n(&c.seg_full[i], 1);
      mbar_init_n(&c.seg_empty[i], kSoftmaxWarps + 1 + (LOW ? 4 : 0));
      mbar_init_n(&c.s_full[i], 1);
      mbar_init_n(&c.p_full[i], kSoftmaxWarps);
      mbar_init_n(&c.pv_done[i], 1);
      c.slow[i] = 0;
    }
    mbar_init_n(&c.o_free, kSoftmaxWarps);
    mbar_init_n(&c.q_free, 1);
    mbar_init_n(&c.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c.tmem)), "r"(S::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == kLoadWarp && lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &mv : &mk) : "memory");
  fence_before();
  find_range<S::kThreads, kProductWarp>(P, c.sums, &c.range);  // ends in a barrier
  fence_after();
  if (c.range.cut.ctas == 0) {
    // no work: straight to the end
  } else if (warp < kSoftmaxWarps) {
    softmax_warps<S, T, D, KEYS>(P, base, ring, c, factors);
  } else if (warp == kLoadWarp) {
    load_warp<S, T, D>(P, &mk, &mv, smem_u32(base), smem_u32(ring), smem_u32(raw_ring), c, factors);
  } else if (warp == kProductWarp) {
    if (lane == 0) product_thread<S, T, D>(P, smem_u32(base), smem_u32(ring), c);
    __syncwarp();
  } else if constexpr (LOW) {
    convert_warps<S, D>(P, raw_ring, ring, c);
  }
  fence_before();
  __syncthreads();
  if (warp == kProductWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(c.tmem), "r"(S::kCols) : "memory");
  }
}

// The kernel for `rows` query rows of a unit, its rings and shared memory.
template <class T, int D, int KEYS, bool LOW, bool BLOCKS>
AttendKernel entry(int rows) {
  using S = Shape<T, D, KEYS, LOW, BLOCKS>;
  const int share = (228 * 1024 / S::kCtas - 1024 - kControl - (BLOCKS ? 1024 : 0) - 1024) & ~1023;  // a CTA's, without the control block
  AttendKernel k;
  k.fn = reinterpret_cast<const void*>(&attend_kernel<T, D, KEYS, LOW, BLOCKS>);
  k.threads = S::kThreads;
  k.ctas = S::kCtas;
  k.tile = kTile;
  k.swizzled = !LOW;
  // What starting and ending a unit takes beside its tiles, about 2 us, in tiles.  Measured (us): 16 bits, 64 x 1 rows of
  // 128 columns with 1, 2, 4: 101, 95.7, 96.3; 96 x 3 rows of 64 columns: 89, 82, 76; 8 bits, 32 x 8 rows of 128
  // columns with 2, 4, 8: 135, 112, 96; 64 x 8 rows of 64 columns with 4, 8, 16: 58, 61, 67.
  k.unit_cost = LOW ? (D == 128 ? 8 : 4) : 256 / D;
  // a second buffer hides the gathering of the next segment's queries; 128 rows of 128 columns leave no room for it, and
  // with 8 bits the rings need it more (16 x 16 rows x 4 query heads of 128 columns: 101 us with it, 98 without)
  const int q_rows = S::kCopies > 1 ? 128 : rows;
  k.q_bufs = q_rows * D <= 64 * 128 && !(LOW && D == 128) ? 2 : 1;
  const int q = k.q_bufs * q_rows * D * 2;
  // the loads fill the ring of products, or (8 bits) that of the copies, which has at least three places
  const int room = share - 1024 - q;
  k.slots = std::min((room - (LOW ? 3 * S::kRaw : 0)) / S::kSlot, kMaxSlots);
  k.raw_slots = LOW ? std::min((room - k.slots * S::kSlot) / S::kRaw, kMaxRaw) : 0;
  k.smem = 1024 + (size_t)q + (size_t)k.slots * S::kSlot + (size_t)k.raw_slots * S::kRaw;
  return k;
}
// With 64 columns few query rows are copied (see above); so are at most 32 of 128 columns in 8 bits, where the softmax
// shares its issue slots with the conversion (32 x 4 rows x 8 query heads: 84 us without copies, 76 with four; 64 rows
// with two: no gain, 98 us; in 16 bits the larger query buffer costs the ring more: 64 x 1 90 -> 103 us).
template <class T, bool LOW, bool BLOCKS = false>
AttendKernel pick(int d, int rows) {
  if (d == 64)
    return rows <= 32    ? entry<T, 64, 16, LOW, BLOCKS>(rows)
           : rows == 64 ? entry<T, 64, 32, LOW, BLOCKS>(rows)
                        : entry<T, 64, kTile, LOW, BLOCKS>(rows);
  if (LOW && d == 128 && rows <= 32) return entry<T, 128, LOW ? 16 : kTile, LOW, BLOCKS>(rows);
  return d == 128 ? entry<T, 128, kTile, LOW, BLOCKS>(rows) : entry<T, 256, kTile, LOW, BLOCKS>(rows);
}

}  // namespace kv
}  // namespace ss
