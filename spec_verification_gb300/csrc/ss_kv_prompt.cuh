// ss_attend_prompt: causal attention of packed prompts over themselves, on the
// 5th-generation tensor cores.
//
// Mathematics.  As in ss_kv_attend.cuh: one pass over the keys that a query
// sees, o = sum_t w_t v_t / sum_t w_t with w_t = 2^(c q.k_t - m), where m is
// near the row's largest exponent and moves only when a weight would pass 2^8.
//
// What bounds it.  4 * head_dim operations for each pair of query and key: at
// prompts of some thousand tokens the tensor pipe, at 128 columns and more also
// the power it may draw.  128 query rows and 64 keys of 128 columns take the
// pipe 640 cycles for S = Q K^T (of which 64 keys use two thirds of it: the
// queries are read from shared memory for so few) and O += P V, the 128 threads
// that weigh them about 1300, so two tiles of rows, or two CTAs, share an SM.
// With 64 columns the weighing is the bound.  Measured (one prompt, causal):
// 16000 tokens of 32/8 heads of 128 1333 us, 1.57 PFLOP/s, called again and
// again, 1190 us, 1.76, in bursts of a few (the library's matrix product: 1.74
// and 1.93); in bursts 28/4 heads of 64 956 us, 0.96; 16/8 of 256 1440 us, 1.46.
//
// Query rows.  The heads that share a key head lie next to each other in a
// tile: `heads` of them for each of `tokens` tokens (heads * tokens <= 128), so
// short prompts fill tiles and keys are loaded once for all.  A unit is
// (prompt, key head, part of its query heads, TILES tiles of tokens) over the
// keys from the first that its first token sees to its last token.  Units are
// handed out by a counter, those of a prompt from its end (the longest) on.
//
// A CTA's warps:
//  - load: takes units, publishes them, runs the ring of key and value tiles
//    (TMA) and brings their queries (TMA; a box of heads by tokens).
//  - scores and values: two warps for each tile of rows issue tcgen05.mma, one
//    the scores, two tiles of keys ahead, one the products with the values.  A
//    warp's waits and issuing take about as long as its products, so they have
//    to overlap: with one warp for all 16000 tokens took 1977 us, with one for
//    each tile of rows 1898, with the four 1372.
//  - softmax: four warps to a tile of rows; a thread owns a row (a lane of
//    tensor memory), reads its scores, writes its weights over them.  Nothing
//    of its loop may be spilled: the 28 KB that the SM has left beside its
//    shared memory hold no stack of 448 threads (1434 us with 100 bytes, 1218
//    without).
//  - guard: a warp looks at every tile of values before the products do.  In
//    one that not every row sees in full, values that no row sees become zeros
//    (0 x NaN must not reach a sum), and if one that only some rows see is not
//    finite, the tile is added key by key by the softmax warps.
// Tensor memory: two buffers of scores of 64 keys for each tile of rows, so that
// the next tile's scores are there when one has been weighed, then outputs.
// 256 columns of output leave room for one tile of rows, and between the two
// for its queries: the softmax warps bring them there as soon as the last
// scores of the unit before are taken, the next unit's queries come meanwhile,
// and outputs leave by way of the room they came to.  (With 128 keys to a tile
// and queries in shared memory, 5 x 9000 tokens with a window of 1024 took 338
// us, so 307; 200 x 60 70, so 60; one prompt of 16000 1395, so 1436: there the
// one tile's softmax is the bound, and it costs less for 128 keys at a time.)
//
// The divisor is the sum of the weights before they are rounded for the
// product.  That of the rounded bf16 weights, as in ss_kv_attend.cuh, costs 10
// to 18 % of the time here and brings the error from 1.31 to 1.26 of that of
// the output's own rounding.
#pragma once

#include <algorithm>

#include "ss_kv_attend.cuh"

namespace ss {
namespace kv {
namespace prompt {

constexpr int kMaxSlots = 16;
constexpr int kGuardWarps = 1;

template <class T_, int D_, int TILES_>
struct Shape {
  using T = T_;
  static constexpr int D = D_, TILES = TILES_;
  static constexpr int kSoftmax = 4 * TILES;                  // warps
  static constexpr int kProducts = 2 * TILES;
  static constexpr int kLoad = kSoftmax, kProduct = kSoftmax + 1, kGuard = kProduct + kProducts;
  static constexpr int kThreads = 32 * (kGuard + kGuardWarps);
  static constexpr int kKeys = 64;                            // keys of a tile
  static constexpr bool kQTensor = D == 256;                  // queries in tensor memory
  static constexpr int kCtas = TILES == 1 && D <= 128 ? 2 : 1;  // CTAs per SM
  static constexpr int kWide = D < 128 ? D : 128;             // columns of a slot
  static constexpr int kHalves = D / kWide;                   // slots of a tile
  static constexpr int kRun = kKeys * 128, kQRun = 128 * 128; // bytes of 64 columns of a tile, of a tile of rows
  static constexpr int kSlot = kWide / 64 * kRun;
  static constexpr int kQ = D / 64 * kQRun;                   // bytes of the queries of a tile of rows
  static constexpr int kQAt = 2 * TILES * kKeys;              // first column of the queries in tensor memory
  static constexpr int kOut = kQAt + (kQTensor ? D / 2 : 0);  // and of the outputs
  static constexpr uint32_t kCols = 512 / kCtas;
  // Outputs on their way out: 64 columns of a softmax warp's 32 rows.  Only where stores from registers are what the end of
  // a unit waits for (64 KB of rows at about 16 bytes a cycle: 4000 cycles of two tiles of 128 columns) and there is room.
  static constexpr int kStage = TILES == 2 ? 32 * 128 : 0;
  // slots: as many as there is room for beside the queries, outputs and the control block
  static constexpr int kFit = (228 * 1024 / kCtas - 1024 - 1024 - 2048 - TILES * kQ - kSoftmax * kStage) / kSlot;
  static constexpr int kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
  static constexpr int kSmem = 1024 + TILES * kQ + kSlots * kSlot + kSoftmax * kStage;
  static constexpr uint32_t kCommon = 1u << 4 | Elem<T>::kFormat << 7 | Elem<T>::kFormat << 10 | (128u >> 4) << 24;
  static constexpr uint32_t kScores = kCommon | (kKeys >> 3) << 17;
  static constexpr uint32_t kValues = kCommon | 1u << 16 | (uint32_t)(kWide >> 3) << 17;
  static_assert(kSlots >= 2 * kHalves + 1, "ring length");
  static_assert(kOut + TILES * D <= (int)kCols, "tensor memory");
};

struct Unit {
  int row, q0, n;            // prompt, its first token and their number
  int t0, h, chunk;          // first token of the unit in its prompt, key head, part of the query heads
  int sink, first, tiles;    // key tiles: `sink` from 0, then from `first` on; 0 tiles: the end
  int live;                  // tiles of rows that have tokens
  int of_first;              // key tiles of the first tile of rows (the last one has all)
  int pos1;                  // last token of the unit
  int cut, edge0, edge1;     // key tiles that not every row sees in full: from `cut` on, and edge0 .. edge1 - 1
};
template <class S>
__device__ __forceinline__ int base_of(const Unit& u, int i) {
  return (i < u.sink ? i : i - u.sink + u.first) * S::kKeys;
}
__device__ __forceinline__ int tiles_of(const Unit& u, int r) { return r + 1 < u.live ? u.of_first : r < u.live ? u.tiles : 0; }
__device__ __forceinline__ bool cuts(const Unit& u, int i) { return i >= u.cut || (i >= u.edge0 && i < u.edge1); }

struct Control {
  unsigned long long full[kMaxSlots], empty[kMaxSlots];  // copies landed; products done
  // Values looked at, by their number in the CTA's run of slots of values (not by their place in the ring, which may have
  // held keys before): number n + kMaxSlots is copied only when number n has been multiplied.
  unsigned long long ready[kMaxSlots];
  unsigned long long seg_full[2], seg_empty[2];
  unsigned long long q_full[2], q_free[2], q_ready;
  unsigned long long s_full[4], p_full[4], pv_done[4];  // by buffer: scores there; weights there; added to the output
  unsigned long long o_free[2];
  unsigned long long drained;
  Unit unit[2];
  int slow[kMaxSlots][kGuardWarps];
  uint32_t tmem;
};
static_assert(sizeof(Control) <= 1024, "control block");

// ------------------------------------------------------------------ units
// Walks the prompts with a warp: where unit `u` (in order) is.
struct Cursor {
  int row = 0;           // first of the 32 prompts looked at
  long long before = 0;  // units before it
  // false: past the last one
  template <class S>
  __device__ __forceinline__ bool find(const PromptParams& P, long long u, Unit& g) {
    const int lane = threadIdx.x & 31, per = S::TILES * P.tokens, kinds = P.hkv * P.chunks;
    for (; row < P.B; row += 32) {
      int q0 = 0, n = 0;
      if (row + lane < P.B) {
        q0 = P.cu[row + lane];
        const int q1 = P.cu[row + lane + 1];
        n = q0 < 0 || q1 < q0 || q1 > P.max_tokens ? 0 : q1 - q0;
      }
      const long long mine = (long long)((n + per - 1) / per) * kinds;
      long long incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + incl > u);
      if (past) {
        const int at = __ffs(past) - 1;
        const long long idx = u - before - __shfl_sync(0xffffffffu, incl - mine, at);
        g.row = row + at;
        g.q0 = __shfl_sync(0xffffffffu, q0, at);
        g.n = __shfl_sync(0xffffffffu, n, at);
        const int tile = (g.n + per - 1) / per - 1 - (int)(idx / kinds), kind = (int)(idx % kinds);
        g.t0 = tile * per;
        g.h = kind / P.chunks;
        g.chunk = kind % P.chunks;
        g.pos1 = min(g.n, g.t0 + per) - 1;
        g.live = (g.pos1 - g.t0) / P.tokens + 1;
        g.first = P.window > 0 ? max(0, g.t0 - P.window + 1) / S::kKeys : 0;
        g.sink = P.window > 0 ? min((P.sinks + S::kKeys - 1) / S::kKeys, g.first) : 0;
        g.tiles = g.sink + g.pos1 / S::kKeys - g.first + 1;
        g.of_first = g.sink + min(g.pos1, g.t0 + P.tokens - 1) / S::kKeys - g.first + 1;
        // the diagonal: tiles that end past the first token; the window's edge: those that start before the last token's
        // window does, unless they are of sinks alone
        const int shift = g.sink - g.first;
        g.cut = (g.t0 + 1) / S::kKeys + shift;
        g.edge0 = g.edge1 = 0;
        if (P.window > 0 && g.pos1 >= P.window) {
          const int all = P.sinks / S::kKeys;
          g.edge0 = all <= g.sink ? all : all + shift;
          g.edge1 = (g.pos1 - P.window) / S::kKeys + shift + 1;
        }
        return true;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }
};

// A wait ran out (not expected): which rows it concerns is not known here, so all report it.
static __device__ __noinline__ void report_all(const PromptParams& P) {
  for (int r = threadIdx.x & 31; r < P.B; r += 32) atomicOr(&P.row_status[r], (uint32_t)SS_ST_COPY_TIMEOUT);
}

// ------------------------------------------------------------------ load warp
template <class S>
__device__ void load_warp(const PromptParams& P, const CUtensorMap* mq, const CUtensorMap* mk, const CUtensorMap* mv, uint32_t sq, uint32_t ring,
                          Control& c) {
  const int lane = threadIdx.x & 31;
  Turn turn;
  int asked = 0;
  uint32_t q_units[2] = {0, 0};  // query tiles brought, by tile of rows
  bool dead = false;
  auto wait = [&](unsigned long long* m, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(m, parity, P.spin_limit, 0u));
  };
  Cursor cursor;
  Unit g;
  long long u = blockIdx.x;
  int sg = 0;
  bool more = true;
  while (more && !dead) {
    more = cursor.template find<S>(P, u, g);
    if (sg >= 2) wait(&c.seg_empty[sg & 1], ((sg >> 1) & 1) ^ 1);
    if (dead) break;
    if (!more) g.tiles = g.live = 0;
    if (lane == 0) {
      c.unit[sg & 1] = g;
      arrive(&c.seg_full[sg & 1]);
    }
    __syncwarp();
    if (!more) break;
    unsigned long long next = 0;
    if (lane == 0) next = atomicAdd(P.next, 1ull);  // looked at after this unit's loads
    auto slot = [&](bool values, int i, int half) {
      wait(&c.empty[turn.slot], turn.parity ^ 1);
      if (dead) return;
      if (lane == 0) {
        expect(&c.full[turn.slot], S::kSlot);
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                ring + turn.slot * S::kSlot),
            "l"(values ? mv : mk), "r"(0), "r"(g.q0 + base_of<S>(g, i)), "r"(half * (S::kWide / 64)), "r"(g.h), "r"(smem_u32(&c.full[turn.slot]))
            : "memory");
      }
      __syncwarp();
      turn.next(S::kSlots);
      asked = min(asked + 1, S::kSlots);
    };
    for (int i = 0; i < g.tiles && !dead; ++i) {
      for (int half = 0; half < S::kHalves; ++half) slot(false, i, half);
      if (i == 0) {
#pragma unroll
        for (int r = 0; r < S::TILES; ++r) {
          if (r >= g.live || dead) continue;
          if (q_units[r] > 0) wait(&c.q_free[r], (q_units[r] - 1) & 1);
          if (dead) continue;
          ++q_units[r];
          if (lane == 0) {
            expect(&c.q_full[r], P.heads * P.tokens * S::D * 2);
            for (int run = 0; run < S::D / 64; ++run)
              asm volatile(
                  "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                      sq + r * S::kQ + run * S::kQRun),
                  "l"(mq), "r"(run * 64), "r"(g.h * P.group + g.chunk * P.heads), "r"(g.q0 + g.t0 + r * P.tokens), "r"(smem_u32(&c.q_full[r]))
                  : "memory");
          }
          __syncwarp();
        }
      }
      for (int half = 0; half < S::kHalves; ++half) slot(true, i, half);
    }
    u = (long long)gridDim.x + (long long)__shfl_sync(0xffffffffu, next, 0);
    ++sg;
  }
  // no copy may be in flight when the CTA ends (all have landed unless a wait ran out)
  for (; asked > 0; --asked) {
    if (--turn.slot < 0) {
      turn.slot = S::kSlots - 1;
      turn.parity ^= 1;
    }
    mbar_wait(&c.full[turn.slot], turn.parity, kDrainPolls, 0u);
  }
#pragma unroll
  for (int r = 0; r < S::TILES; ++r)
    if (q_units[r] > 0) mbar_wait(&c.q_full[r], (q_units[r] - 1) & 1, kDrainPolls, 0u);
  if (dead) report_all(P);
}

// ------------------------------------------------------------------ guard warps
template <class T>
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t sum) {
  uint32_t y;
  if (std::is_same<T, __half>::value) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0u), "r"(sum));
  else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0u), "r"(sum));
  return y;
}

template <class S>
__device__ void guard_warps(const PromptParams& P, unsigned char* ring, Control& c) {
  const int tid = threadIdx.x - 32 * S::kGuard, lane = tid & 31;
  // prompts whose prefix sums are no good: each CTA looks at its share
  for (int r = blockIdx.x * 32 * kGuardWarps + tid; r < P.B; r += gridDim.x * 32 * kGuardWarps) {
    const int q0 = P.cu[r], q1 = P.cu[r + 1];
    if (q0 < 0 || q1 < q0 || q1 > P.max_tokens) atomicOr(&P.row_status[r], (uint32_t)SS_ST_CAPACITY);
  }
  Turn turn;
  uint32_t nth = 0;  // slots of values so far
  bool dead = false;
  auto wait = [&](unsigned long long* m, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(m, parity, P.spin_limit, 0u));
  };
  bool more = true;
  for (int sg = 0; more; ++sg) {
    wait(&c.seg_full[sg & 1], (sg >> 1) & 1);
    if (dead) break;
    const Unit u = c.unit[sg & 1];
    more = u.tiles > 0;
    for (int i = 0; i < u.tiles && !dead; ++i) {
      for (int half = 0; half < S::kHalves; ++half) turn.next(S::kSlots);  // the keys
      const int base = base_of<S>(u, i);
      const bool cut = cuts(u, i);
      for (int half = 0; half < S::kHalves; ++half, ++nth) {
        wait(&c.full[turn.slot], turn.parity);
        if (dead) break;
        if (cut) {
          uint32_t wild = 0;  // x * 0 is 0, or NaN if x is not finite: two values an operation
          for (int in = tid; in < S::kKeys; in += 32 * kGuardWarps) {
            const int key = base + in;
            const bool some = key <= u.pos1 && (P.window <= 0 || key > u.t0 - P.window || key < P.sinks);
            const bool all = key <= u.t0 && (P.window <= 0 || key > u.pos1 - P.window || key < P.sinks);
            if (all) continue;
#pragma unroll
            for (int run = 0; run < S::kWide / 64; ++run) {
              uint4* line = reinterpret_cast<uint4*>(ring + turn.slot * S::kSlot + run * S::kRun + in * 128);
#pragma unroll
              for (int x = 0; x < 8; ++x) {  // (neighbouring lines in another order: other banks)
                if (!some) {
                  line[(x + tid) & 7] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                  const uint4 y = line[(x + tid) & 7];
                  for (const uint32_t w : {y.x, y.y, y.z, y.w}) wild = times_zero<typename S::T>(w, wild);
                }
              }
            }
          }
          const bool slow = __any_sync(0xffffffffu, (wild & 0x7fff7fffu) != 0);
          if (lane == 0) c.slow[nth % kMaxSlots][tid >> 5] = slow;
          proxy_fence();
        } else if (lane == 0) {
          c.slow[nth % kMaxSlots][tid >> 5] = 0;
        }
        __syncwarp();
        if (lane == 0) arrive(&c.ready[nth % kMaxSlots]);
        turn.next(S::kSlots);
      }
    }
    if (lane == 0) arrive(&c.seg_empty[sg & 1]);
  }
  if (dead) report_all(P);
}

// Is the tile with slots of values from number n on one to be added key by key?
template <class S>
__device__ __forceinline__ bool is_slow(const Control& c, uint32_t n) {
  int any = 0;
#pragma unroll
  for (int half = 0; half < S::kHalves; ++half) {
#pragma unroll
    for (int w = 0; w < kGuardWarps; ++w) any |= c.slow[(n + half) % kMaxSlots][w];
  }
  return any != 0;
}
__device__ __forceinline__ uint32_t parity_of(uint32_t n) { return (n / kMaxSlots) & 1; }

// ------------------------------------------------------------------ product warps
// All lanes go through them together and hold the same numbers, which the reductions below tell the compiler, and one of
// them is elected to issue: with operands in uniform registers a product takes some tens of cycles to issue, where a
// thread that is alone from the start takes about a hundred.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }
__device__ __forceinline__ bool elected() {  // always the same lane
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x != 0;
}

// D (+)= A B^T from shared memory, D (+)= A B with A from tensor memory.  Operands as in operand(), of which only the low
// halves differ from one product to the next.
constexpr uint32_t kOperandHigh = (uint32_t)(1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t operand_low(uint32_t at, uint32_t lead) { return (at & 0x3ffffu) >> 4 | (lead >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"(kOperandHigh), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"(kOperandHigh), "r"((uint32_t)add)
      : "memory");
}

// What the product warps have in common: their waits, and the slots that they go through.
template <class S>
struct Issuer {
  const PromptParams& P;
  Control& c;
  bool dead = false;
  Turn turn;  // of the next slot
  __device__ __forceinline__ Issuer(const PromptParams& P_, Control& c_) : P(P_), c(c_) {}
  __device__ __forceinline__ void wait(unsigned long long* m, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(m, parity, P.spin_limit, 0u));
  }
  // Looks at two barriers overlap; one after the other they take twice the time even if both phases are done.
  __device__ __forceinline__ void wait(unsigned long long* m, uint32_t m_parity, unsigned long long* n, uint32_t n_parity) {
    const bool first = done(m, m_parity), second = done(n, n_parity);
    if (!__all_sync(0xffffffffu, first)) wait(m, m_parity);
    if (!__all_sync(0xffffffffu, second)) wait(n, n_parity);
  }
  // A tile that this warp has no use for: the release by the other tile of rows' warp is not to stand for both.
  __device__ __forceinline__ void pass() {
    Turn t = turn;
#pragma unroll
    for (int half = 0; half < S::kHalves; ++half) {
      wait(&c.full[t.slot], t.parity);
      if (!dead && elected()) arrive(&c.empty[t.slot]);
      __syncwarp();
      t.next(S::kSlots);
    }
  }
  __device__ __forceinline__ void skip() {  // to the next tile of the same kind
#pragma unroll
    for (int n = 0; n < 2 * S::kHalves; ++n) turn.next(S::kSlots);
  }
  // The next unit: its tiles, and those of tile of rows r; false at the end.
  __device__ __forceinline__ bool next(int sg, int r, Unit& u, int& n) {
    wait(&c.seg_full[sg & 1], (sg >> 1) & 1);
    if (dead) return false;
    u = c.unit[sg & 1];
    n = uniform(tiles_of(u, r));
    u.tiles = uniform(u.tiles);
    return u.tiles > 0;
  }
  __device__ __forceinline__ void end(int sg) {
    __syncwarp();
    if (!dead && elected()) arrive(&c.seg_empty[sg & 1]);
    __syncwarp();
  }
  // nothing may be in flight when tensor memory is given back
  __device__ __forceinline__ void drain() {
    if (elected()) commit(&c.drained);
    __syncwarp();
    mbar_wait(&c.drained, 0, kDrainPolls, 0u);
  }
};

// S = Q K^T of tile of rows r, two tiles of keys ahead of the products with the values.  (A warp for each of the two kinds
// of products and each tile of rows: what they wait for and the time it takes to issue overlap the others' products.)
template <class S>
__device__ void scores_warp(const PromptParams& P, int r, uint32_t sq, uint32_t ring, Control& c) {
  Issuer<S> w(P, c);
  const uint32_t tmem = uniform(c.tmem + 2 * r * S::kKeys), q = uniform(S::kQTensor ? c.tmem + S::kQAt : operand_low(sq + r * S::kQ, 0));
  uint32_t it = 0, q_units = 0;  // tiles scored, units begun
  Unit u;
  int n;
#pragma unroll 1
  for (int sg = 0; w.next(sg, r, u, n); ++sg) {
    if (n > 0) w.wait(S::kQTensor ? &c.q_ready : &c.q_full[r], q_units++ & 1);
#pragma unroll 1
    for (int i = 0; i < u.tiles && !w.dead; ++i) {
      if (i < n) {
        const uint32_t b = it & 1;
        unsigned long long* const there = &c.s_full[2 * r + b];
        const uint32_t d = tmem + b * S::kKeys;
        Turn t = w.turn;
#pragma unroll
        for (int half = 0; half < S::kHalves; ++half) {
          // the keys, and the weights of two tiles ago, which are in the same columns
          if (half == 0) w.wait(&c.full[t.slot], t.parity, &c.pv_done[2 * r + b], ((it >> 1) & 1) ^ 1);
          else w.wait(&c.full[t.slot], t.parity);
          if (w.dead) break;
          fence_after();
          const uint32_t k = operand_low(ring + t.slot * S::kSlot, 0);
          if (elected()) {
#pragma unroll
            for (int x = 0; x < S::kWide / 16; ++x) {
              const uint32_t run = x >> 2, in = (x & 3) * 32 >> 4;
              if (S::kQTensor) mma_ts(d, q + half * (S::kWide / 2) + x * 8, k + run * (S::kRun >> 4) + in, S::kScores, half + x != 0);
              else mma_ss(d, q + (half * (S::kWide / 64) + run) * (S::kQRun >> 4) + in, k + run * (S::kRun >> 4) + in, S::kScores, half + x != 0);
            }
            if (half + 1 == S::kHalves) commit(there);
            commit(&c.empty[t.slot]);
            if (!S::kQTensor && half + 1 == S::kHalves && i + 1 == n) commit(&c.q_free[r]);
          }
          __syncwarp();
          t.next(S::kSlots);
        }
        ++it;
      } else {
        w.pass();
      }
      w.skip();
    }
    w.end(sg);
  }
  w.drain();
}

// O += P V of tile of rows r.
template <class S>
__device__ void values_warp(const PromptParams& P, int r, uint32_t ring, Control& c) {
  Issuer<S> w(P, c);
  for (int half = 0; half < S::kHalves; ++half) w.turn.next(S::kSlots);
  const uint32_t tmem = uniform(c.tmem + 2 * r * S::kKeys), o = uniform(c.tmem + S::kOut + r * S::D);
  uint32_t it = 0, o_units = 0, nth = 0;  // tiles multiplied, units begun, slots of values passed
  Unit u;
  int n;
#pragma unroll 1
  for (int sg = 0; w.next(sg, r, u, n); ++sg) {
    if (n > 0) w.wait(&c.o_free[r], (o_units++ & 1) ^ 1);
#pragma unroll 1
    for (int i = 0; i < u.tiles && !w.dead; ++i, nth += S::kHalves) {
      if (i < n) {
        const uint32_t b = it & 1;
        const bool cut = cuts(u, i);
        unsigned long long* const added = &c.pv_done[2 * r + b];
        const uint32_t weights = tmem + b * S::kKeys;
        const bool more = i != 0;
        Turn t = w.turn;
        bool slow = false;
#pragma unroll
        for (int half = 0; half < S::kHalves; ++half) {
          // Every slot is waited for by way of the guard, whether it had to look at it or not: a place in the ring is then
          // never brought anew before the guard has passed it.
          const uint32_t number = nth + half;
          const bool looked = done(&c.ready[number % kMaxSlots], parity_of(number));
          if (half == 0) w.wait(&c.full[t.slot], t.parity, &c.p_full[2 * r + b], (it >> 1) & 1);
          else w.wait(&c.full[t.slot], t.parity);
          if (!__all_sync(0xffffffffu, looked)) w.wait(&c.ready[number % kMaxSlots], parity_of(number));
          if (cut && half == 0) {
            if (S::kHalves == 2) w.wait(&c.ready[(number + 1) % kMaxSlots], parity_of(number + 1));
            slow = uniform(is_slow<S>(c, nth));
          }
          if (w.dead) break;
          fence_after();
          const uint32_t v = operand_low(ring + t.slot * S::kSlot, S::kRun);
          if (elected()) {
            if (!slow) {
#pragma unroll
              for (int k = 0; k < S::kKeys / 16; ++k)
                mma_ts(o + half * S::kWide, weights + k * 8, v + k * (2048 >> 4), S::kValues, more || k != 0);
            }
            if (half + 1 == S::kHalves) commit(added);
            commit(&c.empty[t.slot]);
          }
          __syncwarp();
          t.next(S::kSlots);
        }
        ++it;
      } else {
        w.pass();
      }
      w.skip();
    }
    w.end(sg);
  }
  w.drain();
}

// ------------------------------------------------------------------ softmax warps
// Two 32-bit numbers at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) { return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a); }
__device__ __forceinline__ float2 halves(uint64_t x) { return make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32))); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Which keys of a tile a row sees, as bits.
template <int KEYS>
struct Seen {
  uint32_t bits[KEYS / 32];
  // those in [0, end), but for [start, end_of_sinks) of the earlier ones
  __device__ __forceinline__ void set(int end, int start, int sinks) {
#pragma unroll
    for (int n = 0; n < KEYS / 32; ++n) {
      auto below = [&](int key) {  // numbers before `key`
        const int k = key - 32 * n;
        return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u;
      };
      bits[n] = below(end) & (~below(start) | below(sinks));
    }
  }
  __device__ __forceinline__ bool operator()(int n) const { return bits[n >> 5] >> (n & 31) & 1; }
};

// A row's weights of one tile where m is large (see ss_kv_attend.cuh), over its scores; returns their sum.
template <class E, int KEYS>
static __device__ __noinline__ float large_weights(uint32_t at, float scale, float z, Seen<KEYS> sees) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < KEYS; i += 16) {
    uint32_t x[16], w[8];
    tmem_load(x, at + i);
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
      float y[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) y[h] = sees(i + n + h) ? ex2(__fsub_rn(__fmul_rn(__uint_as_float(x[n + h]), scale), z)) : 0.0f;
      w[n / 2] = E::pack(y[0], y[1]);
      sum += y[0] + y[1];
    }
    tmem_store(at + i / 2, w);
  }
  return sum;
}

// Adds a tile whose values are not all finite to the output, key by key and only for the rows that see it.  (Not a call:
// what the loop around it keeps in registers would be spilled for it.)
template <class S>
__device__ __forceinline__ void add_by_key(uint32_t scores, uint32_t out, const unsigned char* ring, uint32_t slot, Seen<S::kKeys> sees, bool first) {
  using E = Elem<typename S::T>;
#pragma unroll 1
  for (int half = 0; half < S::kHalves; ++half) {
    const unsigned char* values = ring + (slot + half) % S::kSlots * S::kSlot;
#pragma unroll 1
    for (int d = 0; d < S::kWide; d += 32) {
      uint32_t o[32];
      if (!first) tmem_load(o, out + half * S::kWide + d);
      float acc[32];
#pragma unroll
      for (int n = 0; n < 32; ++n) acc[n] = first ? 0.0f : __uint_as_float(o[n]);
#pragma unroll 1
      for (int n = 0; n < S::kKeys; ++n) {
        uint32_t pair[1], word = sees.bits[0];
        tmem_load(pair, scores + (n >> 1));
        const float2 ws = E::unpack(pair[0]);
        const float wt = n & 1 ? ws.y : ws.x;
#pragma unroll
        for (int k = 1; k < S::kKeys / 32; ++k) word = n >> 5 == k ? sees.bits[k] : word;
        const bool seen = word >> (n & 31) & 1;
        const unsigned char* line = values + (d >> 6) * S::kRun + n * 128;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 y = *reinterpret_cast<const uint4*>(line + ((((d >> 3) & 7) + q) ^ (n & 7)) * 16);
          const uint32_t ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float2 v = E::unpack(ys[h]);
            if (seen) {
              acc[q * 8 + h * 2] = fmaf(wt, v.x, acc[q * 8 + h * 2]);
              acc[q * 8 + h * 2 + 1] = fmaf(wt, v.y, acc[q * 8 + h * 2 + 1]);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 32; ++n) o[n] = __float_as_uint(acc[n]);
      tmem_store(out + half * S::kWide + d, o);
    }
  }
  store_wait();
}

// 32 bytes of a row: at once where they are aligned.
__device__ __forceinline__ void store16(void* to, bool aligned, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g,
                                        uint32_t h) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
  } else {
    static_cast<uint4*>(to)[0] = make_uint4(a, b, c, d);
    static_cast<uint4*>(to)[1] = make_uint4(e, f, g, h);
  }
}

template <class S>
__device__ void softmax_warps(const PromptParams& P, const CUtensorMap* mo, unsigned char* sq, const unsigned char* ring, unsigned char* stage,
                              Control& c) {
  using T = typename S::T;
  using E = Elem<T>;
  constexpr int D = S::D;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = warp >> 2;
  const int m = threadIdx.x & 127;                                       // row of the tile
  const uint32_t lanes = c.tmem + ((uint32_t)(warp & 3) << 21);          // this warp's lanes of tensor memory
  const uint32_t out_at = lanes + S::kOut + r * D;
  const int token = r * P.tokens + m / P.heads, in_group = m % P.heads;  // of this row: token of the unit, head of the part
  const float scale = P.scale_log2;
  bool dead = false;
  auto wait = [&](unsigned long long* b, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(b, parity, P.spin_limit, 0u));
  };
  uint32_t nth = 0;  // slots of values before the unit
  uint32_t it = 0;   // tiles weighed so far
  // the slot of values number n: of the CTA's slots every 2 * kHalves bring a tile's keys, then its values
  auto slot_of = [](uint64_t n) { return (uint32_t)((n / S::kHalves * 2 * S::kHalves + S::kHalves + n % S::kHalves) % S::kSlots); };
  auto added = [&](uint32_t tile) {  // the output holds everything up to this tile
    wait(&c.pv_done[2 * r + (tile & 1)], (tile >> 1) & 1);
    fence_after();
  };
  // This row's queries of unit sg from shared to tensor memory, once the scores of the unit before are there.
  auto bring_queries = [&](int sg) {
    wait(&c.seg_full[sg & 1], (sg >> 1) & 1);
    if (dead || c.unit[sg & 1].tiles == 0) return;
    wait(&c.q_full[0], sg & 1);
    if (dead) return;
#pragma unroll 1
    for (int run = 0; run < D / 64; ++run) {
      uint32_t x[32];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const uint4 y = *reinterpret_cast<const uint4*>(sq + run * S::kQRun + m * 128 + ((n ^ (m & 7)) << 4));
        x[4 * n] = y.x;
        x[4 * n + 1] = y.y;
        x[4 * n + 2] = y.z;
        x[4 * n + 3] = y.w;
      }
      tmem_store(lanes + S::kQAt + run * 32, x);
    }
    store_wait();
    fence_before();
    __syncwarp();
    if (lane == 0) arrive(&c.q_ready);
  };
  if (S::kQTensor) bring_queries(0);
  bool more = true;
  for (int sg = 0; more; ++sg) {
    wait(&c.seg_full[sg & 1], (sg >> 1) & 1);
    if (dead) break;
    if (S::kQTensor && lane == 0) {  // the outputs have left the queries' room: the next ones may come
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      arrive(&c.q_free[0]);
    }
    const Unit u = c.unit[sg & 1];
    more = u.tiles > 0;
    const int count = tiles_of(u, r);  // 0 at the end
    const int pos = u.t0 + token;
    // Rows that are none hold another prompt's queries, another key head's, or what lies behind the last token.  They are weighed
    // like others and not written, but do not move m, and so have no say in how the warp rounds.  (As a row of m = infinity that
    // none passes it cost prompts of 64 columns 6 %, 100 of up to 700 tokens 90 -> 95 us.)
    const bool mine = m < P.heads * P.tokens && pos <= u.pos1 && u.chunk * P.heads + in_group < P.group;
    float mx = -INFINITY, l = 0.0f;
    bool large = false;
    for (int i = 0; i < count && !dead; ++i, ++it) {
      const uint32_t b = 2 * r + (it & 1), buf = lanes + b * S::kKeys;
      const int base = base_of<S>(u, i);
      const bool cut = cuts(u, i);
      wait(&c.s_full[b], (it >> 1) & 1);
      if (dead) break;
      fence_after();
      auto seen = [&]() {  // which keys of the tile this row sees (all, in one that cuts no row)
        Seen<S::kKeys> sees;
        if (cut) sees.set(pos + 1 - base, P.window > 0 ? pos - P.window + 1 - base : 0, P.sinks - base);
        else sees.set(S::kKeys, 0, 0);
        return sees;
      };
      uint32_t x[S::kKeys];
      float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      tmem_load(x, buf);
      if (cut) {
        const Seen<S::kKeys> sees = seen();
#pragma unroll
        for (int n = 0; n < S::kKeys; ++n)
          if (!sees(n)) x[n] = 0xff800000u;
      }
#pragma unroll
      for (int n = 0; n < S::kKeys; n += 8)
#pragma unroll
        for (int h = 0; h < 4; ++h) t[h] = fmaxf(t[h], fmaxf(__uint_as_float(x[n + h]), __uint_as_float(x[n + 4 + h])));
      const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale;
      const bool grow = mine && top - mx > 8.0f + E::kLift;
      if (__any_sync(0xffffffffu, grow)) {
        const float now = grow ? (fabsf(top) > kLarge ? top : top - E::kLift) : mx;
        const float by = grow ? ex2(mx - now) : 1.0f;  // 0 if nothing was seen before
        mx = now;
        large = __any_sync(0xffffffffu, mx != -INFINITY && fabsf(mx) > kLarge);
        l *= by;
        if (i > 0) {
          added(it - 1);
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            uint32_t o[16];
            tmem_load(o, out_at + d);
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * by);
            tmem_store(out_at + d, o);
          }
          store_wait();
        }
      }
      const float z = mx == -INFINITY ? 0.0f : mx;
      if (large) {
        l += large_weights<E, S::kKeys>(buf, scale, z, seen());
      } else {
        uint64_t s0 = 0, s1 = 0;  // sums of even and odd keys
        const uint64_t by = pair(scale, scale), less = pair(-z, -z);
        auto weigh = [&](const uint32_t* w, int from) {  // 32 keys
          uint32_t p[16];
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const float2 e = halves(fma2(pair(__uint_as_float(w[2 * n]), __uint_as_float(w[2 * n + 1])), by, less));
            const float a = ex2(e.x), b2 = ex2(e.y);
            p[n] = E::pack(a, b2);
            if (n & 1) s1 = add2(s1, pair(a, b2));
            else s0 = add2(s0, pair(a, b2));
          }
          tmem_store(buf + from / 2, p);
        };
        // (weights lie over scores that have been read)
        weigh(x, 0);
        weigh(x + 32, 32);
        const float2 s = halves(add2(s0, s1));
        l += s.x + s.y;
      }
      store_wait();
      if (cut) {
        const uint32_t n = nth + i * S::kHalves;
        for (int half = 0; half < S::kHalves; ++half) wait(&c.ready[(n + half) % kMaxSlots], parity_of(n + half));
        if (!dead && is_slow<S>(c, n)) {
          if (i > 0) added(it - 1);
          add_by_key<S>(buf, out_at, ring, slot_of(n), seen(), i == 0);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(&c.p_full[b]);
    }
    nth += u.tiles * S::kHalves;
    if (S::kQTensor && more && !dead) bring_queries(sg + 1);  // its first scores are taken beside this unit's end
    if (count > 0 && !dead) {
      added(it - 1);
      const float f = l == 0.0f ? 0.0f : 1.0f / l;
      const int head = c.unit[sg & 1].chunk * P.heads + in_group;
      const bool live = m < P.heads * P.tokens && pos <= c.unit[sg & 1].pos1 && head < P.group;
      const int q0 = c.unit[sg & 1].q0, head0 = c.unit[sg & 1].h * P.group;
      const long long q = q0 + pos;
      const int to_head = head0 + head;
      T* const to = static_cast<T*>(P.out) + q * P.out_stride + (long long)to_head * D;
      if (live && P.lse) P.lse[q * (P.group * P.hkv) + to_head] = l == 0.0f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994531f;
      const bool by_copy = (S::kStage > 0 || S::kQTensor) && P.staged && __all_sync(0xffffffffu, live);
#pragma unroll 1
      for (int d = 0; d < D; d += 64) {
        uint32_t o[64];
        tmem_load(o, out_at + d);
        if (by_copy) {
          // (with queries in tensor memory their room is the stage, of all columns)
          unsigned char* const to_stage = S::kQTensor ? sq + (d >> 6) * S::kQRun + (warp & 3) * 4096 : stage;
          if (!S::kQTensor) {  // the last 64 columns have left it
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            auto val = [&](int k) { return __uint_as_float(o[8 * n + k]) * f; };
            *reinterpret_cast<uint4*>(to_stage + lane * 128 + ((n ^ (lane & 7)) << 4)) =
                make_uint4(E::pack(val(0), val(1)), E::pack(val(2), val(3)), E::pack(val(4), val(5)), E::pack(val(6), val(7)));
          }
          proxy_fence();
          __syncwarp();
          if (lane == 0) {  // (this lane's row is the first of the warp's)
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(mo), "r"(d), "r"(to_head),
                         "r"(q0 + pos), "r"(smem_u32(to_stage))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          continue;
        }
        if (!live) continue;
#pragma unroll
        for (int n = 0; n < 64; n += 16) {
          auto val = [&](int k) { return __uint_as_float(o[n + k]) * f; };
          store16(to + d + n, P.aligned, E::pack(val(0), val(1)), E::pack(val(2), val(3)), E::pack(val(4), val(5)), E::pack(val(6), val(7)),
                  E::pack(val(8), val(9)), E::pack(val(10), val(11)), E::pack(val(12), val(13)), E::pack(val(14), val(15)));
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(&c.o_free[r]);
    }
    __syncwarp();
    if (lane == 0 && !dead) arrive(&c.seg_empty[sg & 1]);
  }
  if ((S::kStage > 0 || S::kQTensor) && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  __syncwarp();
  if (dead) report_all(P);
}

// ------------------------------------------------------------------ kernel
template <class T, int D, int TILES>
__global__ void __launch_bounds__((Shape<T, D, TILES>::kThreads), (Shape<T, D, TILES>::kCtas))
    prompt_kernel(const PromptParams P, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
  using S = Shape<T, D, TILES>;
  extern __shared__ unsigned char raw[];
  __shared__ Control c;
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  unsigned char* ring = base + TILES * S::kQ;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init_n(&c.full[i], 1);
      mbar_init_n(&c.empty[i], TILES);
      mbar_init_n(&c.ready[i], kGuardWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init_n(&c.s_full[i], 1);
      mbar_init_n(&c.p_full[i], 4);
      mbar_init_n(&c.pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_n(&c.seg_full[i], 1);
      mbar_init_n(&c.seg_empty[i], S::kSoftmax + S::kProducts + kGuardWarps);
      mbar_init_n(&c.q_full[i], 1);
      mbar_init_n(&c.q_free[i], S::kQTensor ? 4 : 1);
      mbar_init_n(&c.o_free[i], 4);
    }
    mbar_init_n(&c.q_ready, 4);
    mbar_init_n(&c.drained, S::kProducts);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == S::kProduct) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c.tmem)), "r"(S::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == S::kLoad && lane < 3) asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &mq : lane == 1 ? &mk : &mv) : "memory");
  // rows of the queries that no copy fills (128 is no multiple of `heads`): zeros, so that their scores are numbers
  const int filled = P.heads * P.tokens, lines = TILES * (D / 64) * (128 - filled) * 8;
  for (int i = tid; i < lines; i += S::kThreads)
    reinterpret_cast<uint4*>(base)[i / ((128 - filled) * 8) * 1024 + filled * 8 + i % ((128 - filled) * 8)] = make_uint4(0u, 0u, 0u, 0u);
  proxy_fence();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp < S::kSoftmax) {
    softmax_warps<S>(P, &mo, base, ring, ring + S::kSlots * S::kSlot + warp * S::kStage, c);
  } else if (warp == S::kLoad) {
    load_warp<S>(P, &mq, &mk, &mv, smem_u32(base), smem_u32(ring), c);
  } else if (warp < S::kGuard) {
    const int n = warp - S::kProduct;
    if (n & 1) values_warp<S>(P, n >> 1, smem_u32(ring), c);
    else scores_warp<S>(P, n >> 1, smem_u32(base), smem_u32(ring), c);
  } else {
    guard_warps<S>(P, ring, c);
  }
  fence_before();
  __syncthreads();
  if (warp == S::kProduct) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(c.tmem), "r"(S::kCols) : "memory");
  }
  // the counters are left at zero by the last CTA to end: every one has taken its last unit by then
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(P.ended, 1u) + 1 == gridDim.x) {
      *P.next = 0;
      *P.ended = 0;
      __threadfence();
    }
  }
}

template <class T, int D, int TILES>
PromptKernel entry() {
  using S = Shape<T, D, TILES>;
  return {reinterpret_cast<const void*>(&prompt_kernel<T, D, TILES>), S::kThreads, TILES, S::kKeys, S::kCtas, (size_t)S::kSmem};
}
template <class T>
PromptKernel pick(int d, int tiles) {
  if (d == 128 && tiles == 2) return entry<T, 128, 2>();
  return d == 64 ? entry<T, 64, 1>() : d == 128 ? entry<T, 128, 1>() : entry<T, 256, 1>();
}

}  // namespace prompt
}  // namespace kv
}  // namespace ss
