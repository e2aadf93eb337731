// ss_kv_append and ss_kv_commit: page bookkeeping of a serving step.
//
// With P tokens a page, row r holds ceil(len / P) pages and needs
// need_r = ceil((len + n) / P) - ceil(len / P) more; its i-th new page is
// free_pages[count - 1 - (sum of need over the rows before it) - i].  Both
// calls are a prefix sum over the rows and one pass over what is written:
// a few integers a row and a token, so latency is all that counts.  One
// launch each; every CTA scans all rows by itself (a scan of 512 rows costs
// less than a second launch or a hand-over between CTAs would), keeps what it
// needs of each row in shared memory, and the tokens (or returned pages) are
// spread flat over all threads, each finding its row by bisection.
#include "ss_kv_common.cuh"

namespace ss {
namespace {

constexpr int kNT = 512;
constexpr int kClusterCtas = 8;  // the grid is one cluster: commit reads state in every CTA before any writes it

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// Exclusive prefix sum of one value per thread; *total gets the block's sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  __syncthreads();  // warp_sums may still be read from the call before
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) {
    const int s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + incl - v;
}

// The last index r of first[0..n) with first[r] <= i (first[0] <= i).
__device__ __forceinline__ int row_of(const int* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

// What append keeps of a row beside its first token: its cached length and
// the free-page index of its block b as `base - b` (kNone: not served).
struct AppendRow {
  int len, base;
};
constexpr int kNone = INT32_MIN;

__global__ void __launch_bounds__(kNT) append_kernel(const PagesParams P) {
  extern __shared__ int smem[];
  __shared__ int warp_sums[kNT / 32];
  AppendRow* rows = reinterpret_cast<AppendRow*>(smem);  // [B]
  int* first = smem + 2 * P.B;                           // [B + 1] first token of each row
  const int count = min(max(*P.free_count, 0), P.num_pages);
  int used = 0;  // pages wanted by the rows before this chunk; a token needs at most one, so sums stay below 2^30
  for (int r0 = 0; r0 < P.B; r0 += kNT) {
    const int r = r0 + (int)threadIdx.x;
    int need = 0, len = 0, n = 0;
    uint32_t status = 0;
    if (r < P.B) {
      const int from = P.cu_new[r], to = P.cu_new[r + 1];
      len = P.kv_len[r];
      first[r] = from;
      if (r == P.B - 1) first[P.B] = to;
      if (from < 0 || to < from || to > P.max_tokens || len < 0 || len > P.max_blocks << P.page_shift) {
        status = SS_ST_BAD_PARAM;
      } else {
        n = to - from;
        const int want = (int)(((long long)len + n + (1 << P.page_shift) - 1) >> P.page_shift);
        if (want > P.max_blocks) status = SS_ST_KV_TABLE;
        else need = want - pages_of(len, P.page_shift);
      }
    }
    int total;
    const int before = used + block_scan(need, warp_sums, &total);
    used = (int)min((long long)used + total, 1ll << 30);
    if (r < P.B) {
      if (need > 0 && (long long)before + need > count) status = SS_ST_KV_POOL;
      const int held = status == SS_ST_BAD_PARAM ? 0 : len;
      rows[r] = {held, status ? kNone : count - 1 - before + pages_of(held, P.page_shift)};
      if (r % gridDim.x == blockIdx.x) {  // what is written once is shared out between the CTAs
        P.seq_len[r] = status ? len : len + n;
        P.row_status[r] = status;
      }
    }
  }
  __syncthreads();
  if (gridDim.x > 1) cluster_sync();  // row_status is written before bits are added
  const int tokens = min(max(first[P.B], 0), P.max_tokens);
  const int mask = (1 << P.page_shift) - 1;
  for (int i = blockIdx.x * kNT + (int)threadIdx.x; i < tokens; i += gridDim.x * kNT) {
    const int r = row_of(first, P.B, i);
    const AppendRow row = rows[r];
    const int pos = row.len + (i - first[r]);
    int slot = -1;
    if (row.base != kNone && i >= first[r] && i < first[r + 1]) {
      const int block = pos >> P.page_shift;
      const bool fresh = block >= pages_of(row.len, P.page_shift);
      int32_t* entry = P.block_table + (long long)r * P.max_blocks + block;
      const int page = fresh ? P.free_pages[row.base - block] : *entry;
      if ((unsigned)page < (unsigned)P.num_pages) slot = (page << P.page_shift) + (pos & mask);
      else atomicOr(&P.row_status[r], (uint32_t)SS_ST_KV_PAGE);
      if (fresh && (pos & mask) == 0) *entry = page;
    }
    P.positions[i] = pos;
    P.slots[i] = slot;
  }
}

__global__ void __launch_bounds__(kNT) commit_kernel(const PagesParams P) {
  extern __shared__ int smem[];
  __shared__ int warp_sums[kNT / 32];
  int* start = smem;             // [B] pages that the rows before return
  int* block0 = smem + P.B;      // [B] first block that a row returns
  int* after = smem + 2 * P.B;   // [B] new length
  const int count = min(max(*P.free_count, 0), P.num_pages);
  const int cap = P.max_blocks << P.page_shift;
  int back = 0, reserved = 0;
  for (int r0 = 0; r0 < P.B; r0 += kNT) {
    const int r = r0 + (int)threadIdx.x;
    int ret = 0, held = 0;
    if (r < P.B) {
      const int len = min(max(P.kv_len[r], 0), cap), seq = min(max(P.seq_len[r], len), cap);
      const long long want = P.counts ? (long long)P.counts[r] + P.plus : (long long)seq;
      const int keep = (int)min(max(want, 0ll), (long long)(seq - len));
      const int now = P.finished && P.finished[r] != 0 ? 0 : len + keep;
      const int top = pages_of(seq, P.page_shift);
      held = top - pages_of(len, P.page_shift);
      ret = top - pages_of(now, P.page_shift);
      block0[r] = top - ret;
      after[r] = now;
    }
    int total;
    const int before = block_scan(ret, warp_sums, &total);
    if (r < P.B) start[r] = back + before;
    back += total;
    block_scan(held, warp_sums, &total);
    reserved += total;
  }
  __syncthreads();
  const int base = count - reserved;
  for (int i = blockIdx.x * kNT + (int)threadIdx.x; i < back; i += gridDim.x * kNT) {
    const int r = row_of(start, P.B, i);
    const int block = block0[r] + (i - start[r]);
    if ((unsigned)block < (unsigned)P.max_blocks && (unsigned)(base + i) < (unsigned)P.num_pages)
      P.free_pages[base + i] = P.block_table[(long long)r * P.max_blocks + block];
  }
  cluster_sync();  // every CTA has read the count and the lengths
  if (blockIdx.x != 0) return;
  if (threadIdx.x == 0) *P.free_count = min(max(base + back, 0), P.num_pages);
  for (int r = (int)threadIdx.x; r < P.B; r += kNT) P.kv_len[r] = after[r];
}

constexpr int kMaxRows = 8192;
size_t pages_smem(int rows) { return (3 * (size_t)rows + 1) * 4; }

cudaError_t launch_cluster(void (*kernel)(const PagesParams), int ctas, const PagesParams& P, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(kNT);
  c.dynamicSmemBytes = pages_smem(P.B);
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = ctas;
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P);
}

}  // namespace

cudaError_t kv_pages_configure() {
  const int bytes = (int)pages_smem(kMaxRows);
  const cudaError_t e = cudaFuncSetAttribute(append_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(commit_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

cudaError_t kv_append_launch(const PagesParams& P, cudaStream_t st) {
  return launch_cluster(append_kernel, P.max_tokens <= kNT ? 1 : kClusterCtas, P, st);
}

cudaError_t kv_commit_launch(const PagesParams& P, cudaStream_t st) {
  return launch_cluster(commit_kernel, kClusterCtas, P, st);
}

}  // namespace ss
