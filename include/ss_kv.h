/* ss_kv.h -- the serving step around ss_verify: a paged key-value cache on
 * one GB300 GPU.  Part of libss.so; the conventions are those of ss.h: plain
 * pointers and sizes, caller-owned device memory, no allocation, no
 * synchronisation and no copy to the host inside a call, launch shapes that
 * depend only on the plan and on host arguments (so every call can be
 * captured in a CUDA graph and replayed with new device data), host-visible
 * misuse refused before any launch with a negative status, data errors
 * reported as row status bits.
 *
 * One step of a batch of requests ("rows"), each with 1 .. gamma + 1 new
 * tokens (its last token and its drafts; or a piece of its prompt):
 *   ss_kv_append   pages for the new tokens: their slots, positions, lengths
 *   ss_rope_store  per layer: norms of queries and keys, rotary positions,
 *                  queries out, keys and values into the cache
 *   ss_attend      per layer: attention of the new tokens over the cache
 *   ss_verify      (ss.h) which drafts are accepted
 *   ss_kv_commit   lengths move past what was accepted, pages that hold
 *                  nothing kept go back to the pool
 *
 * The cache of one layer is two arrays (keys, values) of num_pages pages of
 * page_size tokens of kv_heads heads of head_dim values, in any order of
 * pages, tokens and heads (ss_kv_cache holds the strides); the values of a
 * head are contiguous.  Token t of row r lives in page
 * block_table[r][t / page_size] at place t % page_size; its slot is
 * page * page_size + place.
 */
#ifndef SS_KV_H_
#define SS_KV_H_

#include "ss.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations (SS_BF16, SS_F16) and of the cache (the
 * activations' type, or SS_E4M3: 8-bit values with one fp32 factor per key
 * head; the value held is x / factor, rounded to nearest, infinities and all
 * beyond 448 as 448 with their sign, NaN as NaN). */
enum { SS_F16 = 2, SS_E4M3 = 3 };

/* Row status bits of these calls, beside those of ss.h. */
enum {
  SS_ST_KV_POOL = 1u << 11,  /* ss_kv_append: too few free pages for this row: not served */
  SS_ST_KV_TABLE = 1u << 12, /* ss_kv_append: the row would need more than max_blocks pages: not served */
  SS_ST_KV_PAGE = 1u << 13   /* a page id outside [0, num_pages) in a place that is in use: ss_kv_append gives
                                the tokens on it slot -1, ss_attend treats them as not visible */
};

/* Sizes fixed at plan creation. */
typedef struct {
  int32_t max_rows;    /* 1 .. 8192 */
  int32_t max_tokens;  /* new tokens of one call, over all rows: 1 .. 2^24 */
  int32_t max_new;     /* new tokens that a row usually has at most: chooses ss_attend's row tile (rows with
                          more are served too); >= 1 */
  int32_t q_heads;     /* a multiple of kv_heads */
  int32_t kv_heads;    /* 1 .. 1024 */
  int32_t head_dim;    /* 64, 128 or 256 */
  int32_t page_size;   /* a power of two, 16 .. 1024 */
  int32_t num_pages;   /* num_pages * page_size < 2^31 */
  int32_t max_blocks;  /* entries of a block-table row; max_blocks * page_size < 2^31 */
  int32_t dtype;       /* SS_BF16 or SS_F16 */
  int32_t cache_dtype; /* dtype, or SS_E4M3 */
  int32_t device;      /* CUDA ordinal */
} ss_kv_config;

/* Opaque, immutable after creation; host memory owned by the caller. */
typedef struct ss_kv_plan ss_kv_plan;

ss_status ss_kv_plan_create(ss_kv_plan** plan, const ss_kv_config* config);
void ss_kv_plan_destroy(ss_kv_plan* plan);

/* Device scratch of ss_attend: partial results of rows whose cached tokens
 * are split over several CTAs, and their counters.  Zeroed once before its
 * first use with a plan; every completed call leaves the counters at zero.
 * Calls that overlap in time need a workspace each. */
size_t ss_kv_workspace_bytes(const ss_kv_plan* plan);

/* One layer's cache (host struct of device pointers); strides in elements,
 * each a positive multiple of 16 bytes, both pointers 16-byte aligned. */
typedef struct {
  void* k;
  void* v;
  int64_t page_stride, token_stride, head_stride;
  const float* k_scale; /* [kv_heads] factors of an SS_E4M3 cache, normal numbers > 0; NULL = 1 (NULL for other caches) */
  const float* v_scale;
} ss_kv_cache;

/* The pool and the rows' tables (host struct of device pointers).
 * Between an append and its commit only block_table entries past a row's
 * held pages are written; an append can be repeated (with other new tokens,
 * too) before the commit. */
typedef struct {
  int32_t B;             /* rows of this call, 1 .. max_rows */
  int32_t tokens;        /* ss_kv_append: entries of slots and positions (those past max_tokens are not used) */
  int32_t* block_table;  /* [B, max_blocks]; entries past a row's pages are not read */
  int32_t* kv_len;       /* [B] tokens held */
  int32_t* free_pages;   /* [num_pages], the first *free_count are free; the last of them goes first */
  int32_t* free_count;   /* [1] */
  void* stream;          /* cudaStream_t */
  const ss_kv_plan* plan;
} ss_kv_pool;

/* Pages for n_r = cu_new[r+1] - cu_new[r] new tokens of each row: new pages
 * are taken from the end of the free pages, rows in order, and entered in
 * block_table.  A row that the free pages left by the rows before it do not
 * cover (SS_ST_KV_POOL), or that would pass its table row (SS_ST_KV_TABLE),
 * is not served: its tokens get slot -1 and its seq_len stays kv_len.  kv_len,
 * free_pages and free_count are not changed.
 * cu_new:     [B+1] prefix sums, cu_new[0] = 0.  A row with a negative count,
 *             a negative kv_len or a token past max_tokens or pool->tokens is
 *             not served (SS_ST_BAD_PARAM).
 * slots:      [tokens] (it and positions may be NULL if pool->tokens is 0)
 * positions:  [tokens] kv_len + index of the token in its row
 * seq_len:    [B] kv_len + n_r (kv_len if not served)
 * row_status: [B] written (0 or bits). */
ss_status ss_kv_append(const ss_kv_pool* pool, const int32_t* cu_new, int32_t* slots, int32_t* positions,
                       int32_t* seq_len, uint32_t* row_status);

/* Ends a step: row r keeps clamp(counts[r] + plus, 0, seq_len[r] - kv_len[r])
 * of its new tokens (all of them with counts NULL), kv_len moves past them,
 * and its pages that hold nothing kept go back to the end of the free pages,
 * in order of row and block.  counts = num_accepted of ss_verify with plus = 1
 * keeps a row's last token and its accepted drafts.  A row with
 * finished[r] != 0 (finished may be NULL) keeps nothing: all its pages go
 * back and its kv_len is 0.  seq_len: as the append wrote it. */
ss_status ss_kv_commit(const ss_kv_pool* pool, const int32_t* seq_len, const int32_t* counts, int32_t plus,
                       const int32_t* finished);

/* Queries, keys and values of T tokens on their way from the projection. */
typedef struct {
  int32_t T;              /* 0 .. max_tokens */
  const void *q, *k, *v;  /* [T, heads, head_dim], heads contiguous; 16-byte aligned */
  int64_t q_stride, k_stride, v_stride; /* between tokens, in elements: a multiple of 8 */
  const void* q_weight;   /* [head_dim] or NULL: no norm of the queries */
  const void* k_weight;   /* [head_dim] or NULL: no norm of the keys */
  float eps;
  const double* inv_freq; /* [rot_dim / 2] angles per position, in radians (scaled for long contexts as the
                             model wants: ss_rope_frequencies) */
  int32_t rot_dim;        /* 0 .. head_dim, a multiple of 16: the first rot_dim values of a head are rotated */
  int32_t interleaved;    /* 0: value i pairs with i + rot_dim / 2; 1: 2i with 2i + 1 */
  float rope_scale;       /* factor of cos and sin (1 unless the scaling of long contexts has one) */
  const int32_t* positions; /* [T] */
  const int32_t* slots;     /* [T]; a slot outside the cache (-1) stores nothing */
  void* q_out;            /* [T, q_heads, head_dim]; may be q itself */
  int64_t q_out_stride;
  void* stream;
  const ss_kv_plan* plan;
} ss_rope_batch;

/* For every head x of q and k: x * rsqrt(mean(x^2) + eps) * weight where a
 * weight is given, then (a, b) -> (a cos - b sin, b cos + a sin) for its
 * pairs, angle = position * inv_freq taken modulo a turn in 64-bit fixed
 * point (exact for every 32-bit position); everything in fp32, rounded once
 * (the mean of squares that pass its range is taken of scaled values; beside an
 * infinite value the others of a normed head become 0, and it and its pair NaN).
 * Queries go to q_out, keys and (unchanged) values to the slots. */
ss_status ss_rope_store(const ss_rope_batch* batch, const ss_kv_cache* cache);

/* Angles per position, base^(-2i / rot_dim), on the host.  factor > 1
 * stretches the positions of a longer context: with original_len 0 every
 * angle is divided by it; otherwise angles that turn at most low_turns times
 * over original_len positions are, those that turn at least high_turns times
 * stay, and between the two the angle is blended linearly in its turns. */
ss_status ss_rope_frequencies(double* inv_freq, int32_t rot_dim, double base, double factor, int32_t original_len,
                              double low_turns, double high_turns);

/* New tokens' queries and where their keys are. */
typedef struct {
  int32_t B;
  int32_t tokens;         /* that q, out and lse hold (those past max_tokens are not used); 0: nothing is done */
  const void* q;          /* [tokens, q_heads, head_dim], heads contiguous; 16-byte aligned */
  int64_t q_stride;       /* between tokens, in elements: a multiple of 8 */
  const int32_t* cu_new;  /* [B+1] prefix sums of the rows' new tokens */
  const int32_t* seq_len; /* [B] tokens of the row, the new ones included */
  const int32_t* block_table; /* [B, max_blocks] */
  float scale;            /* of the scores, > 0 */
  int32_t window;         /* 0: every earlier token; else the last `window` tokens, a token itself included */
  int32_t sinks;          /* with a window: the first `sinks` tokens stay visible */
  void* out;              /* [tokens, q_heads, head_dim] */
  int64_t out_stride;
  float* lse;             /* [tokens, q_heads] ln of the softmax sum, or NULL */
  uint32_t* row_status;   /* [B]: bits are OR-ed in (ss_kv_append writes it anew each step) */
  void* workspace;        /* 256-byte aligned */
  size_t workspace_bytes; /* >= ss_kv_workspace_bytes(plan) */
  void* stream;
  const ss_kv_plan* plan;
} ss_attend_batch;

/* out = sum_t softmax_t(scale q . k_t) v_t over the tokens t that the query
 * sees: with p its position (seq_len - n_r + its index), t <= p and, with a
 * window, t > p - window or t < sinks.  Query head h reads key head
 * h / (q_heads / kv_heads).  Scores, softmax sums and outputs are fp32,
 * rounded once at the end (the softmax weights are rounded to the cache's
 * 16-bit type, f16 for SS_E4M3, before the product with the values; the sum
 * that divides is then that of the rounded bf16 weights; bf16 queries over an
 * SS_E4M3 cache become f16 by a power of two a row and head, so that values
 * below 2^-28 of the largest lose bits; f16 weights keep 11
 * bits down to 2^-21 of the row's largest, and below 2^-32 of it may count as 0).  A query
 * that sees no token (a position below 0), or only scores of -inf, gives
 * zeros and lse -inf.  Values of tokens that a query does not see never reach
 * its result, whatever they hold.  A row whose cu_new passes tokens or
 * max_tokens, or decreases, is left out (SS_ST_CAPACITY); one whose seq_len is
 * negative or passes its table row gives zeros (SS_ST_BAD_PARAM).  An infinite
 * value that a query does see may give NaN in its column.  Every wait inside
 * the kernel is bounded: should one run out (not expected), the rows concerned
 * report SS_ST_COPY_TIMEOUT, and the workspace is to be zeroed before its next
 * use. */
ss_status ss_attend(const ss_attend_batch* batch, const ss_kv_cache* cache);

#ifdef __cplusplus
}
#endif

#endif /* SS_KV_H_ */
