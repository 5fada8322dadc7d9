/*
 * tiered_attn_cache.h -- C ABI of the cached-attention operators of
 * libtiered_attn.so (sm_100a): a paged key-value cache for causal generation,
 * appended to with the position rotation applied on the way, and read by
 * attention of new tokens over the whole cache or over the pages that a cheap
 * score chooses for each of them.
 *
 * The cache.  Keys and values live in pages of `page_size` slots for every
 * key head.  A sequence is a row of the block table: its token at position p
 * lies in page table[s][p / page_size], slot p % page_size.  seq_lens[s] is
 * the length of sequence s AFTER the new tokens of the current step, in every
 * call of the step.
 *
 * Rows.  The new tokens of a step are packed: sequence s owns rows
 * cu[s] .. cu[s+1]-1 of K_new, V_new, Q and O, and row t stands at position
 * seq_lens[s] - (cu[s+1] - t).  cu = NULL means one row for each sequence
 * (row s is sequence s; T must equal S).  A row sees the keys at positions up
 * to its own, also among the new tokens of a step: the tokens of a frame do not
 * see the ones behind them.  (For a frame whose tokens all see each other, append
 * it, then attend with a sequence for each row: cu = NULL, the frame's end as
 * every length, the table's row repeated.)  Rows from cu[S] on are padding:
 * neither read nor written.
 * Sequences may be empty (cu[s] = cu[s+1]).  cu ascends from 0; with one that
 * does not, results are undefined, but nothing outside the buffers is read or
 * written.
 *
 * Conventions are those of tiered_attn.h: host-side validation before any
 * launch, asynchronous work on `stream`, no allocation, device-side errors in
 * the workspace's status word (tiered_attn_get_status).  Lengths, tables,
 * cu and lists are read on the device, so a captured CUDA graph replays with
 * other values in the same buffers; what they must satisfy is checked there:
 *  - a length below 0 or above max_pages * page_size is clamped;
 *  - a page number outside 0 .. n_pages-1 counts as a page without keys, and
 *    nothing is written to it;
 *  - a row before its sequence's first position (seq_lens[s] smaller than the
 *    number of new tokens) is not appended and sees no key;
 * each of these also sets the status word to TA_ERR_BAD_INDEX.
 *
 * The workspace.  tiered_attn_cache_workspace_bytes(p) bytes, 256-byte
 * aligned, set to zero ONCE before its first use (tiered_attn_cache_init);
 * every call leaves it ready for the next, whatever operator or parameters
 * that has.  The status word keeps the first error until the next
 * tiered_attn_cache_init.  Calls whose work can overlap on the GPU need a
 * workspace each.
 */
#ifndef TIERED_ATTN_CACHE_H
#define TIERED_ATTN_CACHE_H

#include "tiered_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TA_CACHE_BF16 = 0,
  TA_CACHE_FP8 = 1           /* e4m3 codes and one power-of-two scale for each
                                token and head: the smallest 2^k, k >= -126,
                                with amax <= 448 * 2^k (1 for a zero token).
                                A token with a value that is not finite (a
                                key: in fp32, after its rotation) gets a NaN
                                scale */
} ta_cache_format;

typedef struct {
  int32_t n_pages;           /* pages of the cache                            */
  int32_t page_size;         /* slots of a page: 16, 32, 64 or 128            */
  int32_t H, Hkv, d;         /* query heads, key heads (H a multiple of Hkv;
                                query head h reads key head h / (H / Hkv)),
                                head dim (64 or 128)                          */
  int32_t format;            /* ta_cache_format                               */
  int32_t S, T;              /* sequences; rows of the new-token buffers      */
  int32_t max_pages;         /* pages of a sequence at most (columns of the
                                block table that may be read)                 */
  int32_t n_select;          /* select / sparse: entries of a row's page list,
                                1 .. 1024                                     */
  int32_t n_first, n_recent; /* select: pages always kept, at the sequence's
                                start (>= 0) and at the row's end (>= 1);
                                n_first + n_recent <= n_select                */
  int32_t rot_dim;           /* append: leading elements of a head that are
                                rotated (a multiple of 16, <= d; 0: none)     */
  int32_t rot_interleaved;   /* 0: element i turns with i + rot_dim/2;
                                1: element 2i with 2i + 1                     */
  int32_t rot_rows;          /* rows of the cos / sin tables                  */
  float softmax_scale;       /* 0 selects 1/sqrt(d)                           */
  /* Element strides; the innermost dimension is contiguous.  Rows of 16-bit
   * tensors start on 16-byte boundaries, and so do the cache's rows. */
  int64_t stride_page, stride_head, stride_slot;   /* codes of K and V        */
  int64_t stride_table;                            /* block table rows        */
  int64_t stride_k_t, stride_k_h;                  /* K_new [T, Hkv, d]       */
  int64_t stride_v_t, stride_v_h;                  /* V_new [T, Hkv, d]       */
  int64_t stride_q_t, stride_q_h;                  /* Q [T, H, d]             */
  int64_t stride_o_t, stride_o_h;                  /* O, rotated Q [T, H, d]  */
} ta_cache_params;

/* Device pointers of the cache.  k and v: bf16 or e4m3 [n_pages, Hkv,
 * page_size, d] with the strides above (any order of the outer three).
 * k_scale and v_scale (TA_CACHE_FP8, else NULL): f32 [n_pages, Hkv,
 * page_size], contiguous.  k_mean: f32 [n_pages, Hkv, d], contiguous, the
 * mean of a page's keys, or NULL where pages are never chosen by it. */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  float* k_mean;
} ta_cache;

/* Bytes of workspace for every operator with these sizes; 0 when `p` is
 * invalid or unsupported.  Host only. */
size_t tiered_attn_cache_workspace_bytes(const ta_cache_params* p);

/* Sets a workspace to zero on `stream`. */
ta_status tiered_attn_cache_init(void* ws_dev, size_t ws_bytes, void* stream);

/* Appends the new tokens: row t of K_new (rotated) and V_new goes to its slot,
 * rounded once to the cache's format.  One launch.
 *  - Rotation by the angle whose cosine and sine stand in row pos[t] of
 *    cos_dev and sin_dev (f32 [rot_rows, rot_dim/2]; pos int32 [T], NULL: the
 *    row's position in its sequence): a pair (x, y) becomes
 *    (x cos - y sin, y cos + x sin).  A pos outside the table leaves the
 *    token (and its rotated query) unwritten and sets TA_ERR_BAD_INDEX; its
 *    page fills all the same, the mean counting what stood in its slot.
 *  - Q_dev, when not NULL, is rotated the same way into Q_out_dev (which may
 *    be Q_dev with equal strides).
 *  - k_mean of every page that these tokens fill up is written: the fp32 sum
 *    of the page's stored keys (decoded, FP8) in slot order, divided by
 *    page_size.  It depends on what the page holds only, not on how many
 *    calls brought it, and a page filled again after a rollback gets its new
 *    mean.  Means of pages that are not full are not touched.
 * No two rows may fall into one slot (two table entries of live sequences
 * with the same page): which of them stays is then undefined. */
ta_status tiered_attn_cache_append(const ta_cache_params* p, const ta_cache* cache,
                                   const void* K_new_dev, const void* V_new_dev,
                                   const void* Q_dev, void* Q_out_dev, const float* cos_dev,
                                   const float* sin_dev, const int32_t* pos_dev,
                                   const int32_t* cu_dev, const int32_t* seq_lens_dev,
                                   const int32_t* table_dev, void* ws_dev, size_t ws_bytes,
                                   void* stream);

/* Attention of one new token of each sequence (row s of Q) over its whole
 * cache: O[s, h] = sum_i softmax_i(scale * q . k_i) v_i, i < seq_lens[s].
 * The keys are split evenly over the GPU and the parts joined in a fixed
 * order; the result depends on the lengths and not on timing.  The softmax's
 * weights multiply V rounded to bf16 (FP8 caches: to f16); maxima, sums and O are
 * fp32 until O's one rounding.  O_dev: bf16
 * [S, H, d]; lse_dev: f32 [S, H] ln sum_i exp(scale * q . k_i), or NULL.  An
 * empty sequence gives O = 0 and lse = -inf.  At most 2048 sequences (else
 * TA_ERR_UNSUPPORTED).  One launch. */
ta_status tiered_attn_cache_decode(const ta_cache_params* p, const ta_cache* cache,
                                   const void* Q_dev, const int32_t* seq_lens_dev,
                                   const int32_t* table_dev, void* O_dev, float* lse_dev,
                                   void* ws_dev, size_t ws_bytes, void* stream);

/* Chooses the pages that each row reads, for each key head: the first n_first
 * and the last n_recent of the pages it sees, and among the others (all of
 * them full) those of greatest pooled mass, ties to the lower page, until the
 * list has n_select entries.  The mass of page j for query head h is
 * softmax_j(scale * q_h . k_mean_j) over the pages that compete, and the
 * page's is the sum over the query heads of the key head, all in fp64: the
 * mass router of tiered_attn_plan with a query block of one row.  A product
 * that is not finite adds no mass.
 * sel_dev: int32 [T, Hkv, n_select], a row's page indices (in its sequence)
 * in ascending order, then -1.  Only k_mean of the cache is read.  At most
 * 16384 pages of a sequence, 128 query heads of a key head, 65535 sequences and
 * 2^31 - 1 (row, key head) pairs (else TA_ERR_UNSUPPORTED).  The workspace
 * holds 8 bytes for each page of the table's width (rounded up to 128) and query
 * head of as many rows as 4 GiB take (one at least), and where T >= 2 S some
 * 4 d for each such page and key head of each sequence.  Two launches for so many
 * rows; where rows share their means, three for so many and one more. */
ta_status tiered_attn_cache_select(const ta_cache_params* p, const ta_cache* cache,
                                   const void* Q_dev, const int32_t* cu_dev,
                                   const int32_t* seq_lens_dev, const int32_t* table_dev,
                                   int32_t* sel_dev, void* ws_dev, size_t ws_bytes, void* stream);

/* Attention of each row over the pages of its list only (sel_dev as written
 * by tiered_attn_cache_select, or any lists: entries below 0 and pages past
 * the row's position are skipped, a page listed twice counts twice).  O_dev:
 * bf16 [T, H, d]; lse_dev: f32 [T, H], or NULL.  A row without keys gives 0
 * and -inf.  Where sequences have many rows, neighbouring rows share the loads
 * of the pages they have in common; a row's result does not depend on what
 * other rows hold but for its rounding.  Weights are rounded as for decode, but
 * where FP8 caches meet many rows to bf16, which is coarser.  A list of every page
 * (n_select of them at most) makes it dense attention.  O may not overlap Q (the same pointer is
 * refused): with many rows some are done again from their queries.  One launch,
 * or three with many rows. */
ta_status tiered_attn_cache_sparse(const ta_cache_params* p, const ta_cache* cache,
                                   const void* Q_dev, const int32_t* sel_dev,
                                   const int32_t* cu_dev, const int32_t* seq_lens_dev,
                                   const int32_t* table_dev, void* O_dev, float* lse_dev,
                                   void* ws_dev, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TIERED_ATTN_CACHE_H */
