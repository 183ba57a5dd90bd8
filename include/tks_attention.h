/*
 * tks_attention.h - C ABI of libtks, second part: a paged key/value cache and
 * the attention that reads it (GB300, sm_103a).
 *
 * The selector of tks.h is step 2 of sparse attention ("Technical Deep Dive |
 * How to Use FlagOS's New Triton-TLE Language to Build a TopK Selector Faster
 * Than FlashInfer", section "01. Why the TopK Selector Needs Optimization").
 * These calls are what stands around it: writing the keys and values of new
 * tokens into a cache (held as bfloat16, or as 8-bit integers with a scale for
 * each token and head), reading them back, the attention of drafted tokens
 * over a whole context, and step 3, the attention over the selected positions.
 *
 * Status codes, streams, workspaces and device-side errors are those of tks.h:
 * calls are asynchronous on `stream`, argument errors return TKS_E_INVAL and
 * launch nothing, and errors found on the device are read with
 * tks_device_status(stream) (which reports one at a time: first those of the
 * selection, then, at its next call, those of the calls below; of several kinds
 * of these, TKS_E_TIMEOUT before TKS_E_INDEX before TKS_E_ROW_LEN, and all are
 * cleared).  The library
 * allocates one workspace for each (device, stream) on the first of these calls
 * on it (make that call before any CUDA-graph capture); later calls allocate
 * nothing and never synchronise, and tks_release frees it with the others.
 * (cudaStreamPerThread is a stream of every host thread, so each thread that
 * passes that handle to these calls gets a workspace, and asks for the errors
 * of its own stream.)
 * The caller owns every buffer, which must stay valid until the work completes.
 *
 * Results do not depend on timing: the same call gives the same bits (but for
 * tokens that are written to one slot, see tks_cache_write).  Waits
 * inside the attention kernels are bounded by TKS_OPT_SPIN_LIMIT_NS; one that
 * runs out is reported as TKS_E_TIMEOUT, and the outputs of that call are then
 * undefined.  (TKS_OPT_TEST_SKIP_ARRIVE makes one run out where a call has more
 * than 16 query rows for a key/value head.)
 */
#ifndef TKS_ATTENTION_H
#define TKS_ATTENTION_H

#include <stdint.h>

#include "tks.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A third element type, beside those of tks_dtype: how a cache may be held. */
#define TKS_I8 2 /* signed 8-bit codes in [-127, 127], value = code * scale */

/* The range of a row's largest magnitude when it is held in 8 bits. */
#define TKS_AMAX_LOW_LOG2 (-40)
#define TKS_AMAX_HIGH_LOG2 80

/* Most drafted tokens of one sequence in tks_tree_attention. */
#define TKS_DRAFTS_MAX 1024

/*
 * A paged cache.  Row (page, token, head) of the keys starts at element
 * page * page_stride + token * token_stride + head * head_stride of `k` and
 * holds head_dim contiguous elements; the values likewise at `v`.  Strides are
 * in elements, not negative, and multiples of 16 bytes; the bases are 16-byte
 * aligned.  Slot s means token s % page_size of page s / page_size.
 */
typedef struct {
    void *k, *v;
    float *scales;       /* held == TKS_I8: [pages][page_size][kv_heads][2], the scale of
                            the key and of the value of each row, 8-byte aligned; else NULL */
    int32_t held;        /* TKS_BF16 or TKS_I8 */
    int32_t pages;       /* >= 1; pages * page_size < 2^31 */
    int32_t page_size;   /* a power of two */
    int32_t kv_heads;    /* >= 1 */
    int32_t head_dim;    /* 64 or 128 */
    int64_t page_stride, token_stride, head_stride;
} tks_cache;

/*
 * tks_cache_write - put the keys and values of n tokens into slots[0..n).
 *
 *   k, v     device pointers, element type `dtype` (TKS_BF16 or TKS_F32); head
 *            h of token i starts at element i * token_stride + h * head_stride
 *            of each (strides for k and v apart; multiples of 16 bytes)
 *   slots    device pointer, int32 [n].  A negative slot skips its token; one
 *            at or beyond pages * page_size is skipped and reported as
 *            TKS_E_INDEX.  Slots are to differ: what two tokens with the same
 *            slot leave there is undefined (it may be a mixture of both, codes
 *            of one under the scale of the other, and differ from run to run)
 *
 * A cache in bfloat16 takes each value rounded to nearest even.  A cache in 8
 * bits takes, for a row x of one token and head,
 *     amax  = max |x|, held to [2^-40, 2^80]
 *     scale = amax * (1/127)                 (32-bit arithmetic)
 *     code  = x * (1/scale), rounded to nearest even, held to [-127, 127]
 * so infinities count as the largest value, and a row with a NaN gets a NaN
 * scale: every query that attends to it has a NaN result, and no other.
 * (2^-40 / 127 lies above 2^-47, below which the attention calls take a value's
 * scale for 2^-47.)
 */
int tks_cache_write(const tks_cache *cache, const void *k, const void *v, int32_t n,
                    int32_t dtype, int64_t k_token_stride, int64_t k_head_stride,
                    int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots,
                    void *stream);

/*
 * tks_cache_read - the values that slots[0..n) stand for, as `dtype` (TKS_BF16
 * or TKS_F32), in k_out and v_out, both [n][kv_heads][head_dim], 16-byte
 * aligned.  Rows of a negative slot are zero; a slot at or beyond pages *
 * page_size reads as zero and is reported as TKS_E_INDEX.
 */
int tks_cache_read(const tks_cache *cache, const int32_t *slots, int32_t n, void *k_out,
                   void *v_out, int32_t dtype, void *stream);

/*
 * The queries of an attention call: bfloat16 [batch][tokens][q_heads][head_dim],
 * q_heads a multiple of kv_heads; query head h reads key/value head h /
 * (q_heads / kv_heads).  Position p of sequence b is token p % page_size of
 * page page_table[b * table_stride + p / page_size].  A position whose page is
 * outside [0, pages) counts as not attended and is reported as TKS_E_INDEX.
 * Sizes whose work cannot be counted in 32 bits (key/value heads times the
 * longest sequence's positions / 64, or sequences times heads, beyond 2^31)
 * return TKS_E_TOO_LARGE and launch nothing.
 */
typedef struct {
    const void *q;              /* 16-byte aligned; strides in elements, multiples of 8 */
    int64_t q_batch_stride, q_token_stride, q_head_stride;
    void *out;                  /* bfloat16 [batch][tokens][q_heads][head_dim], contiguous */
    float *lse;                 /* NULL, or [batch][tokens][q_heads]: the natural logarithm of
                                   the sum of exponentials of the attended, scaled scores */
    int32_t batch, tokens, q_heads;
    const int32_t *page_table;  /* int32 [batch][table_pages], row stride table_stride */
    int64_t table_stride;
    int32_t table_pages;
    float softmax_scale;        /* finite, and times log2(e), too: at most 2.3e38 */
} tks_queries;

/*
 * tks_tree_attention - attention of up to `tokens` drafted tokens of each
 * sequence over its cached context and over each other.  The drafted tokens'
 * own keys and values are in the cache already, draft j of sequence b at
 * position ctx_len[b] + j.
 *
 *   ctx_len    device, int32 [batch]: every query attends to positions
 *              [0, ctx_len[b])
 *   draft_len  device, int32 [batch], or NULL (all `tokens`): how many drafted
 *              tokens sequence b has; queries beyond attend to nothing
 *   tree       device, int32 [batch][tokens][ceil(tokens / 32)], or NULL (a
 *              chain: query i attends to drafts 0..i): query i attends to
 *              draft j < draft_len[b] where bit j % 32 of word j / 32 is set
 *
 * ctx_len is held to [0, table_pages * page_size] (a sequence has at most 2^31 -
 * 65536 positions), draft_len to [0, tokens] and to what is left of the page
 * table; a length that had to be changed is reported as TKS_E_ROW_LEN.  A query that attends to nothing gives zeros, and
 * -inf in lse.  What the cache holds where a query does not attend has no
 * influence on it, NaN and infinities included.  tokens <= TKS_DRAFTS_MAX;
 * tokens = 1 is the attention of an ordinary decode step.
 */
int tks_tree_attention(const tks_cache *cache, const tks_queries *queries,
                       const int32_t *ctx_len, const int32_t *draft_len, const int32_t *tree,
                       void *stream);

/*
 * tks_selected_attention - attention of each query token over its own list of
 * positions, the same for all its heads: indices[b][t][0..k), in any order, as
 * tks_topk_indices writes them.  Negative entries are skipped.  kv_len: device
 * int32 [batch], or NULL (table_pages * page_size): an entry at or beyond
 * kv_len[b] is skipped and reported as TKS_E_INDEX (kv_len itself is held to
 * [0, table_pages * page_size] and reported as TKS_E_ROW_LEN).  A position
 * that is listed twice counts twice.  A query whose list is empty gives zeros,
 * and -inf in lse.
 */
int tks_selected_attention(const tks_cache *cache, const tks_queries *queries,
                           const int32_t *indices, int32_t k, const int32_t *kv_len,
                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TKS_ATTENTION_H */
