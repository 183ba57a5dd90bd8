/*
 * tks_blocks.h - C ABI of libtks, third part: sparse attention by blocks, and
 * what is done with a cache's pages between steps (GB300, sm_103a).
 *
 * A sequence's block j is its positions [j * block, (j + 1) * block), `block` a
 * power of two.  tks_cache_bounds keeps, beside the cache of tks_attention.h,
 * the least and the largest value of each block's keys in every channel;
 * tks_block_scores makes of them, for every query token and key/value head, a
 * score of every block, which no key of the block exceeds (over 8 bits: but for the
 * bounds' rounding); the selector of tks.h
 * picks the best (rows of scores, with the row lengths that come with them); and
 * tks_block_attention attends to the blocks picked.
 *
 * The page calls work on page tables as the attention calls take them: a
 * sequence of n tokens holds the first ceil(n / page_size) entries of its row,
 * and a page that no sequence holds is free.  There is no other state: which
 * pages are free follows from the tables, so a sequence that is not carried over
 * to the next tables has thereby freed its pages.
 *
 * Status codes, streams, device-side errors and the ownership of buffers are
 * those of tks_attention.h.  So is the workspace of a stream, which of these
 * calls tks_block_attention alone uses for more than its status: graphs that
 * were captured on one stream share it, and those with that call (or another
 * attention call) in them must not run at the same time.
 */
#ifndef TKS_BLOCKS_H
#define TKS_BLOCKS_H

#include <stdint.h>

#include "tks_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The bounds of a cache's blocks. */
typedef struct {
    void *bounds;      /* bfloat16 [pages][page_size / block][kv_heads][2][head_dim], contiguous,
                          16-byte aligned: the least value of the block's keys in each channel, then the largest */
    int32_t block;     /* tokens of a block: a power of two, at most page_size */
    int32_t pages;     /* these four are the cache's */
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
} tks_bounds;

/*
 * tks_cache_bounds - the bounds of the blocks that the positions [start[b],
 * end[b]) of each sequence lie in.
 *
 *   bounds      sizes as the cache's
 *   page_table  device, int32 [batch][table_pages], row stride table_stride
 *   start       device, int32 [batch], or NULL (0): the first new position
 *   end         device, int32 [batch]: the sequence's length
 *
 * Each of these blocks is taken anew, from its own first position to the last
 * one below end[b], so that a call with start[b] the length before the last
 * tks_cache_write keeps them up to date; the others are left as they are.  A
 * value is the key as tks_cache_read gives it in 32 bits, held to the finite
 * range of bfloat16 and, at last, rounded to it; a channel with a NaN has NaN
 * bounds.  start and end are held to [0, table_pages * page_size] and reported
 * as TKS_E_ROW_LEN; a block whose page is outside [0, pages) is skipped and
 * reported as TKS_E_INDEX.  Where sequences of the call hold a page at the same
 * place of their rows and end differently within a block of it, the block is taken
 * up to the furthest of their ends, whichever of them has new positions there, so
 * that its bounds hold for all of them.  (A page at different places of rows, in
 * blocks that their sequences do not fill alike, has no such order: its bounds
 * there are undefined.)
 */
int tks_cache_bounds(const tks_cache *cache, const tks_bounds *bounds, const int32_t *page_table,
                     int64_t table_stride, int32_t table_pages, int32_t batch,
                     const int32_t *start, const int32_t *end, void *stream);

/*
 * tks_block_scores - for query token t of sequence b, key/value head g and
 * block j that the token sees,
 *     scores[b][t][g][j] = max over the query heads h of g of
 *         sum over the channels d of max(q_h,d * least_j,d, q_h,d * largest_j,d)
 * (as sum of max(q, 0) * largest + min(q, 0) * least, in 32 bits), which, but for
 * the sum's rounding, is at least the product of any of these heads with any finite
 * key of the block in a bfloat16 cache.  Over 8 bits, bounds are rounded to nearest,
 * and a key's product can exceed its block's score by up to 2^-8 of
 * sum |q_d| max(|least_d|, |largest_d|).
 *
 *   queries   out, lse and softmax_scale are not looked at
 *   kv_len    device, int32 [batch][tokens], or NULL (n * block): the token
 *             sees positions below it, so the blocks below ceil(kv_len / block)
 *   first, last  that many of the blocks that a token sees, from its first and
 *             up to its last one, score +inf: they are always picked
 *   scores    float32 [batch][tokens][kv_heads][n]; blocks that a token does
 *             not see score -inf
 *   n         blocks of a row of scores, at most table_pages * page_size / block
 *   row_len   NULL, or int32 [batch][tokens][kv_heads]: how many blocks the
 *             token sees, as tks_topk_indices takes it
 *
 * kv_len is held to [0, n * block] and reported as TKS_E_ROW_LEN.  A block
 * whose page is outside [0, pages) scores -inf and is reported as TKS_E_INDEX.  A
 * score that is not a number becomes +inf, so that a key that is none is
 * attended to, as it would be without a selection.  Where tokens * q_heads /
 * kv_heads is more than 16, waits inside the kernel are bounded, as those of the
 * attention calls are (TKS_E_TIMEOUT; scores are then undefined).  Sizes that cannot be
 * counted in 32 bits (batch * tokens * kv_heads, or batch * n / 8) return
 * TKS_E_TOO_LARGE.  Work follows kv_len for up to 1024 sequences, or, where there
 * are more than 16 rows (as above), tiles of tokens (of 256 / group, the group being
 * q_heads / kv_heads filled up to a power of two; 2 from 128 on); beyond, all n
 * blocks are read for every token, whatever it sees, so that n is better no larger
 * than the longest sequence needs.
 */
int tks_block_scores(const tks_bounds *bounds, const tks_queries *queries, const int32_t *kv_len,
                     int32_t first, int32_t last, float *scores, int32_t n, int32_t *row_len,
                     void *stream);

/*
 * tks_block_attention - attention of each query token and key/value head over
 * its own list of blocks: blocks[b][t][g][0..n), in any order, as
 * tks_topk_indices writes them.  Negative entries are skipped.  Of a block, the
 * positions below kv_len[b][t] are attended to (kv_len: device int32
 * [batch][tokens], or NULL: table_pages * page_size); a block that starts at or
 * beyond it is skipped and reported as TKS_E_INDEX.  kv_len itself is held to
 * [0, table_pages * page_size] and reported as TKS_E_ROW_LEN.  A block that is
 * listed twice counts twice.  A query without a position gives zeros, and -inf in
 * lse.  `block` is a power of two and need not go with the pages; n * block is
 * at most TKS_K_MAX.
 */
int tks_block_attention(const tks_cache *cache, const tks_queries *queries, const int32_t *blocks,
                        int32_t n, int32_t block, const int32_t *kv_len, void *stream);

/* Elements of the scratch buffer of a page call (int32, device, 16-byte aligned; what
 * it holds before the call does not matter; calls that may run at the same time need
 * one each). */
#define TKS_PAGES_SCRATCH(pages, rows) (2 * (int64_t)(pages) + (int64_t)(rows) + 1056)

/*
 * tks_cache_fork - the page tables of the next step's sequences, each a
 * continuation of one of this step's, or a new one: how sequences grow, end,
 * branch and are reordered.
 *
 *   page_table  device, int32 [sequences][table_pages], row stride table_stride
 *   lens        device, int32 [sequences]
 *   parents     device, int32 [children]: the sequence that child i goes on
 *               from, or a negative number: from nothing
 *   new_lens    device, int32 [children]: the length that child i is to have
 *               pages for; below its parent's, it is cut to that
 *   keep        device, uint8 [pages], or NULL: pages that are held outside
 *               the tables where not 0 (they are not handed out, nor written to)
 *   pages, page_size  the cache's
 *   table       int32 [children][table_pages], contiguous: the children's
 *               pages, -1 behind the last.  Must not overlap page_table
 *   src, dst    int32 [children]: the page that is to be copied for child i,
 *               and where to (tks_cache_copy), or -1 and -1
 *   scratch     int32 [TKS_PAGES_SCRATCH(pages, children)]
 *
 * A child keeps its parent's pages as far as both lengths reach.  It is going to
 * write to the last of these if that is partly filled and new_lens[i] lies
 * beyond; if another child holds that page too, or `keep` does, it gets a copy,
 * but the page stays with the lowest of the children that hold it if all of them
 * are going to write to it and `keep` does not hold it.  Free pages (those that
 * neither a child nor `keep` holds) go, lowest first, to the children in order,
 * first for the copy, then for the positions behind.  When none is left, entries
 * (src and dst too) are -1, reported as TKS_E_NO_PAGE.  Copies read pages that
 * are held and write pages that were free.
 *
 * Lengths are held to [0, table_pages * page_size] and reported as
 * TKS_E_ROW_LEN; a parent beyond the sequences counts as none, and an entry
 * outside [0, pages) is carried over as it is, both reported as TKS_E_INDEX.
 */
int tks_cache_fork(const int32_t *page_table, int64_t table_stride, int32_t table_pages,
                   int32_t sequences, const int32_t *lens, const int32_t *parents,
                   const int32_t *new_lens, int32_t children, const uint8_t *keep, int32_t pages,
                   int32_t page_size, int32_t *table, int32_t *src, int32_t *dst,
                   int32_t *scratch, void *stream);

/*
 * tks_cache_compact - moves what is in use to the lowest pages.  Let u be the
 * number of pages that a sequence or `keep` holds.  The i-th held page at or
 * beyond u (in order; those of `keep` stay where they are) goes to the i-th
 * page below u that is not held.
 *
 *   table       int32 [sequences][table_pages], contiguous: the sequences'
 *               pages afterwards, -1 behind the last.  May be page_table itself
 *               (if that is contiguous), else must not overlap it
 *   src, dst    int32 [pages / 2]: the moves, in order, then -1
 *   count       int32 [2]: the number of moves, and u
 *   scratch     int32 [TKS_PAGES_SCRATCH(pages, sequences)]
 *   (the others as for tks_cache_fork)
 */
int tks_cache_compact(const int32_t *page_table, int64_t table_stride, int32_t table_pages,
                      int32_t sequences, const int32_t *lens, const uint8_t *keep, int32_t pages,
                      int32_t page_size, int32_t *table, int32_t *src, int32_t *dst,
                      int32_t *count, int32_t *scratch, void *stream);

/*
 * tks_cache_copy - copies pages src[i] to dst[i], i < n: keys, values, scales
 * where the cache has them, and bounds where given (NULL: none).
 *
 *   src, dst  device, int32 [n]; a pair with a negative page is none, one with
 *             a page at or beyond `pages` is skipped and reported as TKS_E_INDEX.
 *             A page that is in dst twice, or in src and dst, is undefined afterwards
 *   count     NULL, or device int32: only the pairs before it are looked at
 */
int tks_cache_copy(const tks_cache *cache, const tks_bounds *bounds, const int32_t *src,
                   const int32_t *dst, int32_t n, const int32_t *count, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TKS_BLOCKS_H */
