// Internal interface between the cache and attention translation units of
// libtks (not part of the C ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tks {
namespace attn {

// Status bits of the workspace's first word.
constexpr unsigned kStatTimeoutBit = 1u << 0;
constexpr unsigned kStatRowLenBit = 1u << 1;
constexpr unsigned kStatIndexBit = 1u << 3;
constexpr unsigned kStatNoPageBit = 1u << 4;

// Most positions of a sequence: indices of keys stay below 2^31 with a tile to spare.
constexpr int kMaxPositions = 0x7fff0000;

// Most keys that an output is summed over in one go. The matrix instructions add products to a 32-bit
// accumulator whose small ones, below 2^-24 of it, are dropped: of a flat tail of weights behind a
// dominant one, n * 2^-24 at most. A longer run of a unit's keys is summed in pieces, joined as the
// partials of blocks are; at 32,768 the dropped part is 2^-9 at most, half a step of the bfloat16 output,
// and the pieces cost 0.3 to 2.4 % (304 sequences of 65,536 positions of int8 and one token of 4 heads
// 846 us, in one go 843; 152 of 131,072 and 32 rows 1351 and 1325; 152 of 65,536 and 128 rows 802 and
// 784).
constexpr int kPieceKeys = 32768;

// Arguments of the cache kernels.
struct CacheParams {
  unsigned char *k, *v;
  float* scales;
  long long page_b, token_b, head_b;  // strides of the cache in bytes
  int page_shift, kv_heads;
  int head_shift;  // log2 of kv_heads where it is a power of two, else -1
  int slots_held;  // pages * page_size
  const int32_t* slots;
  int n;
  const void *src_k, *src_v;                   // write: rows to put in,
  long long k_token, k_head, v_token, v_head;  // and their strides in elements
  void *out_k, *out_v;                         // read: where rows go
  unsigned* status;
};
cudaError_t launch_cache_write(const CacheParams& p, int head_dim, bool i8, bool f32, cudaStream_t s);
cudaError_t launch_cache_read(const CacheParams& p, int head_dim, bool i8, bool f32, cudaStream_t s);

// A segment costs a block as much as this many tiles, beside its own.
constexpr int kSegmentTiles = 6;

// How W tiles are split over G blocks.
struct Split {
  long long W;
  unsigned share;  // blocks of a unit (even shares), or 0 (one run)
  unsigned q, r;   // one run: tiles of a block, q or, for the first r blocks, q + 1
  unsigned step;   // (lists of blocks: times this; 0: 1)

  __host__ __device__ void set(long long w, unsigned longest, long long units, int G) {
    W = w;
    if (w >> 31) {
      q = (unsigned)(w / G);
      r = (unsigned)(w % G);
    } else {
      q = (unsigned)w / (unsigned)G;
      r = (unsigned)w - q * (unsigned)G;
    }
    share = 0;
    if (units <= G) {
      const unsigned s = (unsigned)G / (unsigned)units;
      if ((longest + s - 1) / s <= q + (r > 0) + kSegmentTiles) share = s;
    }
  }
  __host__ __device__ long long start(int c) const { return (long long)c * q + ((unsigned)c < r ? (unsigned)c : r); }
  // One run: the block that holds tile w.
  __host__ __device__ int block_of(long long w) const {
    const long long more = (long long)r * (q + 1);
    if (w < more) return W >> 31 ? (int)(w / (q + 1)) : (int)((unsigned)w / (q + 1));
    return (int)r + (W >> 31 ? (int)((w - more) / q) : (int)((unsigned)(w - more) / q));
  }
};

// Arguments of the attention kernels.
struct Params {
  const unsigned char *k, *v;
  const float2* scales;
  long long page_b, token_b, head_b;  // strides of the cache in bytes
  int pages, page_shift, kv_heads;
  const __nv_bfloat16* q;
  long long q_batch, q_token, q_head;  // elements
  __nv_bfloat16* out;
  float* lse;
  int batch, tokens, q_heads, group;
  const int32_t* table;
  long long table_stride;
  int table_pages;
  const int32_t *ctx_len, *draft_len, *tree;  // tree attention
  int tree_words;
  const int32_t *indices, *kv_len;  // selected attention: lists, and the lengths that their entries keep to,
  int k_sel;                        // and the keys of a list
  bool blocks;                      // attention over blocks: lists of blocks, one for each head, and lengths of tokens
  int block_shift;                  // log2 of a block's keys
  long long list_seq;               // a list's stride in entries, from token to token
  int list_head;                    // and from head to head
  float scale_log2;  // softmax_scale * log2(e)
  int seqs;          // tree: batch; selected: batch * tokens
  int rows;          // query rows of one (sequence, head)
  int row_tiles;
  unsigned* status;
  float* parts;
  int cluster;  // > 0: the blocks of a unit are one thread-block cluster of this size, which joins itself
  Split* plan;  // trees: the split, for the kernel that joins
  Split split;  // selected, and clusters: the split
  long long spin_limit_ns;
  int test_skip_arrive;
};

// Blocks of a cluster at most. (Clusters of 16 start later: one token over 2048 selected positions
// takes 10.6 us with them and 9.0 with 8.)
constexpr int kClusterMax = 8;

// The kernels for few rows (16 a block; mma.sync).
constexpr int kRowsTile = 16;  // query rows of a block
constexpr int kRowsKeys = 64;  // keys of a tile
constexpr int kRowsBlocksPerSm = 2;
// Whether a list's blocks, and the pages, are at least as long as the chunks (32 keys of int8, 16 of bfloat16) that warps take.
inline bool blocks_by_chunks(const Params& p, bool i8) {
  const int chunk = i8 ? 5 : 4;
  return p.blocks && p.block_shift >= chunk && p.page_shift >= chunk;
}
// Lists of bfloat16 blocks that together are longer than the sequence come from L2, which answers sooner than memory: more
// warps with less under way each (512 tokens of 64 heads on 4 over 32 blocks of 64: 228 us so, some 255 otherwise). Of memory,
// or in 8 bits, they do not help (64 tokens over 64 blocks of int8 of 8 heads: 156 us so, 125 otherwise; the former in int8
// 199 and 198).
constexpr int kRowsManyPerSm = 3;
inline bool rows_many(const Params& p, bool i8) {
  return !i8 && blocks_by_chunks(p, i8) && (long long)p.tokens * p.k_sel >= (long long)p.table_pages << p.page_shift;
}
cudaError_t setup_rows();
cudaError_t launch_rows(const Params& p, int head_dim, bool i8, bool selected, int grid,
                        cudaStream_t stream);

// The kernels for many rows (128 a block, one block an SM; tcgen05).
constexpr int kTilesRows = 128;
constexpr int kTilesKeys = 128;
cudaError_t setup_tiles();
cudaError_t setup_tiles_bf16();  // (tks_attn_tiles_bf16.cu, called by setup_tiles and launch_tiles)
cudaError_t launch_tiles_bf16(const Params& p, int head_dim, bool selected, int grid, cudaStream_t stream);
cudaError_t launch_tiles(const Params& p, int head_dim, bool i8, bool selected, int grid,
                         cudaStream_t stream);

}  // namespace attn

// The time limit of device-side waits, and the test option that makes one run
// out (tks_set_option; host side, tks_select.cu).
long long spin_limit_ns();
int test_skip_arrive();

// The workspace of the cache and attention calls on a stream: a status word
// (256 bytes) and the partial results.  Host side, tks_attn.cu.
int attn_status(int dev, void* stream);  // a tks_status; the stream has been synchronised
int attn_release();

}  // namespace tks
