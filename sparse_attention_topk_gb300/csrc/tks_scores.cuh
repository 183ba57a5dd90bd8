// What the kernels that score blocks share.
#pragma once

#include "tks_attn.cuh"

namespace tks {
namespace attn {

struct ScoreParams {
  const __nv_bfloat16* bounds;
  int pages, block_shift, of_page_shift, kv_heads;  // of_page_shift: log2 of the blocks of a page
  const __nv_bfloat16* q;
  long long q_batch, q_token, q_head;
  int batch, tokens;
  int group, group_all, first_of_group;  // query heads of a key/value head: those of this launch, all, and where they begin
  const int32_t* table;
  long long table_stride;
  const int32_t* kv_len;
  int first, last;
  float* out;
  int n;
  int32_t* row_len;
  unsigned* status;
  bool stream_out;                     // scores are more than stay in L2
  bool join;                           // the largest of this launch's heads and of what is there
  int tile_tokens, token_tiles;        // tokens of a tile of query rows, and how many tiles a sequence has
  int chunks;                          // few rows: thread blocks of a unit
  int group_room;                      // many rows: columns of a token, a power of two,
  int half_rows, half_tokens;          // columns of half a tile, and tokens
  long long spin_limit_ns;
  int test_skip_arrive;
};

// The blocks that a token sees, of n.
__device__ __forceinline__ int blocks_seen(const ScoreParams& p, int b, int t, bool& bad) {
  if (!p.kv_len) return p.n;
  const int given = __ldg(p.kv_len + (long long)b * p.tokens + t);
  const long long most = (long long)p.n << p.block_shift;
  const int len = given < 0 ? 0 : given > most ? (int)most : given;
  bad |= len != given;
  return (int)(((long long)len + (1 << p.block_shift) - 1) >> p.block_shift);
}
__device__ __forceinline__ float final_score(const ScoreParams& p, float x, int j, int seen) {
  if (j >= seen) return -INFINITY;
  return !(x == x) || j < p.first || j >= seen - p.last ? INFINITY : x;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Two bfloat16's positive parts, or their negative ones. (A NaN stays one in either.)
__device__ __forceinline__ uint32_t part_of_pair(uint32_t w, bool positive) {
  const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w), zero = __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 y = positive ? __hmax2_nan(x, zero) : __hmin2_nan(x, zero);
  return *reinterpret_cast<const uint32_t*>(&y);
}
// The first element of a token's query of head g of this launch.
__device__ __forceinline__ const __nv_bfloat16* score_query(const ScoreParams& p, int b, int t, int head, int g) {
  return p.q + b * p.q_batch + t * p.q_token + ((long long)head * p.group_all + p.first_of_group + g) * p.q_head;
}

cudaError_t setup_scores();  // the kernel for few query rows (tks_blocks.cu)

// The kernel for many query rows (tks_scores_tiles.cu).
constexpr int kScoreTileRows = 256;  // query rows of a tile, in two halves
constexpr int kScoreTileBlocks = 128;
cudaError_t setup_score_tiles();
cudaError_t launch_score_tiles(const ScoreParams& p, int head_dim, int sms, cudaStream_t stream);

}  // namespace attn
}  // namespace tks
