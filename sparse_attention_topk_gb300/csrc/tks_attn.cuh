// Shared parts of the attention kernels: their parameters, how work is split
// over blocks, where a key lives in the paged cache, and PTX helpers.
//
// Work is counted in tiles of keys.  A unit is (sequence, key/value head, tile
// of query rows); its tiles are the keys that its rows attend to.  All units'
// tiles, in order, form one axis of W tiles, and block c of G takes tiles
// [W*c/G, W*(c+1)/G): every block has the same work however ragged the
// sequences are, a long unit is split over many blocks and short ones share a
// block.  A block that holds all of a unit writes its output; otherwise it
// writes a partial result (unnormalised output, running maximum, sum) to its
// slot of the workspace and combine_kernel joins the unit's partials in block
// order, so results do not depend on timing.  A block has at most two partial
// segments, its first (slot 0) and its last (slot 1).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tks_attn_internal.h"

namespace tks {
namespace attn {

// ---------------------------------------------------------------------------
// PTX helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// 16- and 8-byte asynchronous copies to shared memory; bytes = 0 writes zeros
// and reads nothing.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Two codes as a pair of halves, exactly: `biased` holds codes + 128 as bytes
// (code ^ 0x80), a byte u under the exponent 0x64 is 1024 + u, and 1152 is
// taken off again.  SEL picks the bytes: 0x4140 the lower two, 0x4342 the upper.
template <int SEL>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t biased) {
  const uint32_t u = __byte_perm(biased, 0x64646464u, SEL);
  const uint32_t c = 0x64806480u;  // 1152, twice
  __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<uint32_t*>(&r);
}

// ---------------------------------------------------------------------------
// Lengths and positions
// ---------------------------------------------------------------------------
struct Seq {
  int ctx;     // positions every row attends to (selected: entries of the list)
  int drafts;  // drafted tokens behind them (selected: 0)
  int len;     // ctx + drafts
};

__device__ __forceinline__ void report(unsigned* status, unsigned bit) { atomicOr(status, bit); }

// The number of positions that a page table row can name.
__device__ __forceinline__ int capacity(const Params& p) {
  const long long room = (long long)p.table_pages << p.page_shift;
  return room > kMaxPositions ? kMaxPositions : (int)room;
}

template <bool SEL>
__device__ __forceinline__ Seq seq_of(const Params& p, int s) {
  Seq q;
  if (SEL) {
    q.ctx = p.k_sel;
    q.drafts = 0;
    q.len = p.k_sel;
    return q;
  }
  const int cap = capacity(p);
  const int c = p.ctx_len[s], d = p.draft_len ? p.draft_len[s] : p.tokens;
  q.ctx = min(max(c, 0), cap);
  q.drafts = min(min(max(d, 0), p.tokens), cap - q.ctx);
  q.len = q.ctx + q.drafts;
  if (q.ctx != c || q.drafts != d) report(p.status, kStatRowLenBit);
  return q;
}

// The number of positions that a list's entries may name.
__device__ __forceinline__ int kv_limit(const Params& p, int b) {
  const int cap = capacity(p);
  if (!p.kv_len) return cap;
  const int n = p.kv_len[b], r = min(max(n, 0), cap);
  if (r != n) report(p.status, kStatRowLenBit);
  return r;
}

// Tiles of TK keys of a unit; at least one, so that every unit is visited.
template <int TK>
__device__ __forceinline__ int tiles_of(int len) {
  return len <= TK ? 1 : (int)(((unsigned)len + TK - 1) / TK);
}

// First tile of block c, and the block that holds tile w.
__device__ __forceinline__ long long block_start(long long W, int c, int G) { return W * c / G; }
__device__ __forceinline__ int block_of(long long W, long long w, int G) {
  return (int)((G * (w + 1) - 1) / W);
}

// Where a block starts: filled by warp 0, read by all after a barrier.
struct Start {
  long long total;  // W
  long long cum;    // first tile of sequence `seq`
  int seq;
};

// All tiles of all sequences, and the sequence that holds tile `w` (w is
// given as block index times total over blocks).  Called by one warp.
template <bool SEL, int TK>
__device__ __forceinline__ void find_start(const Params& p, int block, int blocks, Start* st) {
  const int lane = threadIdx.x & 31;
  const long long per = (long long)p.kv_heads * p.row_tiles;
  if (SEL) {
    const long long each = per * tiles_of<TK>(p.k_sel);
    const long long W = each * p.seqs, w = block_start(W, block, blocks);
    if (lane == 0) {
      st->total = W;
      st->seq = (int)(w / each);
      st->cum = (w / each) * each;
    }
    return;
  }
  long long sum = 0;
  for (int s = lane; s < p.seqs; s += 32) sum += tiles_of<TK>(seq_of<SEL>(p, s).len);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const long long W = sum * per, w = block_start(W, block, blocks);
  long long base = 0;
  for (int s0 = 0; s0 < p.seqs; s0 += 32) {
    const int s = s0 + lane;
    const long long mine = s < p.seqs ? per * tiles_of<TK>(seq_of<SEL>(p, s).len) : 0;
    long long end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    end += base;
    const unsigned m = __ballot_sync(0xffffffffu, s < p.seqs && w < end);
    if (m) {
      if (lane == __ffs(m) - 1) {
        st->total = W;
        st->seq = s;
        st->cum = end - mine;
      }
      return;
    }
    base = __shfl_sync(0xffffffffu, end, 31);
  }
  if (lane == 0) {  // an empty tail: no tile of this block's
    st->total = W;
    st->seq = p.seqs;
    st->cum = W;
  }
}

// Whether query row t sees drafted token j.
__device__ __forceinline__ bool sees_draft(const Params& p, int b, int t, int j) {
  if (!p.tree) return j <= t;
  const int w = p.tree[((long long)b * p.tokens + t) * p.tree_words + (j >> 5)];
  return (w >> (j & 31)) & 1;
}

// The place of query row R of a unit among the rows of out and lse.
template <bool SEL>
__device__ __forceinline__ long long out_row(const Params& p, int seq, int head, int R) {
  const long long token = SEL ? seq : (long long)seq * p.tokens + R / p.group;
  return token * p.q_heads + (long long)head * p.group + (SEL ? R : R % p.group);
}
// The first element of that row's query.
template <bool SEL>
__device__ __forceinline__ const __nv_bfloat16* q_row(const Params& p, int seq, int head, int R) {
  const int b = SEL ? seq / p.tokens : seq, t = SEL ? seq % p.tokens : R / p.group;
  const int h = head * p.group + (SEL ? R : R % p.group);
  return p.q + b * p.q_batch + t * p.q_token + h * p.q_head;
}

// Floats of a partial slot: ROWS x D of output, then ROWS pairs (maximum, sum).
template <int ROWS, int D>
constexpr int kPartFloats = ROWS * (D + 2);

}  // namespace attn
}  // namespace tks
