// Shared parts of the attention kernels: their parameters, how work is split
// over blocks, where a key lives in the paged cache, and PTX helpers.
//
// Work is counted in tiles of keys.  A unit is (sequence, key/value head, tile
// of query rows); its tiles are the keys that its rows attend to.  Two ways:
//  * even shares: every unit is split over the same number of blocks.  A block
//    has one segment of one unit.
//  * one run: all units' tiles, in order, form one axis, and every block takes an
//    equal run of it, whatever units it crosses: every block has the same work
//    however ragged the sequences are.
// Starting a segment costs a block as much as kSegmentTiles tiles (lookups and
// queries come first, and the joining and the output last), so even shares are
// taken where the longest of them is not longer than an equal run and that (one
// token over 16,384 positions of 8 heads: 19.6 us as a run, 17.0 in even shares;
// 8 drafts of it over 8,000 21.4 and 16.7; one over 8,000 of 4 heads of bfloat16
// 13.3 and 13.4).
// A block that holds all of a unit writes its output; otherwise it writes a
// partial result (unnormalised output, running maximum, sum) to its slot of the
// workspace, and the unit's partials are joined in block order, so results do
// not depend on timing.  A block has at most two partial segments, its first
// (slot 0) and its last (slot 1).  (A long run's pieces meet in these slots, too.)  Where shares are even and short (the host can
// tell from the list's or the page table's length), the blocks of a unit are a
// thread-block cluster: they leave their partials in their shared memory, and
// join them from there without another kernel (one token over 2048 selected
// positions: 10.8 us with the other kernel, 9.3 as clusters).
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
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
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
// Two weights as sums of two bfloat16 each: `first`, cut off a little below the weight, and what is
// left, rounded. Both parts of a positive weight are positive, so that an infinite value times
// them is that infinity.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& first, uint32_t& rest) {
  const uint32_t x = __float_as_uint(a * 0.99609375f), y = __float_as_uint(b * 0.99609375f);
  first = __byte_perm(x, y, 0x7632);
  rest = pack_bf16(a - __uint_as_float(x & 0xffff0000u), b - __uint_as_float(y & 0xffff0000u));
}

// Weights are 2^(x - m), m near a row's running maximum: when that has grown to more than this and 8
// beyond m, m becomes the maximum less this. Over 8 bits weights go into the products as halves, so with
// 11 bits down to 2^-14, in steps of 2^-24 below, and up to 2^16: with the largest at 2^7 to 2^15, a
// weight is off by 2^-11 of itself or by 2^-32 of the largest. (With the largest at 1 to 2^8, those below
// 2^-25 of it were 0 in the output, and not in the sum: a flat tail of 2^20 keys behind a dominant one
// lost the 2.7 % that it is of the row.) Weights over bfloat16 have the range of 32 bits.
template <bool I8>
constexpr float kWeightLog2 = I8 ? 7.f : 0.f;

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

// (lengths out of range are reported by the warps that read all of them: make_split)
template <bool SEL>
__device__ __forceinline__ Seq seq_of(const Params& p, int s, bool* bad = nullptr) {
  Seq q;
  if (SEL) {
    q.ctx = p.k_sel;
    q.drafts = 0;
    q.len = p.k_sel;
    return q;
  }
  const int cap = capacity(p);
  const int c = __ldg(p.ctx_len + s), d = p.draft_len ? __ldg(p.draft_len + s) : p.tokens;
  q.ctx = min(max(c, 0), cap);
  q.drafts = min(min(max(d, 0), p.tokens), cap - q.ctx);
  q.len = q.ctx + q.drafts;
  if (bad) *bad |= q.ctx != c || q.drafts != d;
  return q;
}

// Lists of positions, or (BLK) of blocks. (Lists of positions as blocks of one: one token over 2048 of them takes 9.65 us
// instead of 9.2, 512 of 64 heads 103.8 instead of 101.6.)
// The list of a token (seq) and head.
template <bool BLK>
__device__ __forceinline__ const int32_t* list_of(const Params& p, int seq, int head) {
  return BLK ? p.indices + seq * p.list_seq + (long long)head * p.list_head : p.indices + (long long)seq * p.k_sel;
}
// The place of key j's entry in a list.
template <bool BLK>
__device__ __forceinline__ int list_entry(const Params& p, int j) { return BLK ? j >> p.block_shift : j; }
// The position of key j of a list, given its entry, or -1.
template <bool BLK>
__device__ __forceinline__ int list_position(const Params& p, int entry, int j, int limit, bool& bad) {
  if (!BLK) {
    bad |= entry >= limit;
    return entry >= limit ? -1 : entry;
  }
  if (entry < 0) return -1;
  if (entry > (0x7fffffff >> p.block_shift) || entry << p.block_shift >= limit) {
    bad = true;
    return -1;
  }
  const int pos = entry << p.block_shift | (j & ((1 << p.block_shift) - 1));
  return pos >= limit ? -1 : pos;  // (a block may reach beyond the length)
}

// The number of positions that a list's entries may name; `given`: kv_len of the sequence (or token), or INT_MAX.
template <bool BLK>
__device__ __forceinline__ int kv_given(const Params& p, int b, int seq) { return p.kv_len ? __ldg(p.kv_len + (BLK ? seq : b)) : 0x7fffffff; }
__device__ __forceinline__ int kv_limit(const Params& p, int given) {
  const int r = min(max(given, 0), capacity(p));
  if (r != given && p.kv_len) report(p.status, kStatRowLenBit);
  return r;
}

// Tiles of TK keys of a unit; at least one, so that every unit is visited.
template <int TK>
__device__ __forceinline__ int tiles_of(int len) {
  return len <= TK ? 1 : (int)(((unsigned)len + TK - 1) / TK);
}

// The split, for all lanes of a warp, and the lengths of sequence `lane`. Selected: the host has made
// it. Trees: it depends on the lengths, and block 0 leaves it for the kernel that joins.
template <bool SEL, int TK>
__device__ __forceinline__ Split make_split(const Params& p, Seq& mine) {
  if (SEL || p.cluster) {
    if (SEL) mine = seq_of<SEL>(p, 0);
    return p.split;
  }
  const int lane = threadIdx.x & 31;
  const unsigned per = (unsigned)(p.kv_heads * p.row_tiles);
  bool bad = false;
  mine.ctx = mine.drafts = mine.len = 0;
  if (lane < p.seqs) mine = seq_of<SEL>(p, lane, &bad);
  unsigned longest = lane < p.seqs ? (unsigned)tiles_of<TK>(mine.len) : 0;
  long long sum = longest;
  for (int s = lane + 32; s < p.seqs; s += 32) {
    const unsigned t = (unsigned)tiles_of<TK>(seq_of<SEL>(p, s, &bad).len);
    sum += t;
    longest = max(longest, t);
  }
  if (p.seqs > 1) {
    longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  } else {
    longest = __shfl_sync(0xffffffffu, longest, 0);
    sum = longest;
  }
  Split split;
  split.set(sum * per, longest, (long long)per * p.seqs, gridDim.x);
  if (blockIdx.x == 0) {
    if (bad) report(p.status, kStatRowLenBit);
    if (lane == 0) *p.plan = split;
  }
  return split;
}

// Where a block starts: filled by one warp, read by all after a barrier.
struct Start {
  int seq;        // the sequence of the block's first tile
  unsigned rel;   // the tile's number among the sequence's (they fit: the host checks)
  unsigned left;  // the block's tiles
  Seq len;        // of that sequence
};

template <bool SEL, int TK>
__device__ __forceinline__ void find_start(const Params& p, Start* st) {
  const int lane = threadIdx.x & 31, block = blockIdx.x;
  const unsigned per = (unsigned)(p.kv_heads * p.row_tiles);
  Seq mine;
  const Split split = make_split<SEL, TK>(p, mine);
  if (split.share) {
    const unsigned unit = (unsigned)block / split.share, i = (unsigned)block - unit * split.share;
    const unsigned seq = unit / per, in = unit - seq * per;
    Seq len = mine;
    if (!SEL && p.cluster) {
      bool bad = false;
      len.ctx = len.drafts = len.len = 0;
      if (seq < (unsigned)p.seqs) len = seq_of<SEL>(p, (int)seq, &bad);
      if (bad && lane == 0) report(p.status, kStatRowLenBit);
    } else if (!SEL) {
      if (seq < 32) {
        len.ctx = __shfl_sync(0xffffffffu, mine.ctx, (int)seq);
        len.drafts = __shfl_sync(0xffffffffu, mine.drafts, (int)seq);
        len.len = len.ctx + len.drafts;
      } else if (seq < (unsigned)p.seqs) {
        len = seq_of<SEL>(p, (int)seq);
      }
    }
    if (lane == 0) {
      st->seq = (int)seq;
      st->rel = st->left = 0;
      st->len = len;
      const unsigned tiles = (unsigned)tiles_of<TK>(len.len), n = min(split.share, tiles);
      if (seq < (unsigned)p.seqs && i < n) {
        const unsigned tq = tiles / n, tr = tiles - tq * n;
        st->rel = in * tiles + i * tq + min(i, tr);
        st->left = tq + (i < tr ? 1 : 0);
      }
    }
    return;
  }
  long long w = split.start(block);
  unsigned left = split.q + ((unsigned)block < split.r ? 1 : 0);
  if (SEL && split.step) {  // (whole units)
    w *= split.step;
    left *= split.step;
  }
  if (SEL) {
    if (lane == 0) {
      const unsigned each = per * (unsigned)tiles_of<TK>(p.k_sel);
      st->seq = w >> 31 ? (int)(w / each) : (int)((unsigned)w / each);
      st->rel = (unsigned)(w - (long long)st->seq * each);
      st->left = left;
      st->len = mine;
    }
    return;
  }
  long long base = 0;
  for (int s0 = 0; s0 < p.seqs; s0 += 32) {
    const int s = s0 + lane;
    if (s0 > 0 && s < p.seqs) mine = seq_of<SEL>(p, s);
    const long long tiles = s < p.seqs ? (long long)per * tiles_of<TK>(mine.len) : 0;
    long long end = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    end += base;
    const unsigned m = __ballot_sync(0xffffffffu, s < p.seqs && w < end);
    if (m) {
      if (lane == __ffs(m) - 1) {
        st->seq = s;
        st->rel = (unsigned)(w - (end - tiles));
        st->left = left;
        st->len = mine;
      }
      return;
    }
    base = __shfl_sync(0xffffffffu, end, 31);
  }
  if (lane == 0) {  // past the last tile: a block without work
    st->seq = p.seqs;
    st->rel = st->left = 0;
  }
}

// A block's segments: runs of tiles of one unit, or pieces of them.
struct Segment {
  int seq, head, row_tile, b;
  int t0, t1, tiles;  // tiles [t0, t1) of the unit's
  int from;           // where the block's run of the unit begins: t0, or in a piece before
  bool first;         // of the block's runs
  bool more;          // the run goes on behind this piece
  Seq len;
  __device__ __forceinline__ bool whole() const { return from == 0 && t1 == tiles; }  // (the last piece)
  __device__ __forceinline__ bool goes_on() const { return from != t0; }              // pieces came before
};
template <bool SEL, int TK>
struct Segments {
  unsigned left, rel;
  int seq;
  Seq len0;  // of the first segment's sequence
  bool first, more;
  int from;
  __device__ __forceinline__ void begin(const Start& st) {
    left = st.left;
    rel = st.rel;
    seq = st.seq;
    len0 = st.len;
    first = true;
    more = false;
  }
  __device__ __forceinline__ bool next(const Params& p, Segment& s) {
    if (left == 0) return false;
    s.len = first ? len0 : seq_of<SEL>(p, seq);
    const unsigned tiles = (unsigned)tiles_of<TK>(s.len.len);
    const unsigned unit = rel / tiles, t0 = rel - unit * tiles, run = min(tiles - t0, left), n = min(run, (unsigned)(kPieceKeys / TK));
    s.seq = seq;
    s.b = SEL ? seq / p.tokens : seq;
    s.head = TK == kRowsKeys ? (int)unit : (int)(unit / (unsigned)p.row_tiles);  // (few rows: one tile)
    s.row_tile = TK == kRowsKeys ? 0 : (int)(unit - (unsigned)s.head * p.row_tiles);
    if (!more) from = (int)t0;
    more = n < run;
    s.from = from;
    s.t0 = (int)t0;
    s.t1 = (int)(t0 + n);
    s.tiles = (int)tiles;
    s.first = first;
    s.more = more;
    first = first && more;
    left -= n;
    rel += n;
    if (rel == tiles * (unsigned)(p.kv_heads * p.row_tiles)) {
      rel = 0;
      ++seq;
    }
    return true;
  }
};

// Whether query row t sees drafted token j.
__device__ __forceinline__ bool sees_draft(const Params& p, int b, int t, int j) {
  if (!p.tree) return j <= t;
  const int w = p.tree[((long long)b * p.tokens + t) * p.tree_words + (j >> 5)];
  return (w >> (j & 31)) & 1;
}

// 32 bits of row t's view of the drafted tokens j0 .. j0 + 31 (those before 0 are context: seen).
__device__ __forceinline__ unsigned draft_bits(const Params& p, int b, int t, int j0) {
  if (j0 + 31 < 0) return ~0u;
  if (!p.tree) {
    const int n = t - j0;  // the last one seen
    return n >= 31 ? ~0u : n < 0 ? 0u : (2u << n) - 1u;
  }
  const int32_t* row = p.tree + ((long long)b * p.tokens + t) * p.tree_words;
  auto word = [&](int w) -> unsigned { return w < p.tree_words ? (unsigned)row[w] : 0u; };
  if (j0 < 0) return (word(0) << -j0) | ((1u << -j0) - 1u);
  const int w = j0 >> 5, sh = j0 & 31;
  return sh ? (word(w) >> sh) | (word(w + 1) << (32 - sh)) : word(w);
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

// Block c's partial of a unit whose first block is c0; `slot0`: which of that block's slots is the unit's.
template <int ROWS, int D>
__device__ __forceinline__ const float* part_of(const float* parts, int c, int c0, int slot0) {
  return parts + (2LL * c + (c == c0 ? slot0 : 0)) * (ROWS * (D + 2));
}

// One warp joins partials c0 + from, c0 + from + step, ... <= c1 of row r of a unit's tile:
//     out = sum_s 2^(m_s - m) o_s,  l = sum_s 2^(m_s - m) l_s,  m = max_s m_s
// (partials that saw nothing have l_s = 0 and count for nothing). A lane has D / 32 elements.
// 32 partials' weights are made at once, a lane each; their rows are read eight at a time.
template <int ROWS, int D>
__device__ __forceinline__ void join_row(const float* parts, int c0, int c1, int slot0, int r,
                                         int from, int step, float (&acc)[D / 32], float& m, float& l) {
  constexpr int kVec = D / 32;
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
  for (int b = c0 + from; b <= c1; b += 32 * step) {
    const int c = b + lane * step;
    const float* mine = part_of<ROWS, D>(parts, min(c, c1), c0, slot0) + r * D;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (c <= c1) ml = __ldcg(reinterpret_cast<const float2*>(mine + (ROWS - r) * D + 2 * r));
    float top = ml.y != 0.f ? ml.x : -INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, m);
    const float back = m == top ? 1.f : ex2(m - top);
    const float w = ml.y == 0.f ? 0.f : ml.x == top ? 1.f : ex2(ml.x - top);
    float sum = w * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * back + sum;
    m = top;
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] *= back;
    const int n = min(32, (c1 - b) / step + 1);
    for (int j = 0; j < n; j += 8) {
      float v[8][kVec];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float* row = part_of<ROWS, D>(parts, min(b + (j + e) * step, c1), c0, slot0) + r * D + lane * kVec;
        if (kVec == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(row));
          v[e][0] = x.x; v[e][1] = x.y; v[e][2 % kVec] = x.z; v[e][3 % kVec] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(row));
          v[e][0] = x.x; v[e][1] = x.y;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = __shfl_sync(0xffffffffu, w, (j + e) & 31);
        if (j + e < n && f != 0.f)
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] += f * v[e][i];
      }
    }
  }
}

// A lane's part of an output row, and the row's log-sum-exp.
template <int D>
__device__ __forceinline__ void store_joined(const Params& p, long long row, const float (&acc)[D / 32], float m, float l) {
  const int lane = threadIdx.x & 31;
  const float g = l == 0.f ? 0.f : 1.f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + row * D + lane * (D / 32));
#pragma unroll
  for (int i = 0; i < D / 64; ++i) out[i] = pack_bf16(acc[2 * i] * g, acc[2 * i + 1] * g);
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + lg2(l)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// Joining in a cluster
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t of_rank(uint32_t addr, unsigned rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
// All threads of all blocks of a unit's cluster. `part`: where each block has its partial in shared
// memory (outputs [row][D], then pairs (maximum, sum) at `ml`, 8 bytes a row; a block without keys
// has sums of zero). The first `threads` threads of each block share the unit's rows, four
// elements each.
template <int ROWS, int D, bool SEL>
__device__ __forceinline__ void join_cluster(const Params& p, uint32_t part, uint32_t ml, unsigned threads) {
  const unsigned size = (unsigned)p.cluster, rank = blockIdx.x % size, unit = blockIdx.x / size;
  const unsigned per = (unsigned)(p.kv_heads * p.row_tiles);
  const int seq = (int)(unit / per), in = (int)(unit % per);
  const int head = in / p.row_tiles, first = (in % p.row_tiles) * ROWS, live = min(p.rows - first, ROWS);
  __syncwarp();  // (the cluster's barrier takes whole warps; some lanes may have written their partial's sums last)
  cluster_sync();
  for (unsigned x = rank * threads + threadIdx.x; threadIdx.x < threads && x < (unsigned)live * (D / 4); x += size * threads) {
    const int r = x / (D / 4), d = (x % (D / 4)) * 4;
    float top = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (unsigned c0 = 0; c0 < size; c0 += 8) {  // eight blocks' at a time
      float2 q[8];
      float4 v[8];
#pragma unroll
      for (unsigned i = 0; i < 8; ++i) {
        q[i] = make_float2(-INFINITY, 0.f);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + i < size) {
          q[i] = ld_cluster2(of_rank(ml + 8 * r, c0 + i));
          v[i] = ld_cluster4(of_rank(part + (r * D + d) * 4, c0 + i));
        }
      }
      float most = top;
#pragma unroll
      for (unsigned i = 0; i < 8; ++i)
        if (q[i].y != 0.f) most = fmaxf(most, q[i].x);
      const float back = top == most ? 1.f : ex2(top - most);
      top = most;
      l *= back;
      o.x *= back; o.y *= back; o.z *= back; o.w *= back;
#pragma unroll
      for (unsigned i = 0; i < 8; ++i) {
        if (q[i].y == 0.f) continue;  // saw nothing
        const float f = q[i].x == top ? 1.f : ex2(q[i].x - top);
        l += f * q[i].y;
        o.x += f * v[i].x; o.y += f * v[i].y; o.z += f * v[i].z; o.w += f * v[i].w;
      }
    }
    const float g = l == 0.f ? 0.f : 1.f / l;
    const long long row = out_row<SEL>(p, seq, head, first + r);
    *reinterpret_cast<uint2*>(p.out + row * D + d) = make_uint2(pack_bf16(o.x * g, o.y * g), pack_bf16(o.z * g, o.w * g));
    if (p.lse && d == 0) p.lse[row] = l == 0.f ? -INFINITY : (top + lg2(l)) * 0.6931471805599453f;
  }
  __syncwarp();
  cluster_sync();  // no block leaves while its partial is read
}

// Host: the launch attributes of an attention kernel, and what it asks for once.
inline unsigned launch_attributes(cudaLaunchAttribute* a, int cluster) {
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  if (cluster <= 1) return 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = (unsigned)cluster;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  return 2;
}
template <typename K>
cudaError_t allow(K kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

// Floats of a partial slot: ROWS x D of output, then ROWS pairs (maximum, sum).
template <int ROWS, int D>
constexpr int kPartFloats = ROWS * (D + 2);

}  // namespace attn
}  // namespace tks
