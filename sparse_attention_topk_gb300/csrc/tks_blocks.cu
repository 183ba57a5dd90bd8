// Bounds of a cache's blocks, and the scores that queries give them.
//
// Mathematics.  Of a block's keys k_i, lo_d = min_i k_i,d and hi_d = max_i k_i,d.
// For a query q and any key of the block,
//     q . k_i <= sum_d max(q_d lo_d, q_d hi_d) = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// so a block's score is a product with a summed index of twice the head's size:
// the queries' positive and negative parts against the largest and the least
// values. Both parts are exact in bfloat16, as the products are in 32 bits; their
// sum is in 32 bits.  Bounds are rounded to bfloat16, to nearest: a score is off by
// at most 2^-8 of the sum of its terms' magnitudes for that.
//
// What bounds it: bytes, or the way to them.  Bounds read each key once, and
// write 1/16 as much (blocks of 64 in 8 bits); scores read those, and write 4 bytes a block
// and head. A decode step's calls are short: they are chains of lookups (lengths,
// page, rows) that a lone call cannot hide, so what a chain does not need is loaded
// beside it.
// Measured: bounds of a prompt of 32,768 tokens of 8 int8 heads of 128 (37 MB) 10.2
// us, 3.6 TB/s, 12.7 from memory; of 64 decode steps 4.1 us.  Scores of one token
// of 32 heads on 8 over 2048 blocks (8.5 MB) 4.7 us; of 64 ragged sequences of 16
// heads on 2 over up to 2048 blocks (71 MB) 14.8 us, 4.8 TB/s, 18.8 from memory (with a
// thread block for every 128 blocks, as for one token, 20.7).

#include <algorithm>
#include <cmath>

#include "tks_attn.cuh"
#include "tks_attn_host.h"
#include "tks_scores.cuh"

namespace tks {
namespace attn {
namespace {

constexpr float kBf16Max = 3.3895313892515355e38f;

// ---------------------------------------------------------------------------
// Bounds.
// ---------------------------------------------------------------------------
struct BoundsParams {
  const unsigned char* k;
  const float* scales;
  long long page_b, token_b, head_b;
  int pages, page_shift, block_shift, kv_heads;
  __nv_bfloat16* bounds;
  const int32_t *table, *start, *end;
  long long table_stride;
  int table_pages, batch;
  unsigned* status;
};

__device__ __forceinline__ float finite_bf16(float x) { return x > kBf16Max ? kBf16Max : x < -kBf16Max ? -kBf16Max : x; }

// The least (or largest) of three; a NaN among them wins.
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// The least and largest of a lane's 16-byte piece of the rows it has seen, two rows at a time. At the end they are
// bfloat16 (rounding keeps the order, so the least of rounded values is the rounded least).
template <bool I8>
struct Extent;
template <>
struct Extent<true> {
  static constexpr int kPairs = 8;
  float lo[16], hi[16];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 16; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  }
  // Four codes' values: codes become halves, exactly, then 32-bit floats.
  static __device__ __forceinline__ void values(uint32_t codes, float scale, float (&x)[4]) {
    const uint32_t u = codes ^ 0x80808080u, a = codes_to_half2<0x4140>(u), b = codes_to_half2<0x4342>(u);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a)), g = __half22float2(*reinterpret_cast<const __half2*>(&b));
    x[0] = f.x * scale;
    x[1] = f.y * scale;
    x[2] = g.x * scale;
    x[3] = g.y * scale;
  }
  __device__ __forceinline__ void add(const uint4& w, const uint4& v, float ws, float vs) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[4], y[4];
      values(a[i], ws, x);
      values(b[i], vs, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[4 * i + j] = min3_nan(lo[4 * i + j], x[j], y[j]);
        hi[4 * i + j] = max3_nan(hi[4 * i + j], x[j], y[j]);
      }
    }
  }
  __device__ __forceinline__ void rounded(__nv_bfloat162 (&l)[8], __nv_bfloat162 (&h)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      l[i] = __floats2bfloat162_rn(finite_bf16(lo[2 * i]), finite_bf16(lo[2 * i + 1]));
      h[i] = __floats2bfloat162_rn(finite_bf16(hi[2 * i]), finite_bf16(hi[2 * i + 1]));
    }
  }
};
template <>
struct Extent<false> {
  static constexpr int kPairs = 4;
  __nv_bfloat162 lo[4], hi[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __floats2bfloat162_rn(INFINITY, INFINITY);
      hi[i] = __floats2bfloat162_rn(-INFINITY, -INFINITY);
    }
  }
  __device__ __forceinline__ void add(const uint4& w, const uint4& v, float, float) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&a[i]), y = *reinterpret_cast<const __nv_bfloat162*>(&b[i]);
      lo[i] = __hmin2_nan(lo[i], __hmin2_nan(x, y));
      hi[i] = __hmax2_nan(hi[i], __hmax2_nan(x, y));
    }
  }
  __device__ __forceinline__ void rounded(__nv_bfloat162 (&l)[4], __nv_bfloat162 (&h)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[i] = __floats2bfloat162_rn(finite_bf16(__low2float(lo[i])), finite_bf16(__high2float(lo[i])));
      h[i] = __floats2bfloat162_rn(finite_bf16(__low2float(hi[i])), finite_bf16(__high2float(hi[i])));
    }
  }
};

// (Sixteen pieces a lane under way in four thread blocks an SM: 64 decode steps take 3.7 us, with eight in seven 5.1.)
constexpr int kBoundsThreads = 128, kBoundsPerSm = 4;

// The furthest end (of `end` and on) of the sequences that hold this page at the same place of their rows.
__device__ __forceinline__ int furthest_end(const BoundsParams& p, int end, int page, int at, int cap) {
  const int lane = threadIdx.x & 31;
  int furthest = end;
  for (int s = lane; s - lane < p.batch; s += 128) {
    int e[4], held[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = s + 32 * i < p.batch ? min(__ldg(p.end + s + 32 * i), cap) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) held[i] = e[i] > end ? __ldg(p.table + (s + 32 * i) * p.table_stride + at) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (held[i] == page) furthest = max(furthest, e[i]);
  }
  return __reduce_max_sync(0xffffffffu, furthest);
}

// An item is (block, head), of all sequences' new blocks in order, head fastest; a warp takes one at a time, or (ALL, many sequences)
// all heads of a block. Of a block that a sequence does not fill, another may hold more: both take it as far as either does, so that
// it does not matter who stores last. Looking the others up takes 0.5 of 64 decode steps' 4.1 us, 1.9 of 256
// steps' 10.5, and, of 4096 steps' 249, which look at 2048 rows each, 105 (434 in all where each head looks for itself).
template <int D, bool I8, bool ALL>
__global__ void __launch_bounds__(kBoundsThreads, kBoundsPerSm) bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int kElem = I8 ? 1 : 2, kPieces = D * kElem / 16, kRows = 32 / kPieces, kE = 16 / kElem, kAhead = 16;
  __shared__ long long upto[kBoundsThreads];  // blocks of the sequences up to and with this one
  __shared__ int first_s[kBoundsThreads], end_s[kBoundsThreads];
  __shared__ long long warps_s[kBoundsThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = lane % kPieces, sub = lane / kPieces;
  grid_wait();
  grid_launch_dependents();
  const long long room = (long long)p.table_pages << p.page_shift;
  const int cap = room > kMaxPositions ? kMaxPositions : (int)room;
  const long long warps = (long long)gridDim.x * (kBoundsThreads / 32);
  long long next = (long long)warp * gridDim.x + blockIdx.x;  // this warp's next item, among these sequences'
  for (int s0 = 0; s0 < p.batch; s0 += kBoundsThreads) {
    const int s = s0 + threadIdx.x;
    int from = 0, end = 0;
    if (s < p.batch) {
      const int a = p.start ? __ldg(p.start + s) : 0, e = __ldg(p.end + s);
      from = min(max(a, 0), cap);
      end = min(max(e, 0), cap);
      if (blockIdx.x == 0 && (from != a || end != e)) report(p.status, kStatRowLenBit);
    }
    const int first = from >> p.block_shift;
    long long sum = from < end ? ((end - 1) >> p.block_shift) + 1 - first : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) warps_s[warp] = sum;
    first_s[threadIdx.x] = first;
    end_s[threadIdx.x] = end;
    __syncthreads();
    for (int i = 0; i < warp; ++i) sum += warps_s[i];
    upto[threadIdx.x] = sum;
    __syncthreads();
    const int of_block = ALL ? 1 : p.kv_heads;
    const long long items = upto[kBoundsThreads - 1] * of_block;
    for (; next < items; next += warps) {
      const long long number = next / of_block;
      const int head0 = ALL ? 0 : (int)(next - number * of_block);
      int at = 0;
#pragma unroll
      for (int step = kBoundsThreads / 2; step; step >>= 1)
        if (upto[at + step - 1] <= number) at += step;
      const int block = first_s[at] + (int)(number - (at ? upto[at - 1] : 0));
      const int pos = block << p.block_shift, place = pos >> p.page_shift, end = end_s[at];
      const int page = __ldg(p.table + (s0 + at) * p.table_stride + place);
      if ((unsigned)page >= (unsigned)p.pages) {
        if (lane == 0) report(p.status, kStatIndexBit);
        continue;
      }
      int upto_end = end;
      if (end - pos < 1 << p.block_shift && p.batch > 1) upto_end = furthest_end(p, end, page, place, cap);
      const int count = min(1 << p.block_shift, upto_end - pos);
      const int in_page = pos & ((1 << p.page_shift) - 1);
      for (int head = head0; head < (ALL ? p.kv_heads : head0 + 1); ++head) {
        const unsigned char* base = p.k + page * p.page_b + in_page * p.token_b + head * p.head_b + piece * 16;
        const float* scales = I8 ? p.scales + 2 * ((((long long)page << p.page_shift) + in_page) * p.kv_heads + head) : nullptr;
        Extent<I8> x;
        x.clear();
        for (int r0 = sub; r0 < count; r0 += kRows * kAhead) {  // (rows past the last are the last again)
          uint4 w[kAhead];
          float sc[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int r = min(r0 + i * kRows, count - 1);
            w[i] = __ldg(reinterpret_cast<const uint4*>(base + r * p.token_b));
            sc[i] = I8 ? __ldg(scales + 2LL * r * p.kv_heads) : 0.f;
          }
#pragma unroll
          for (int i = 0; i < kAhead; i += 2) x.add(w[i], w[i + 1], sc[i], sc[i + 1]);
        }
        __syncwarp();
        constexpr int kPairs = Extent<I8>::kPairs;
        __nv_bfloat162 lo[kPairs], hi[kPairs];
        x.rounded(lo, hi);
#pragma unroll
        for (int o = kPieces; o < 32; o <<= 1)
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
            hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
          }
        const int of_page = 1 << (p.page_shift - p.block_shift);
        uint4* to = reinterpret_cast<uint4*>(p.bounds + (((long long)page * of_page + (in_page >> p.block_shift)) * p.kv_heads + head) * (2 * D) + piece * kE);
        if (sub == 0) {
#pragma unroll
          for (int i = 0; i < kPairs; i += 4) {
            to[i / 4] = make_uint4(bits_of(lo[i]), bits_of(lo[i + 1]), bits_of(lo[i + 2]), bits_of(lo[i + 3]));
            to[D / 8 + i / 4] = make_uint4(bits_of(hi[i]), bits_of(hi[i + 1]), bits_of(hi[i + 2]), bits_of(hi[i + 3]));
          }
        }
      }
    }
    next -= items;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Scores.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
constexpr int kScoreWarps = 4, kScoreThreads = kScoreWarps * 32;
constexpr int kScoreCols = 32;  // blocks that a warp scores at once

template <int D>
struct ScoreShape {
  static constexpr int kRow = 4 * D;            // bytes of a block's bounds
  static constexpr int kWarp = kScoreCols * kRow;
  static constexpr int kPieces = kRow / 16;     // 16-byte pieces
  static constexpr int kSteps = 2 * D / 16;     // products of 16 of the summed elements
  static constexpr int kQs = kSteps * 32 * 16;  // the query rows' fragments
  static constexpr int kSmem = kScoreWarps * kWarp + kQs;
  static_assert(16 * (kScoreCols + 1) * 4 <= kWarp, "a warp's scores fit where its bounds were");
};

// Up to 16 query rows of a key/value head: a tile of tokens. A thread block takes one (sequence, tile, head) and 128 blocks,
// a warp 32 of them, whose copies to shared memory are all under way at once, and start before the queries and
// lengths are there. The query rows lie in shared memory as matrix fragments: of product step s, lane 4n + c takes the
// elements that it has of column n's bytes: pieces c, c + 4, ... (XOR-swizzled, so that eight lanes' reads do not meet).
template <int D>
__global__ void __launch_bounds__(kScoreThreads) scores_kernel(const __grid_constant__ ScoreParams p) {
  using S = ScoreShape<D>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
  unsigned char* mine = smem + warp * S::kWarp;
  float(*tile)[kScoreCols + 1] = reinterpret_cast<float(*)[kScoreCols + 1]>(mine);
  uint4* qs = reinterpret_cast<uint4*>(smem + kScoreWarps * S::kWarp);
  const unsigned unit = blockIdx.x / p.chunks;
  const int chunk = blockIdx.x - unit * p.chunks;
  const int head = unit % p.kv_heads, bt = unit / p.kv_heads, b = bt / p.token_tiles, t0 = (bt - b * p.token_tiles) * p.tile_tokens;
  const int tokens = min(p.tile_tokens, p.tokens - t0), rows = tokens * p.group;
  const int32_t* table = p.table + b * p.table_stride;
  // the lane's pieces of a row, and its first row, in the copies
  constexpr int kPer = 32 / S::kPieces > 0 ? 32 / S::kPieces : 1;  // rows that 32 lanes cover
  const int piece = lane % S::kPieces, row0 = lane / S::kPieces;
  grid_wait();
  grid_launch_dependents();

  const long long j0 = ((long long)chunk * kScoreWarps + warp) * kScoreCols;
  const int col = (int)j0 + lane;
  const int page = j0 < p.n && col < p.n ? __ldg(table + (col >> p.of_page_shift)) : -1;
  // the tokens' lengths, a lane each (16 at most), and the query rows
  bool bad = false;
  const int seen = lane < tokens ? blocks_seen(p, b, t0 + lane, bad) : 0;
  for (int x = threadIdx.x; x < S::kSteps * 32; x += kScoreThreads) {
    const int l = x & 31, s = x >> 5, r = l >> 2;
    // elements of the doubled index: the first D are the least's, with the queries' negative parts
    const int d = 8 * ((l & 3) + 4 * (s >> 1)) + 4 * (s & 1);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(score_query(p, b, t0 + r / p.group, head, r % p.group) + d % D));
      w.x = part_of_pair(y.x, d >= D);
      w.z = part_of_pair(y.y, d >= D);
    }
    if (r + 8 < rows) {
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(score_query(p, b, t0 + (r + 8) / p.group, head, (r + 8) % p.group) + d % D));
      w.y = part_of_pair(y.x, d >= D);
      w.w = part_of_pair(y.y, d >= D);
    }
    qs[x] = w;
  }
  const int most = __reduce_max_sync(0xffffffffu, seen);
  const bool ok = (unsigned)page < (unsigned)p.pages;
  if (j0 < most) {
    if (!ok && col < most) report(p.status, kStatIndexBit);
    const long long at = ok && col < most ? (((long long)page << p.of_page_shift) + (col & ((1 << p.of_page_shift) - 1))) * p.kv_heads + head : -1;
    const uint32_t to = smem_addr(mine) + row0 * S::kRow;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int i = 0; i < 8 / kPer; ++i) {
        const int r = 8 * t + i * kPer + row0;  // the column; its pieces lie swizzled
        const long long of = __shfl_sync(0xffffffffu, at, r);
        cp16(to + (8 * t + i * kPer) * S::kRow + ((piece ^ ((r & 1) << 2)) << 4),
             reinterpret_cast<const unsigned char*>(p.bounds) + (of < 0 ? 0 : of * S::kRow) + piece * 16, of < 0 ? 0 : 16);
      }
      cp_commit();
    }
  }
  if (warp == 0 && chunk == 0) {
    if (bad) report(p.status, kStatRowLenBit);
    if (p.row_len && lane < tokens) p.row_len[((long long)b * p.tokens + t0 + lane) * p.kv_heads + head] = seen;
  }
  __syncthreads();
  if (j0 < most) {
    float acc[4][4];
    auto columns = [&](int t) {  // (in two sums, which neither wait for each other nor round at one size)
      __syncwarp();
      float odd[4] = {0.f, 0.f, 0.f, 0.f};
      acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
      const unsigned char* row = mine + (8 * t + n) * S::kRow;
#pragma unroll
      for (int i = 0; i < S::kPieces / 4; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(row + (((c + 4 * i) ^ ((n & 1) << 2)) << 4));
        mma_bf16(acc[t], qs[2 * i * 32 + lane], w.x, w.y);
        mma_bf16(odd, qs[(2 * i + 1) * 32 + lane], w.z, w.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] += odd[e];
    };
    cp_wait<3>();
    columns(0);
    cp_wait<2>();
    columns(1);
    cp_wait<1>();
    columns(2);
    cp_wait<0>();
    columns(3);
    __syncwarp();  // (scores go where the bounds were)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[n + 8 * (e >> 1)][8 * t + 2 * c + (e & 1)] = acc[t][e];
    __syncwarp();
  }
  if (j0 >= p.n) return;
  for (int t = 0; t < tokens; ++t) {
    const int blocks = __shfl_sync(0xffffffffu, seen, t);
    float x = -INFINITY;
    if (j0 < most)
      for (int r = t * p.group; r < (t + 1) * p.group; ++r) x = max_nan(x, tile[r][lane]);
    if (col < p.n) p.out[(((long long)b * p.tokens + t0 + t) * p.kv_heads + head) * p.n + col] = !ok ? -INFINITY : final_score(p, x, col, blocks);
  }
}

// The same for more blocks than the device holds at once, 128 to a thread block: every warp takes an equal run of the axis of all (sequence,
// head)s' groups of eight blocks that any token sees, brings them through a ring of its own, and keeps the query rows of the
// (sequence, head) that it is at in registers, so that warps wait for nobody.
constexpr int kStreamWarps = 16, kStreamThreads = kStreamWarps * 32, kStreamCounted = 1024;
template <int D>
struct StreamShape {
  static constexpr int kRow = 4 * D, kGroup = 8 * kRow, kPieces = kRow / 16, kSteps = 2 * D / 16;
  static constexpr int kDepth = D == 128 ? 3 : 6;
  static constexpr int kRing = kDepth * kGroup, kTile = 16 * 9 * 4;
  static constexpr int kSmem = kStreamWarps * (kRing + kTile);
};

// A warp's run, piece by piece: groups g0 .. g1 - 1 of a (sequence, head).
struct Piece {
  int b, head, g0, g1;
};
struct Pieces {
  long long at, end;
  int b;
  __device__ __forceinline__ bool next(const ScoreParams& p, const int* upto, Piece& x) {
    if (at >= end) return false;
    const bool counted = p.batch <= kStreamCounted;
    const int all = (p.n + 7) / 8;
    if (!counted) {
      b = (int)(at / ((long long)all * p.kv_heads));
    } else {
      while ((long long)upto[b + 1] * p.kv_heads <= at) ++b;
    }
    const long long before = counted ? upto[b] : (long long)all * b;
    const int mine = counted ? upto[b + 1] - upto[b] : all;
    const long long in = at - before * p.kv_heads;
    x.b = b;
    x.head = (int)(in / mine);
    x.g0 = (int)(in - (long long)x.head * mine);
    x.g1 = (int)min((long long)mine, x.g0 + end - at);
    at += x.g1 - x.g0;
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kStreamThreads, 1) scores_stream_kernel(const __grid_constant__ ScoreParams p) {
  using S = StreamShape<D>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int upto[kStreamCounted + 1];  // groups of the sequences before this one, each counted for one head
  __shared__ int warps_s[kStreamWarps];
  __shared__ unsigned there_s[kStreamWarps][S::kDepth];  // which of a group's blocks lie in a page of the cache
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
  unsigned char* ring = smem + warp * S::kRing;
  float(*tile)[9] = reinterpret_cast<float(*)[9]>(smem + kStreamWarps * S::kRing + warp * S::kTile);
  constexpr int kPer = 32 / S::kPieces > 0 ? 32 / S::kPieces : 1;
  const int piece = lane % S::kPieces, row0 = lane / S::kPieces, rows = p.tokens * p.group, all = (p.n + 7) / 8;
  const bool counted = p.batch <= kStreamCounted;
  grid_wait();
  grid_launch_dependents();

  if (counted) {
    int sum = 0, mine[kStreamCounted / kStreamThreads];
#pragma unroll
    for (int i = 0; i < kStreamCounted / kStreamThreads; ++i) {
      const int b = threadIdx.x * (kStreamCounted / kStreamThreads) + i;
      int most = 0;
      bool bad = false;
      if (b < p.batch)
        for (int t = 0; t < p.tokens; ++t) most = max(most, blocks_seen(p, b, t, bad));
      mine[i] = (most + 7) / 8;
      sum += mine[i];
    }
    int end = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    if (lane == 31) warps_s[warp] = end;
    __syncthreads();
    int at = end - sum;
    for (int i = 0; i < warp; ++i) at += warps_s[i];
    if (threadIdx.x == 0) upto[0] = 0;
#pragma unroll
    for (int i = 0; i < kStreamCounted / kStreamThreads; ++i) {
      at += mine[i];
      upto[threadIdx.x * (kStreamCounted / kStreamThreads) + i + 1] = at;
    }
    __syncthreads();
  }

  const long long work = (counted ? (long long)upto[kStreamCounted] : (long long)all * p.batch) * p.kv_heads;
  const int warps = gridDim.x * kStreamWarps, me = warp * gridDim.x + blockIdx.x;
  Pieces copies;
  copies.at = work / warps * me + min((long long)me, work % warps);
  copies.end = copies.at + work / warps + (me < work % warps ? 1 : 0);
  copies.b = 0;
  if (counted && copies.at < copies.end) {  // the first one's sequence: the last with upto * heads <= at
    int low = 0;
#pragma unroll
    for (int step = kStreamCounted / 2; step; step >>= 1)
      if ((long long)upto[low + step] * p.kv_heads <= copies.at) low += step;
    copies.b = low;
  }
  Pieces scored = copies;
  int groups = (int)(copies.end - copies.at);

  // ---- copies, a group at a time; blocks are looked up 32 at once, and their pages 32 ahead
  Piece from{0, 0, 0, 0};
  const int32_t* table = nullptr;
  int base = 0, page = -1, most = 0, slot = 0;
  long long place = -1;
  bool more = true;
  auto page_of = [&](int col) -> int { return col < most ? __ldg(table + (col >> p.of_page_shift)) : -1; };
  auto issue = [&] {
    if (more && from.g0 == from.g1) {
      more = copies.next(p, upto, from);
      if (more) {
        table = p.table + from.b * p.table_stride;
        // (the columns of the piece's groups: those that no token sees are masked when they are written)
        most = (int)min((long long)p.n, 8LL * from.g1);
        base = 8 * from.g0 - 32;
        page = page_of(base + 32 + lane);
      }
    }
    if (more) {
      if (8 * from.g0 == base + 32) {
        base += 32;
        const int col = base + lane;
        place = (unsigned)page < (unsigned)p.pages
                    ? (((long long)page << p.of_page_shift) + (col & ((1 << p.of_page_shift) - 1))) * p.kv_heads + from.head : -1;
        page = page_of(col + 32);
      }
      const int in = 8 * from.g0 - base;
      const uint32_t to = smem_addr(ring) + slot * S::kGroup + row0 * S::kRow;
#pragma unroll
      for (int i = 0; i < 8 / kPer; ++i) {
        const int r = i * kPer + row0;
        const long long of = __shfl_sync(0xffffffffu, place, in + r);
        cp16(to + i * kPer * S::kRow + ((piece ^ ((r & 1) << 2)) << 4), reinterpret_cast<const unsigned char*>(p.bounds) + (of < 0 ? 0 : of * S::kRow) + piece * 16,
             of < 0 ? 0 : 16);
      }
      const unsigned there = __ballot_sync(0xffffffffu, place >= 0) >> in & 0xffu;
      if (lane == 0) there_s[warp][slot] = there;
      ++from.g0;
      slot = slot + 1 == S::kDepth ? 0 : slot + 1;
    }
    cp_commit();
  };
  for (int i = 0; i < S::kDepth - 1; ++i) issue();

  // ---- while these are under way: the rows' lengths, a lane each, and the groups that no token of a sequence sees, a row each warp
  const int out_rows = p.batch * p.tokens * p.kv_heads;
  for (long long r = me * 32LL + lane; r < out_rows; r += warps * 32LL) {
    const int bt = (int)r / p.kv_heads, b = bt / p.tokens;
    bool bad = false;
    const int blocks = blocks_seen(p, b, bt - b * p.tokens, bad);
    if (bad) report(p.status, kStatRowLenBit);
    if (p.row_len) p.row_len[r] = blocks;
  }
  if (counted && upto[kStreamCounted] < (long long)all * p.batch)
    for (long long r = me; r < out_rows; r += warps) {
      const int b = (int)r / p.kv_heads / p.tokens;
      for (long long j = 8LL * (upto[b + 1] - upto[b]) + lane; j < p.n; j += 32) p.out[r * p.n + j] = -INFINITY;
    }

  // ---- scores
  Piece at{0, 0, 0, 0};
  uint4 a[S::kSteps];
  int seen = 0, stage = 0;
  float* out = nullptr;
  for (; groups > 0; --groups) {
    if (at.g0 == at.g1) {
      scored.next(p, upto, at);
      bool bad = false;
      seen = lane < p.tokens ? blocks_seen(p, at.b, lane, bad) : 0;
      auto row = [&](int r) { return score_query(p, at.b, r / p.group, at.head, r % p.group); };
      const __nv_bfloat16 *q0 = row(n < rows ? n : 0), *q1 = row(n + 8 < rows ? n + 8 : 0);
#pragma unroll
      for (int s = 0; s < S::kSteps / 2; ++s) {  // the same elements of the least's and of the largest's half
        const int d = 8 * (c + 4 * (s >> 1)) + 4 * (s & 1);
        const uint2 x = n < rows ? __ldg(reinterpret_cast<const uint2*>(q0 + d)) : make_uint2(0u, 0u);
        const uint2 y = n + 8 < rows ? __ldg(reinterpret_cast<const uint2*>(q1 + d)) : make_uint2(0u, 0u);
        a[s] = make_uint4(part_of_pair(x.x, false), part_of_pair(y.x, false), part_of_pair(x.y, false), part_of_pair(y.y, false));
        a[s + S::kSteps / 2] = make_uint4(part_of_pair(x.x, true), part_of_pair(y.x, true), part_of_pair(x.y, true), part_of_pair(y.y, true));
      }
      out = p.out + ((long long)at.b * p.tokens * p.kv_heads + at.head) * p.n;
    }
    cp_wait<S::kDepth - 2>();
    __syncwarp();
    issue();  // (where the group before was)
    float acc[2][4] = {};
    const unsigned char* row = ring + stage * S::kGroup + n * S::kRow;
#pragma unroll
    for (int i = 0; i < S::kPieces / 4; ++i) {
      const uint4 w = *reinterpret_cast<const uint4*>(row + (((c + 4 * i) ^ ((n & 1) << 2)) << 4));
      mma_bf16(acc[0], a[2 * i], w.x, w.y);
      mma_bf16(acc[1], a[2 * i + 1], w.z, w.w);
    }
    const unsigned there = there_s[warp][stage];
    stage = stage + 1 == S::kDepth ? 0 : stage + 1;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = acc[0][e] + acc[1][e];
    const int col0 = 8 * at.g0++;
    if (p.tokens == 1) {
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[e] = n < rows ? x[e] : -INFINITY;
        if (n + 8 < rows) v[e] = max_nan(v[e], x[2 + e]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v[e] = max_nan(v[e], __shfl_xor_sync(0xffffffffu, v[e], o));
      }
      const float v0 = __shfl_sync(0xffffffffu, v[0], lane >> 1), v1 = __shfl_sync(0xffffffffu, v[1], lane >> 1);
      const int blocks = __shfl_sync(0xffffffffu, seen, 0), col = col0 + lane;
      if (lane < 8 && col < p.n) {
        const bool ok = there >> lane & 1u;
        if (!ok && col < blocks) report(p.status, kStatIndexBit);
        out[col] = ok ? final_score(p, lane & 1 ? v1 : v0, col, blocks) : -INFINITY;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[n + 8 * (e >> 1)][2 * c + (e & 1)] = x[e];
      __syncwarp();
      for (int i = lane; i < (p.tokens * 8 + 31) / 32 * 32; i += 32) {
        const int t = i >> 3, col = col0 + (i & 7);
        const int blocks = __shfl_sync(0xffffffffu, seen, t & 31);
        if (t < p.tokens && col < p.n) {
          float y = -INFINITY;
          for (int r = t * p.group; r < (t + 1) * p.group; ++r) y = max_nan(y, tile[r][i & 7]);
          const bool ok = there >> (i & 7) & 1u;
          if (!ok && col < blocks) report(p.status, kStatIndexBit);
          out[(long long)t * p.kv_heads * p.n + col] = ok ? final_score(p, y, col, blocks) : -INFINITY;
        }
      }
    }
  }
  cp_wait<0>();

}

template <int D>
cudaError_t launch_bounds(const BoundsParams& p, bool i8, bool all, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute a[1] = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kBoundsThreads);
  cfg.stream = stream;
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, 0);
  if (all) return i8 ? cudaLaunchKernelEx(&cfg, bounds_kernel<D, true, true>, p) : cudaLaunchKernelEx(&cfg, bounds_kernel<D, false, true>, p);
  return i8 ? cudaLaunchKernelEx(&cfg, bounds_kernel<D, true, false>, p) : cudaLaunchKernelEx(&cfg, bounds_kernel<D, false, false>, p);
}

template <int D>
cudaError_t launch_scores(const ScoreParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute a[1] = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kScoreThreads);
  cfg.dynamicSmemBytes = ScoreShape<D>::kSmem;
  cfg.stream = stream;
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, 0);
  return cudaLaunchKernelEx(&cfg, scores_kernel<D>, p);
}

template <int D>
cudaError_t launch_scores_stream(const ScoreParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute a[1] = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = StreamShape<D>::kSmem;
  cfg.stream = stream;
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, 0);
  return cudaLaunchKernelEx(&cfg, scores_stream_kernel<D>, p);
}

}  // namespace

cudaError_t setup_scores() {
  cudaError_t e = allow(scores_kernel<64>, ScoreShape<64>::kSmem);
  if (e == cudaSuccess) e = allow(scores_kernel<128>, ScoreShape<128>::kSmem);
  if (e == cudaSuccess) e = allow(scores_stream_kernel<64>, StreamShape<64>::kSmem);
  return e != cudaSuccess ? e : allow(scores_stream_kernel<128>, StreamShape<128>::kSmem);
}

int check_bounds(const tks_bounds* b) {
  if (b == nullptr || !b->bounds || !aligned(b->bounds, 16)) return TKS_E_INVAL;
  if (b->head_dim != 64 && b->head_dim != 128) return TKS_E_INVAL;
  if (b->kv_heads < 1 || b->pages < 1 || b->page_size < 1 || (b->page_size & (b->page_size - 1))) return TKS_E_INVAL;
  if (b->block < 1 || b->block > b->page_size || (b->block & (b->block - 1))) return TKS_E_INVAL;
  if ((int64_t)b->pages * b->page_size > INT32_MAX) return TKS_E_INVAL;
  const __int128 rows = (__int128)b->pages * (b->page_size / b->block) * b->kv_heads;
  return rows < ((__int128)1 << 50) ? TKS_OK : TKS_E_INVAL;
}

bool bounds_of(const tks_bounds* b, const tks_cache* c) {
  return b->pages == c->pages && b->page_size == c->page_size && b->kv_heads == c->kv_heads && b->head_dim == c->head_dim;
}

}  // namespace attn
}  // namespace tks

using namespace tks;
using namespace tks::attn;

extern "C" int tks_cache_bounds(const tks_cache* cache, const tks_bounds* bounds, const int32_t* page_table, int64_t table_stride,
                                int32_t table_pages, int32_t batch, const int32_t* start, const int32_t* end, void* stream) {
  if (check_cache(cache) != TKS_OK || check_bounds(bounds) != TKS_OK || !bounds_of(bounds, cache)) return TKS_E_INVAL;
  if (batch < 0 || table_pages < 0 || table_stride < 0 || table_stride > ((int64_t)1 << 56) / (batch > 0 ? batch : 1)) return TKS_E_INVAL;
  if (batch == 0) return TKS_OK;
  if (!end || !aligned(end, 4) || !aligned(start, 4)) return TKS_E_INVAL;
  if (table_pages > 0 && (!page_table || !aligned(page_table, 4))) return TKS_E_INVAL;
  Place place;
  const int rc = place_of(stream, &place);
  if (rc != TKS_OK) return rc;
  BoundsParams p{};
  const bool i8 = cache->held == TKS_I8;
  const long long size = i8 ? 1 : 2;
  p.k = static_cast<const unsigned char*>(cache->k);
  p.scales = cache->scales;
  p.page_b = cache->page_stride * size;
  p.token_b = cache->token_stride * size;
  p.head_b = cache->head_stride * size;
  p.pages = cache->pages;
  p.page_shift = log2_of(cache->page_size);
  p.block_shift = log2_of(bounds->block);
  p.kv_heads = cache->kv_heads;
  p.bounds = static_cast<__nv_bfloat16*>(bounds->bounds);
  p.table = page_table;
  p.start = start;
  p.end = end;
  p.table_stride = table_stride;
  p.table_pages = table_pages;
  p.batch = batch;
  p.status = place.status;
  // as many blocks as there may be items for, and no more than the device holds at once
  const __int128 items = (__int128)batch * std::max(1, table_pages) * (bounds->page_size / bounds->block) * cache->kv_heads;
  const int grid = (int)std::min<__int128>(items, place.sms * kBoundsPerSm);
  std::lock_guard<std::mutex> lock(*place.order);
  // (where every sequence has a new block, a block each warp and more)
  const bool all = (int64_t)batch >= (int64_t)place.sms * kBoundsPerSm * (kBoundsThreads / 32) / 4;
  const cudaError_t e = cache->head_dim == 64 ? launch_bounds<64>(p, i8, all, grid, (cudaStream_t)stream)
                                              : launch_bounds<128>(p, i8, all, grid, (cudaStream_t)stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}

extern "C" int tks_block_scores(const tks_bounds* bounds, const tks_queries* queries, const int32_t* kv_len, int32_t first, int32_t last,
                                float* scores, int32_t n, int32_t* row_len, void* stream) {
  if (check_bounds(bounds) != TKS_OK || check_q(bounds->kv_heads, queries) != TKS_OK) return TKS_E_INVAL;
  const int of_page = bounds->page_size / bounds->block;
  if (first < 0 || last < 0 || n < 0 || n > (int64_t)queries->table_pages * of_page) return TKS_E_INVAL;
  if (queries->batch == 0 || queries->tokens == 0) return TKS_OK;
  if (!aligned(kv_len, 4) || !aligned(row_len, 4) || !aligned(scores, 4) || (n > 0 && !scores)) return TKS_E_INVAL;
  if ((int64_t)queries->batch * queries->tokens * bounds->kv_heads > INT32_MAX || (int64_t)queries->batch * (n / 8 + 1) > INT32_MAX) return TKS_E_TOO_LARGE;
  Place place;
  const int rc = place_of(stream, &place);
  if (rc != TKS_OK) return rc;
  ScoreParams p{};
  p.bounds = static_cast<const __nv_bfloat16*>(bounds->bounds);
  p.pages = bounds->pages;
  p.block_shift = log2_of(bounds->block);
  p.of_page_shift = log2_of(of_page);
  p.kv_heads = bounds->kv_heads;
  p.q = static_cast<const __nv_bfloat16*>(queries->q);
  p.q_batch = queries->q_batch_stride;
  p.q_token = queries->q_token_stride;
  p.q_head = queries->q_head_stride;
  p.batch = queries->batch;
  p.tokens = queries->tokens;
  p.group = p.group_all = queries->q_heads / bounds->kv_heads;
  p.table = queries->page_table;
  p.table_stride = queries->table_stride;
  p.kv_len = kv_len;
  p.first = first;
  p.last = last;
  p.out = scores;
  p.n = n;
  p.row_len = row_len;
  p.status = place.status;
  p.spin_limit_ns = spin_limit_ns();
  p.test_skip_arrive = test_skip_arrive();
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  std::lock_guard<std::mutex> lock(*place.order);
  // Three ways: at once (a thread block for each 16 rows and 128 blocks, three an SM, some 6.5 us each); as streams, where all
  // of a head's rows are 16 at most and there is more than one wave of these; as tiles on the tensor cores, whose start takes
  // some 8 us, a tile of queries 3.5 and one of blocks 1.1. What is likely to take longer is left (8 * 8 drafts of 32 heads
  // on 8 over up to 1024 blocks: 17 us at once, 10.3 as tiles; 62 * 18 tokens of 8 heads over one block 19.5 and 22).
  const bool wide = bounds->head_dim == 128, few = (int64_t)p.tokens * p.group <= 16;
  const int64_t chunks = std::max<int64_t>(1, ((int64_t)n + kScoreThreads - 1) / kScoreThreads), heads = (int64_t)p.batch * p.kv_heads;
  p.tile_tokens = std::min(p.tokens, std::max(1, 16 / p.group));
  p.token_tiles = (p.tokens - 1) / p.tile_tokens + 1;
  p.chunks = (int)chunks;
  const double at_once = (double)heads * p.token_tiles * chunks, of_tile = std::max(1, 2 * (kScoreTileRows / 2 / p.group)),
               as_tiles = 8 + heads * std::ceil(p.tokens / of_tile) * (3.5 + 1.1 * chunks) / place.sms;
  if (p.group <= 16 && (few ? at_once <= 3 * place.sms : at_once < 65536 && 2 + 2.2 * at_once / place.sms < as_tiles)) {
    e = wide ? launch_scores<128>(p, (int)at_once, s) : launch_scores<64>(p, (int)at_once, s);
  } else if (few) {
    e = wide ? launch_scores_stream<128>(p, place.sms, s) : launch_scores_stream<64>(p, place.sms, s);
  } else {
    // (134 MB of scores, stored as what is not read again soon: 58 us, 63 without; fewer stay for the selector)
    p.stream_out = (int64_t)p.batch * p.tokens * p.kv_heads * n > (64 << 20) / 4;
    // a token's rows lie in one half of a tile: larger groups are scored in parts
    constexpr int half = kScoreTileRows / 2;
    const int parts = (p.group_all + half - 1) / half, each = (p.group_all + parts - 1) / parts;
    for (p.first_of_group = 0; p.first_of_group < p.group_all && e == cudaSuccess; p.first_of_group += each) {
      p.group = std::min(each, p.group_all - p.first_of_group);
      p.group_room = 1 << log2_of(p.group);
      // Whole tiles, or smaller ones where these leave SMs without work (2 * 300 tokens of 4 heads over 938 blocks: 17.5 us,
      // 25 in whole ones).
      for (p.half_rows = half;; p.half_rows /= 2) {
        p.half_tokens = p.half_rows / p.group_room;
        p.tile_tokens = 2 * p.half_tokens;
        p.token_tiles = (p.tokens - 1) / p.tile_tokens + 1;
        const int64_t tiles = (int64_t)p.batch * p.token_tiles * p.kv_heads * (((int64_t)n + kScoreTileBlocks - 1) / kScoreTileBlocks);
        if (tiles >= place.sms || p.half_rows <= std::max(32, p.group_room)) break;
      }
      e = launch_score_tiles(p, bounds->head_dim, place.sms, s);
      p.join = true;
      p.row_len = nullptr;
    }
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}
