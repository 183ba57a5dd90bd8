// Bounds of a cache's blocks, and the scores that queries give them.
//
// Mathematics.  Of a block's keys k_i, lo_d = min_i k_i,d and hi_d = max_i k_i,d.
// For a query q and any key of the block,
//     q . k_i <= sum_d max(q_d lo_d, q_d hi_d) = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// so a block's score is a product with a summed index of twice the head's size:
// the queries' positive and negative parts against the largest and the least
// values. Both parts are exact in bfloat16, as the products are in 32 bits.

#include <algorithm>

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

// The least and largest of a lane's 16-byte piece of the rows it has seen.
template <bool I8>
struct Extent;
template <>
struct Extent<true> {
  float lo[16], hi[16];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 16; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  }
  __device__ __forceinline__ void add(const uint4& w, float scale) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = (float)(int)(signed char)(u[i >> 2] >> (8 * (i & 3))) * scale;
      lo[i] = min_nan(lo[i], x);
      hi[i] = max_nan(hi[i], x);
    }
  }
  __device__ __forceinline__ void join(int o) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      hi[i] = max_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
    }
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* to, const float (&x)[16]) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = pack_bf16(finite_bf16(x[2 * i]), finite_bf16(x[2 * i + 1]));
    reinterpret_cast<uint4*>(to)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
};
template <>
struct Extent<false> {
  __nv_bfloat162 lo[4], hi[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __floats2bfloat162_rn(INFINITY, INFINITY);
      hi[i] = __floats2bfloat162_rn(-INFINITY, -INFINITY);
    }
  }
  __device__ __forceinline__ void add(const uint4& w, float) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&u[i]);
      lo[i] = __hmin2_nan(lo[i], x);
      hi[i] = __hmax2_nan(hi[i], x);
    }
  }
  __device__ __forceinline__ void join(int o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
    }
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* to, const __nv_bfloat162 (&x)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack_bf16(finite_bf16(__low2float(x[i])), finite_bf16(__high2float(x[i])));
    *reinterpret_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};

constexpr int kBoundsThreads = 256;

// An item is (block, head), of all sequences' new blocks in order, head fastest; a warp takes one at a time.
template <int D, bool I8>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int kElem = I8 ? 1 : 2, kPieces = D * kElem / 16, kRows = 32 / kPieces, kE = 16 / kElem, kAhead = 4;
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
    const long long items = upto[kBoundsThreads - 1] * p.kv_heads;
    for (; next < items; next += warps) {
      const long long number = next / p.kv_heads;
      const int head = (int)(next - number * p.kv_heads);
      int at = 0;
#pragma unroll
      for (int step = kBoundsThreads / 2; step; step >>= 1)
        if (upto[at + step - 1] <= number) at += step;
      const int block = first_s[at] + (int)(number - (at ? upto[at - 1] : 0));
      const int pos = block << p.block_shift, count = min(1 << p.block_shift, end_s[at] - pos);
      const int page = __ldg(p.table + (s0 + at) * p.table_stride + (pos >> p.page_shift));
      if ((unsigned)page >= (unsigned)p.pages) {
        if (lane == 0) report(p.status, kStatIndexBit);
        continue;
      }
      const int in_page = pos & ((1 << p.page_shift) - 1);
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
        for (int i = 0; i < kAhead; ++i) x.add(w[i], sc[i]);
      }
      __syncwarp();
#pragma unroll
      for (int o = kPieces; o < 32; o <<= 1) x.join(o);
      const int of_page = 1 << (p.page_shift - p.block_shift);
      __nv_bfloat16* to = p.bounds + (((long long)page * of_page + (in_page >> p.block_shift)) * p.kv_heads + head) * (2 * D) + piece * kE;
      if (sub == 0) {
        Extent<I8>::put(to, x.lo);
        Extent<I8>::put(to + D, x.hi);
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

// Up to 16 query rows of a key/value head (all tokens' together). A thread block takes one (sequence, head) and a run of
// blocks; its query rows lie in shared memory as matrix fragments: of product step s, lane 4n + c takes the elements that
// it has of column n's 4 * D bytes: 16-byte pieces c, c + 4, ...
template <int D>
__global__ void __launch_bounds__(kScoreThreads) scores_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int kPieces = 2 * D * 2 / 16 / 4;  // of a lane
  constexpr int kSteps = 2 * kPieces;
  __shared__ uint4 qs[kSteps * 32];
  __shared__ float tile_s[kScoreWarps][16][kScoreCols + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
  const unsigned unit = blockIdx.x / p.chunks;
  const int chunk = blockIdx.x - unit * p.chunks;
  const int head = unit % p.kv_heads, b = unit / p.kv_heads, rows = p.tokens * p.group;
  grid_wait();
  grid_launch_dependents();

  for (int x = threadIdx.x; x < kSteps * 32; x += kScoreThreads) {
    const int l = x & 31, s = x >> 5, r = l >> 2;
    // elements of the doubled index: the first D are the least's, with the queries' negative parts
    const int d = 8 * ((l & 3) + 4 * (s >> 1)) + 4 * (s & 1);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(score_query(p, b, r / p.group, head, r % p.group) + d % D));
      w.x = part_of_pair(y.x, d >= D);
      w.z = part_of_pair(y.y, d >= D);
    }
    if (r + 8 < rows) {
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(score_query(p, b, (r + 8) / p.group, head, (r + 8) % p.group) + d % D));
      w.y = part_of_pair(y.x, d >= D);
      w.w = part_of_pair(y.y, d >= D);
    }
    qs[x] = w;
  }
  // the tokens' lengths, a lane each (16 at most)
  bool bad = false;
  const int mine = lane < p.tokens ? blocks_seen(p, b, lane, bad) : 0;
  const int most = __reduce_max_sync(0xffffffffu, mine);
  if (warp == 0 && chunk == 0) {
    if (bad) report(p.status, kStatRowLenBit);
    if (p.row_len && lane < p.tokens) p.row_len[((long long)b * p.tokens + lane) * p.kv_heads + head] = mine;
  }
  __syncthreads();

  const int32_t* table = p.table + b * p.table_stride;
  for (long long j0 = ((long long)chunk * kScoreWarps + warp) * kScoreCols; j0 < p.n; j0 += (long long)p.chunks * kScoreThreads) {
    const int col = (int)j0 + lane;
    bool ok = true;
    if (j0 < most) {
      const int page = col < most ? __ldg(table + (col >> p.of_page_shift)) : 0;
      ok = (unsigned)page < (unsigned)p.pages;
      if (!ok) report(p.status, kStatIndexBit);
      const long long at = ok && col < most ? (((long long)page << p.of_page_shift) + (col & ((1 << p.of_page_shift) - 1))) * p.kv_heads + head : -1;
      float acc[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const long long of = __shfl_sync(0xffffffffu, at, 8 * t + n);
        const uint4* from = reinterpret_cast<const uint4*>(p.bounds + of * (2 * D)) + c;
        uint4 w[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) w[i] = of >= 0 ? __ldg(from + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
        acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          mma_bf16(acc[t], qs[2 * i * 32 + lane], w[i].x, w[i].y);
          mma_bf16(acc[t], qs[(2 * i + 1) * 32 + lane], w[i].z, w[i].w);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) tile_s[warp][n + 8 * (e >> 1)][8 * t + 2 * c + (e & 1)] = acc[t][e];
      __syncwarp();
    }
    for (int t = 0; t < p.tokens; ++t) {
      const int seen = __shfl_sync(0xffffffffu, mine, t);
      float x = -INFINITY;
      if (j0 < most)
        for (int r = t * p.group; r < (t + 1) * p.group; ++r) x = max_nan(x, tile_s[warp][r][lane]);
      if (col < p.n) p.out[(((long long)b * p.tokens + t) * p.kv_heads + head) * p.n + col] = !ok ? -INFINITY : final_score(p, x, col, seen);
    }
    __syncwarp();
  }
}

void with_pdl(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* a) {
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
}

template <int D>
cudaError_t launch_bounds(const BoundsParams& p, bool i8, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute a[1] = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kBoundsThreads);
  cfg.stream = stream;
  with_pdl(cfg, a);
  return i8 ? cudaLaunchKernelEx(&cfg, bounds_kernel<D, true>, p) : cudaLaunchKernelEx(&cfg, bounds_kernel<D, false>, p);
}

template <int D>
cudaError_t launch_scores(const ScoreParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute a[1] = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kScoreThreads);
  cfg.stream = stream;
  with_pdl(cfg, a);
  return cudaLaunchKernelEx(&cfg, scores_kernel<D>, p);
}

}  // namespace

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
  const int grid = (int)std::min<__int128>(items, place.sms * 4);
  std::lock_guard<std::mutex> lock(*place.order);
  const cudaError_t e = cache->head_dim == 64 ? launch_bounds<64>(p, i8, grid, (cudaStream_t)stream) : launch_bounds<128>(p, i8, grid, (cudaStream_t)stream);
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
  if ((int64_t)queries->batch * queries->tokens * bounds->kv_heads > INT32_MAX) return TKS_E_TOO_LARGE;
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
  if ((int64_t)p.tokens * p.group <= 16) {
    const int64_t units = (int64_t)p.batch * p.kv_heads;
    const int64_t most = std::max<int64_t>(1, ((int64_t)n + kScoreThreads - 1) / kScoreThreads);
    p.chunks = (int)std::min<int64_t>(most, std::max<int64_t>(1, place.sms * 16 / units));
    if (units * p.chunks > INT32_MAX) return TKS_E_TOO_LARGE;
    e = bounds->head_dim == 64 ? launch_scores<64>(p, (int)(units * p.chunks), s) : launch_scores<128>(p, (int)(units * p.chunks), s);
  } else {
    // (134 MB of scores, stored as what is not read again soon: 58 us, 63 without; fewer stay for the selector)
    p.stream_out = (int64_t)p.batch * p.tokens * p.kv_heads * n > (64 << 20) / 4;
    // a token's rows lie in one half of a tile: larger groups are scored in parts
    constexpr int half = kScoreTileRows / 2;
    const int parts = (p.group_all + half - 1) / half, each = (p.group_all + parts - 1) / parts;
    for (p.first_of_group = 0; p.first_of_group < p.group_all && e == cudaSuccess; p.first_of_group += each) {
      p.group = std::min(each, p.group_all - p.first_of_group);
      p.half_tokens = half / p.group;
      p.tile_tokens = 2 * p.half_tokens;
      p.token_tiles = (p.tokens - 1) / p.tile_tokens + 1;
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
