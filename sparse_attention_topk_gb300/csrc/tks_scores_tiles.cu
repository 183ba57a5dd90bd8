// Scores of a cache's blocks for many query rows of each key/value head: chunks of
// prompts, drafted tokens, wide head groups, on the tcgen05 tensor cores.
//
// Mathematics: that of tks_blocks.cu, a product of blocks' bounds (128 a tile,
// 2 * dim elements each) with queries' negative and positive parts (256 rows a
// tile). The blocks are the product's rows and the queries its columns, so that a
// lane of tensor memory is a block, a token's query heads are neighbouring columns
// of it, their maximum is taken within a thread, and a warp's stores are whole
// 128-byte pieces of a row of scores.
//
// Layout.  One thread block an SM. Its query tile (128 KB at dim = 128) stays in
// shared memory while tiles of bounds pass through a ring of K blocks (64 of the
// summed elements, 16 KB, of 128 blocks), four producer warps' cp.async; one warp
// issues the products into one of two accumulators of 256 columns; eight warps take
// the other's maxima and store them. Three more bring the query tile.
//
// Work is the axis of all (sequence, tile of tokens)s' heads' tiles of blocks that any of their
// tokens sees, of which every thread block takes an equal run.
//
// What bounds it: while products run, the tensor cores (one of 128 blocks, 256 rows and 16
// elements takes 128 cycles, and reads 96 of shared memory's 128 bytes a cycle; the ring's
// copies write 32 more), but they run less than half of the time.
// Measured: 2048 tokens of 32 heads on 8 over 131,072 positions in blocks of 64 (68
// Gflop, 134 MB of scores) 58 us, 1.17 PFLOP/s, 63 from memory. Of these, tensor cores are
// busy 29 (27 tiles of blocks an SM); the start takes some 7, each of the 2.7 changes of query
// tile an SM some 4, since the queries have one buffer, refilled only as the last products
// before release it; without most of the stores it takes 50, without maxima and stores 48.
// (A pair of SMs on one product would have room for two tiles of queries: not tried.)
//
// Every wait is bounded: a wait that runs out reports TKS_E_TIMEOUT and ends its
// warp's role, which makes the waits on that warp run out; when all roles have
// ended the thread block frees its tensor memory and returns.

#include <algorithm>
#include <climits>

#include "tks_scores.cuh"
#include "tks_tensor.cuh"

namespace tks {
namespace attn {
namespace {

constexpr int kRows = kScoreTileRows, kBlocks = kScoreTileBlocks;
constexpr int kMaxWarps = 8, kProducer0 = 8, kQuery0 = 12, kQueryWarps = 3, kMulWarp = 15, kThreads = 16 * 32;
constexpr int kUnits = 1024;  // tiles of tokens whose lengths are looked at before the work is split

template <int D>
struct Shape {
  static constexpr int kSteps = 2 * D / 64;             // K blocks, taken in this order: 64 elements' negative parts, their
  static constexpr int kParts = kSteps / 2;             // positive ones, the next 64 elements'
  static __device__ __forceinline__ int k_block(int step) { return (step >> 1) + (step & 1) * kParts; }
  static constexpr int kStage = kBlocks * 128;          // of bounds
  static constexpr int kQueries = kRows * 128;          // of queries
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kRing = kSteps * kQueries;       // where the ring begins
  static constexpr int kSmem = kRing + kStages * kStage + 1024;  // and room to align the base
};

enum Bar { kFull = 0, kEmpty = kFull + 8, kSumFull = kEmpty + 8, kSumEmpty = kSumFull + 2, kQFull = kSumEmpty + 2, kQEmpty = kQFull + 2,
           kFinal = kQEmpty + 2, kBars = kFinal + 1 };

struct Shared {
  unsigned long long bars[kBars];
  uint32_t tmem;
  int upto[kUnits + 1];             // tiles of blocks of the tiles of tokens before this one, each counted for one head
  int seen[kMaxWarps][kRows / 2];   // the blocks that a half's tokens see (a copy for each warp)
  long long row[kRows];             // a query row's place behind its tile's first, in elements,
  int token[kRows];                 // and its token in the tile (one beyond all of them: none)
};

struct Block {
  uint32_t bars, queries, ring;
  unsigned char* smem;
  unsigned* status;
  long long limit;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  template <bool NAP = false>
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const { return bar_wait<NAP>(bar(i), parity, limit, status); }
};

// A run of tiles of blocks of one (sequence, tile of tokens, head).
struct Item {
  int b, t0, tokens, head;  // tokens: of this tile
  int j0, j1;               // tiles of blocks
};
// A thread block's items, in order.
struct Items {
  long long at, end;
  int unit, upto0, upto1;  // the tile of tokens that `at` lies in, and the tiles of blocks before it and up to its end
  __device__ __forceinline__ int all(const ScoreParams& p) const { return (p.n + kBlocks - 1) / kBlocks; }
  __device__ __forceinline__ void begin(const ScoreParams& p, const Shared& s) {
    const int units = p.batch * p.token_tiles;
    const bool counted = units <= kUnits;
    const long long work = (counted ? (long long)s.upto[units] : (long long)units * all(p)) * p.kv_heads;
    at = work / gridDim.x * blockIdx.x + min((long long)blockIdx.x, work % gridDim.x);
    end = at + work / gridDim.x + (blockIdx.x < work % gridDim.x ? 1 : 0);
    if (at >= end) return;
    if (!counted) {
      const long long one = (long long)all(p) * p.kv_heads;
      unit = (int)(at / one);
      upto0 = 0;  // (counted from the unit's begin on)
      upto1 = all(p);
      at -= unit * one;
      end -= unit * one;
    } else {
      unit = 0;  // the last with no more before it
      for (int high = units; high - unit > 1;) {
        const int mid = (unit + high) / 2;
        if ((long long)s.upto[mid] * p.kv_heads <= at) unit = mid;
        else high = mid;
      }
      upto0 = s.upto[unit];
      upto1 = s.upto[unit + 1];
    }
  }
  __device__ __forceinline__ bool next(const ScoreParams& p, const Shared& s, Item& it) {
    if (at >= end) return false;
    const int tiles = upto1 - upto0;
    const long long in = at - (long long)upto0 * p.kv_heads;
    it.b = unit / p.token_tiles;
    it.t0 = (unit - it.b * p.token_tiles) * p.tile_tokens;
    it.tokens = min(p.tile_tokens, p.tokens - it.t0);
    it.head = (int)(in / tiles);
    it.j0 = (int)(in - (long long)it.head * tiles);
    it.j1 = (int)min((long long)tiles, it.j0 + end - at);
    at += it.j1 - it.j0;
    if (at == (long long)upto1 * p.kv_heads && at < end) {
      if (p.batch * p.token_tiles > kUnits) {
        at = 0;
        end -= (long long)upto1 * p.kv_heads;
        ++unit;
      } else {
        do {
          ++unit;
          upto0 = upto1;
          upto1 = s.upto[unit + 1];
        } while (upto1 == upto0);
      }
    }
    return true;
  }
};

// The rows of an item's query tile that are in use, up to the last one.
__device__ __forceinline__ int used_rows(const ScoreParams& p, const Item& it) {
  return it.tokens > p.half_tokens ? p.half_rows + (it.tokens - p.half_tokens) * p.group_room : it.tokens * p.group_room;
}

// Where a block's bounds lie, in elements, or -1 where its page is outside the cache.
__device__ __forceinline__ long long bounds_at(const ScoreParams& p, int page, int j, int head, int dim) {
  if ((unsigned)page >= (unsigned)p.pages) return -1;
  return ((((long long)page << p.of_page_shift) + (j & ((1 << p.of_page_shift) - 1))) * p.kv_heads + head) * (2 * dim);
}

// Warps 8-11: bounds into the ring. A warp brings 32 blocks of every tile: lane l looks block l up, a tile ahead, and takes
// piece l % 8 of every fourth block of a K block.
template <int D>
__device__ __forceinline__ void bring_bounds(const ScoreParams& p, const Block& k, const Shared& s) {
  using S = Shape<D>;
  const int lane = threadIdx.x & 31, mine = (threadIdx.x >> 5) - kProducer0, piece = lane & 7, row0 = 32 * mine + (lane >> 3);
  Items ahead;
  ahead.begin(p, s);
  Item a;
  bool more = ahead.next(p, s, a);
  auto look_up = [&]() -> int {  // the page of this lane's block of the tile ahead (its first block's, behind the row's end)
    const int j = a.j0 * kBlocks + 32 * mine + lane;
    return j < p.n ? __ldg(p.table + a.b * p.table_stride + (j >> p.of_page_shift)) : -1;
  };
  int page = more ? look_up() : 0;
  Ring<S::kStages> st;
  unsigned g = 0;  // stages filled
  while (uniform((int)more)) {
    const long long at = bounds_at(p, page, a.j0 * kBlocks + 32 * mine + lane, a.head, D);
    long long from[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) from[i] = __shfl_sync(0xffffffffu, at, 4 * i + (lane >> 3));
    if (++a.j0 == a.j1) more = ahead.next(p, s, a);
    if (more) page = look_up();
#pragma unroll 1
    for (int step = 0; step < S::kSteps; ++step, ++g) {
      if (g >= S::kStages && !k.wait(kEmpty + st.i, st.parity ^ 1)) {
        cp_wait<0>();
        return;
      }
      const uint32_t to = k.ring + st.i * S::kStage + row0 * 128;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = row0 + 4 * i;
        const __nv_bfloat16* src = p.bounds + (from[i] < 0 ? 0 : from[i] + S::k_block(step) * 64 + piece * 8);
        cp16(to + i * 512 + ((piece ^ (r & 7)) << 4), src, from[i] < 0 ? 0 : 16);
      }
      // the copies announce themselves, a thread's when they are all there
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(k.bar(kFull + st.i)) : "memory");
      cp_commit();
      st.next();
    }
  }
  cp_wait<0>();
}

// 64 elements of the first N * kQueryPer query rows at most, of `rows` in use, and what is waited for before they are stored.
constexpr int kQueryPer = kQueryWarps * 32 / 8;  // rows that the threads cover, eight pieces each
template <int D, int N, typename F>
__device__ __forceinline__ bool bring_rows(const Block& k, const Shared& s, const __nv_bfloat16* q, int rows, int tokens, int part, F&& wait) {
  using S = Shape<D>;
  const int t = threadIdx.x - kQuery0 * 32, piece = t % 8;
  uint4 w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = t / 8 + i * kQueryPer;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && s.token[r] < tokens) w[i] = __ldg(reinterpret_cast<const uint4*>(q + s.row[r] + part * 64 + piece * 8));
  }
  __syncwarp();
  if (!wait()) return false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = t / 8 + i * kQueryPer;
    if (r >= rows) continue;
    unsigned char* to = k.smem + part * S::kQueries + r * 128 + ((piece ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(to) = make_uint4(part_of_pair(w[i].x, false), part_of_pair(w[i].y, false), part_of_pair(w[i].z, false), part_of_pair(w[i].w, false));
    *reinterpret_cast<uint4*>(to + S::kParts * S::kQueries) =
        make_uint4(part_of_pair(w[i].x, true), part_of_pair(w[i].y, true), part_of_pair(w[i].z, true), part_of_pair(w[i].w, true));
  }
  return true;
}

// Warps 12-14: an item's query rows, 64 elements of all of them after the other. Row half_rows * h + i is row i of the h-th half
// of the tile's tokens. The item before still needs what is there: meanwhile the first rows are loaded.
template <int D>
__device__ __forceinline__ void bring_queries(const ScoreParams& p, const Block& k, const Shared& s) {
  using S = Shape<D>;
  constexpr int kSome = 4;
  static_assert(22 * kQueryPer >= kRows, "all rows at once");
  Items items;
  items.begin(p, s);
  Item it;
  for (unsigned n = 0; uniform((int)items.next(p, s, it)); ++n) {
    const __nv_bfloat16* q = score_query(p, it.b, it.t0, it.head, 0);
    const int rows = uniform(used_rows(p, it));
#pragma unroll 1
    for (int part = 0; part < S::kParts; ++part) {
      auto wait = [&] { return n == 0 || k.wait(kQEmpty + part, (n - 1) & 1); };
      if (!(rows <= kSome * kQueryPer ? bring_rows<D, kSome>(k, s, q, rows, it.tokens, part, wait)
            : rows <= 11 * kQueryPer  ? bring_rows<D, 11>(k, s, q, rows, it.tokens, part, wait)
                                      : bring_rows<D, 22>(k, s, q, rows, it.tokens, part, wait)))
        return;
      __syncwarp();
      bar_arrive(k.bar(kQFull + part));
    }
  }
}

// One K block's product: 64 elements, sixteen an instruction, and an arrival when it is done.
__device__ __forceinline__ void multiply_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 x, y;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"((unsigned)add), "r"(bar)
      : "memory");
}

// Warp 15: the products.
template <int D>
__device__ __forceinline__ void multiply(const ScoreParams& p, const Block& k, const Shared& s, uint32_t tmem) {
  using S = Shape<D>;
  Items items;
  items.begin(p, s);
  Item it;
  Ring<S::kStages> st;
  const uint64_t ring = operand(k.ring, 16), queries = operand(k.queries, 16);
  uint32_t g = 0;  // tiles
  bool ok = true;
  for (unsigned n = 0; ok && uniform((int)items.next(p, s, it)); ++n) {
    const uint32_t idesc = uniform(instr(false, false, (used_rows(p, it) + 15) / 16 * 16));
    const int tiles = uniform(it.j1 - it.j0);
#pragma unroll 1
    for (int i = 0; i < tiles && ok; ++i, ++g) {
      if (g >= 2 && !k.wait(kSumEmpty + (g & 1), (g >> 1 & 1) ^ 1)) { ok = false; break; }
#pragma unroll 1
      for (int step = 0; step < S::kSteps; ++step) {
        if (i == 0 && (step & 1) == 0 && !k.wait(kQFull + (step >> 1), n & 1)) { ok = false; break; }
        if (!k.wait(kFull + st.i, st.parity)) { ok = false; break; }
        proxy_fence();
        tc_fence_after();
        multiply_step(tmem + (g & 1) * kRows, ring + (uint32_t)(st.i * (S::kStage >> 4)), queries + (uint32_t)(S::k_block(step) * (S::kQueries >> 4)), idesc, step > 0,
                      k.bar(kEmpty + st.i));
        if (i == tiles - 1 && (step & 1)) tc_commit(k.bar(kQEmpty + (step >> 1)));
        st.next();
      }
      if (ok) tc_commit(k.bar(kSumFull + (g & 1)));
    }
  }
  // nothing may be under way when tensor memory is freed
  tc_commit(k.bar(kFinal));
  k.wait(kFinal, 0);
}

// Warps 0-7: maxima over a token's heads, and the stores. Warps w and w + 4 have the lanes (blocks) 32w .. 32w + 31, and each
// one half's columns. GROUP: columns of a token, a power of two; 32: or some thirty-twos. (Heads that are not a power of two
// are filled up with the last one again, which changes no maximum: of 7 heads and 4 * 200 tokens of size 64 over up to 1250
// blocks 17 us, 49 where columns were counted.) 32 columns are on their way while the 32 before them are joined. Most tiles hold
// blocks that all their tokens see, and that are not picked anyway: what their scores go through is kept short (2048 tokens of
// 32 heads over 2048 blocks 58 us, 131 by the whole way for all of them).
template <int GROUP>
__device__ __forceinline__ void take_maxima(const ScoreParams& p, const Block& k, Shared& s, uint32_t tmem) {
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31, quarter = warp & 3, half = warp >> 2;
  Items items;
  items.begin(p, s);
  Item it;
  int* seen_s = s.seen[warp];
  uint32_t g = 0;
  while (uniform((int)items.next(p, s, it))) {
    const int tokens = uniform(min(p.half_tokens, it.tokens - half * p.half_tokens)), first = it.t0 + half * p.half_tokens;
    const int chunks = tokens <= 0 ? 0 : uniform((tokens * p.group_room + 31) / 32), each = GROUP < 32 ? 1 : p.group_room / 32;
    int least = p.n;  // blocks that all of these tokens see, and that are not among the last ones of any
    __syncwarp();
    for (int t = lane; t < tokens; t += 32) {
      bool bad = false;
      const int seen = blocks_seen(p, it.b, first + t, bad);
      seen_s[t] = seen;
      least = min(least, seen - p.last);
    }
    least = __reduce_min_sync(0xffffffffu, least);
    __syncwarp();
    const long long stride = (long long)p.kv_heads * p.n;
    const int j1 = uniform(it.j1);
    auto page_of = [&](int j) -> int { return j < p.n ? __ldg(p.table + it.b * p.table_stride + (j >> p.of_page_shift)) : 0; };
    int next_page = page_of(it.j0 * kBlocks + 32 * quarter + lane);  // (looked up a tile ahead)
    for (int i = uniform(it.j0); i < j1; ++i, ++g) {
      const int j0 = i * kBlocks + 32 * quarter, j = j0 + lane, page = next_page;
      if (i + 1 < j1) next_page = page_of(j + kBlocks);
      if (!k.wait(kSumFull + (g & 1), g >> 1 & 1)) return;
      tc_fence_after();
      const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + (g & 1) * kRows + half * p.half_rows;
      float* to = p.out + (((long long)it.b * p.tokens + first) * p.kv_heads + it.head) * p.n + j;
      const bool there = (unsigned)page < (unsigned)p.pages;
      const bool simple = !p.join && j0 >= p.first && j0 + 32 <= least && __all_sync(0xffffffffu, there);
      bool missing = false;
      auto put = [&](float x, int t) {
        const int seen = seen_s[t];
        x = final_score(p, x, j, seen);
        if (!there) {
          missing |= j < seen;
          x = -INFINITY;
        }
        if (j < p.n) {
          if (p.join) x = fmaxf(x, *to);
          *to = x;
        }
        to += stride;
      };
      float top = -INFINITY;  // of the token's columns so far
      int in = 0;             // and how many thirty-twos
      auto join = [&](const uint32_t (&x)[32], int c) {
        float m[32 / GROUP];
#pragma unroll
        for (int u = 0; u < 32 / GROUP; ++u) {
          m[u] = __uint_as_float(x[u * GROUP]);
#pragma unroll
          for (int e = 1; e < GROUP; ++e) m[u] = max_nan(m[u], __uint_as_float(x[u * GROUP + e]));
        }
        int t0 = c * (32 / GROUP);
        if (GROUP == 32) {
          m[0] = max_nan(m[0], top);
          top = m[0];
          if (++in < each) return;
          in = 0;
          top = -INFINITY;
          t0 = c / each;
        }
        if (simple && t0 + 32 / GROUP <= tokens) {
#pragma unroll
          for (int u = 0; u < 32 / GROUP; ++u) {
            const float x = m[u] == m[u] ? m[u] : INFINITY;
            if (p.stream_out) __stcs(to, x);
            else *to = x;
            to += stride;
          }
        } else {
#pragma unroll
          for (int u = 0; u < 32 / GROUP; ++u)
            if (t0 + u < tokens) put(m[u], t0 + u);
        }
      };
      if (chunks > 0) {
        uint32_t x[32], y[32];
        __syncwarp();
        tc_ld32(x, from);
#pragma unroll 1
        for (int c = 0; c < chunks; c += 2) {
          tc_wait_ld();
          __syncwarp();
          if (c + 1 < chunks) tc_ld32(y, from + 32 * (c + 1));
          join(x, c);
          if (c + 1 < chunks) {
            tc_wait_ld();
            __syncwarp();
            if (c + 2 < chunks) tc_ld32(x, from + 32 * (c + 2));
            join(y, c + 1);
          }
        }
      }
      if (missing && j < p.n) report(p.status, kStatIndexBit);
      tc_fence_before();
      __syncwarp();
      if (!(p.test_skip_arrive && g == 0)) bar_arrive(k.bar(kSumEmpty + (g & 1)));
    }
  }
}

template <int D, int GROUP>
__global__ void __launch_bounds__(kThreads, 1) score_tiles_kernel(const __grid_constant__ ScoreParams p) {
  using S = Shape<D>;
  extern __shared__ unsigned char raw[];
  __shared__ Shared s;
  unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  Block k;
  k.smem = smem;
  k.queries = smem_addr(smem);
  k.ring = k.queries + S::kRing;
  k.bars = smem_addr(s.bars);
  k.status = p.status;
  k.limit = p.spin_limit_ns;
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (warp == kMulWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      bar_init(k.bar(kFull + i), 4 * 32);
      bar_init(k.bar(kEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(k.bar(kSumFull + i), 1);
      bar_init(k.bar(kSumEmpty + i), kMaxWarps);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(k.bar(kQFull + i), kQueryWarps);
      bar_init(k.bar(kQEmpty + i), 1);
    }
    bar_init(k.bar(kFinal), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  grid_wait();
  grid_launch_dependents();

  if (threadIdx.x < kRows) {
    const int r = threadIdx.x, half = r / p.half_rows, in = r - half * p.half_rows, tl = in / p.group_room, token = half * p.half_tokens + tl;
    s.token[r] = half < 2 ? token : INT_MAX;
    s.row[r] = token * p.q_token + min(in - tl * p.group_room, p.group - 1) * p.q_head;
  }
  // how many tiles of blocks the tiles of tokens see
  const int units = p.batch * p.token_tiles, all = (p.n + kBlocks - 1) / kBlocks;
  if (units <= kUnits) {
    for (int u = threadIdx.x; u <= units; u += kThreads) s.upto[u] = 0;
    __syncthreads();
    const int tokens = p.batch * p.tokens;  // (no more than units * tokens of a tile)
#pragma unroll 4
    for (int i = threadIdx.x; i < (tokens + 31) / 32 * 32; i += kThreads) {
      const int b = min(i, tokens - 1) / p.tokens, t = min(i, tokens - 1) - b * p.tokens, u = b * p.token_tiles + t / p.tile_tokens;
      bool bad = false;
      const int tiles = (blocks_seen(p, b, t, bad) + kBlocks - 1) / kBlocks;
      const int most = __reduce_max_sync(0xffffffffu, tiles);
      if (__shfl_sync(0xffffffffu, u, 0) == __shfl_sync(0xffffffffu, u, 31)) {
        if (lane == 0) atomicMax(&s.upto[u + 1], most);
      } else {
        atomicMax(&s.upto[u + 1], tiles);
      }
    }
    __syncthreads();
    if (warp == 0) {
      int sum = 0;
      if (lane == 0) s.upto[0] = 0;
      for (int u0 = 0; u0 < units; u0 += 32) {
        int x = u0 + lane < units ? s.upto[u0 + lane + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (u0 + lane < units) s.upto[u0 + lane + 1] = sum + x;
        sum += __shfl_sync(0xffffffffu, x, 31);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s.tmem);

  if (warp < kMaxWarps) {
    // the rows' lengths, a lane each
    const int rows = p.batch * p.tokens * p.kv_heads, warps = gridDim.x * kMaxWarps, mine = warp * gridDim.x + blockIdx.x;
    for (long long r = mine * 32LL + lane; r < rows; r += warps * 32LL) {
      const int bt = (int)r / p.kv_heads, b = bt / p.tokens;
      bool bad = false;
      const int seen = blocks_seen(p, b, bt - b * p.tokens, bad);
      if (bad) report(p.status, kStatRowLenBit);
      if (p.row_len) p.row_len[r] = seen;
    }
    // the tiles of blocks that no token of a tile sees, a row each warp
    if (units <= kUnits && s.upto[units] < units * (long long)all)
      for (long long r = mine; r < rows; r += warps) {
        const int bt = (int)r / p.kv_heads, b = bt / p.tokens, u = b * p.token_tiles + (bt - b * p.tokens) / p.tile_tokens;
        for (long long j = (long long)(s.upto[u + 1] - s.upto[u]) * kBlocks + lane; j < p.n; j += 32) p.out[r * p.n + j] = -INFINITY;
      }
    take_maxima<GROUP>(p, k, s, tmem);
  } else if (warp < kQuery0) {
    bring_bounds<D>(p, k, s);
  } else if (warp < kMulWarp) {
    bring_queries<D>(p, k, s);
  } else {
    multiply<D>(p, k, s, tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMulWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D, int GROUP>
cudaError_t launch(const ScoreParams& p, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute a[2] = {};
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, 0);
  return cudaLaunchKernelEx(&cfg, score_tiles_kernel<D, GROUP>, p);
}
template <int D>
cudaError_t launch_dim(const ScoreParams& p, int sms, cudaStream_t stream) {
  switch (p.group_room) {
    case 1: return launch<D, 1>(p, sms, stream);
    case 2: return launch<D, 2>(p, sms, stream);
    case 4: return launch<D, 4>(p, sms, stream);
    case 8: return launch<D, 8>(p, sms, stream);
    case 16: return launch<D, 16>(p, sms, stream);
    default: return launch<D, 32>(p, sms, stream);
  }
}
template <int D>
cudaError_t opt_in() {
  cudaError_t e = cudaSuccess;
  for (auto kernel : {score_tiles_kernel<D, 1>, score_tiles_kernel<D, 2>, score_tiles_kernel<D, 4>, score_tiles_kernel<D, 8>, score_tiles_kernel<D, 16>,
                      score_tiles_kernel<D, 32>})
    if (e == cudaSuccess) e = allow(kernel, Shape<D>::kSmem);
  return e;
}

}  // namespace

cudaError_t setup_score_tiles() {
  const cudaError_t e = opt_in<64>();
  return e != cudaSuccess ? e : opt_in<128>();
}

cudaError_t launch_score_tiles(const ScoreParams& p, int head_dim, int sms, cudaStream_t stream) {
  return head_dim == 64 ? launch_dim<64>(p, sms, stream) : launch_dim<128>(p, sms, stream);
}

}  // namespace attn
}  // namespace tks
