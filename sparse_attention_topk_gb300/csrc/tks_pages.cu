// Page tables of a step's new sequences, moving pages in use together, and
// copying pages.
//
// The two calls that make tables are a few passes over the tables and over the
// pages, with nothing between them but that all of one is done before the next
// begins: one thread-block cluster makes them, in one launch, its barrier between
// the passes; small tables a single thread block. Who holds a page is a bit:
// every thread block sets the bits of its part of the rows in its own shared
// memory, and after the one barrier reads all of them. Then each knows by itself
// how many pages of a kind lie before each 32, and so the r-th free page, or the
// number of moving pages before one. Where the bits, or a fork's children, do not
// fit into shared memory, there is a word for each page in the caller's scratch
// buffer instead, and a barrier more; nothing is shared between calls.
//
// What bounds it: latency, of launch, barrier and loads that wait for each other.
// Measured: 64 beams of 16 prompts over up to 65,536 positions in pages of 64 8.8 us
// (12.4 by words: the scattered stores and the counts over them take longest); a pool
// of 8192 pages compacted 6.9 us (11.5 by words); a few short beams 4.4 us (7.4 by words
// and cluster), a pool of 639 pages compacted 4.4 (9.2). Many: 2048 rows of 1024 pages
// forked in 88 us, 319 by words.
// Copies: 2048 pages of 135 KB 92 us, 6.0 TB/s; more under way (five or six thread blocks
// an SM instead of four) 95.

#include <algorithm>
#include <iterator>

#include "tks_attn.cuh"
#include "tks_attn_host.h"

namespace tks {
namespace attn {
namespace {

constexpr int kBlocks = 8, kThreads = 1024, kWarps = kThreads / 32;
constexpr int kFree = 0x7fffffff, kShared = -1;  // a page that nobody holds; one that is held and not to be written to

// Of 32 pages: those that are free (fork), or held (compact), those that move (compact), and how many of either lie before
// them in the warp's run of pages.
struct __align__(16) Tally {
  uint32_t a, b;
  int before_a, before_b;
};

struct PlanParams {
  const int32_t* table;
  long long table_stride;
  int table_pages, sequences;
  const int32_t *lens, *parents, *new_lens;
  int children;
  const uint8_t* keep;
  int pages, page_shift;
  int32_t *out, *src, *dst, *count;
  int lanes, spans;  // how rows are cut up (kLanes)
  int words;         // of a bit for each page, a multiple of four
  // scratch: what the warps have counted, 32 pages' tallies, a word a page, a word a child
  int32_t* sums;
  Tally* tallies;
  int32_t *owner, *base;
  unsigned* status;
};

// The threads of a cluster, or (ONE) of a single thread block; the barrier also orders their accesses to global memory.
template <bool ONE>
struct Team {
  static constexpr int kBlocksOf = ONE ? 1 : kBlocks, kAllWarps = kBlocksOf * kWarps, kAllThreads = kBlocksOf * kThreads;
  int rank, warp, lane, thread;  // warps and threads of all its blocks
  __device__ __forceinline__ Team() {
    rank = ONE ? 0 : blockIdx.x;
    warp = rank * kWarps + (threadIdx.x >> 5);
    lane = threadIdx.x & 31;
    thread = rank * kThreads + threadIdx.x;
  }
  __device__ __forceinline__ void meet() const {
    if (ONE) {
      __syncthreads();
    } else {
      __syncwarp();
      cluster_sync();
    }
  }
};
using Cluster = Team<false>;
constexpr int kAllWarps = Cluster::kAllWarps;

// Of two numbers that each warp of the cluster has counted: the sums over the warps before each one, in shared memory.
struct Sums {
  int a[kAllWarps + 1], b[kAllWarps + 1], warps[2][kAllWarps / 32];
};
__device__ __forceinline__ void sum_up(const Cluster& me, const PlanParams& p, Sums& s, int a, int b) {
  if (me.lane == 0) {
    p.sums[me.warp] = a;
    p.sums[kAllWarps + me.warp] = b;
  }
  me.meet();
  const int t = threadIdx.x, w = t >> 5;
  int x = 0, y = 0;
  if (t < kAllWarps) {
    x = __ldcg(p.sums + t);
    y = __ldcg(p.sums + kAllWarps + t);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (me.lane >= o) {
        x += u;
        y += v;
      }
    }
    if (me.lane == 31) {
      s.warps[0][w] = x;
      s.warps[1][w] = y;
    }
  }
  __syncthreads();
  if (t < kAllWarps) {
    for (int i = 0; i < w; ++i) {
      x += s.warps[0][i];
      y += s.warps[1][i];
    }
    s.a[t + 1] = x;
    s.b[t + 1] = y;
    if (t == 0) s.a[0] = s.b[0] = 0;
  }
  __syncthreads();
}
// A warp's run of n things, in order: [begin, end), begin a multiple of 32.
__device__ __forceinline__ int share(int n) { return (int)((((long long)n + kAllWarps - 1) / kAllWarps + 31) / 32 * 32); }
__device__ __forceinline__ void share(const Cluster& me, int n, int& begin, int& end) {
  const long long each = share(n);
  begin = (int)min((long long)n, each * me.warp);
  end = (int)min((long long)n, each * (me.warp + 1));
}
// The place of the n-th set bit (n < the bits' number).
__device__ __forceinline__ int nth_bit(uint32_t bits, int n) {
  int at = 0;
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    const int low = __popc(bits & ((1u << w) - 1u));
    if (n >= low) {
      n -= low;
      bits >>= w;
      at += w;
    }
  }
  return at;
}
// The free page of this rank (FORK: of the tallies' a; else, a being held ones, of those without a bit there, below page `end`).
template <bool FORK>
__device__ __forceinline__ int free_page(const PlanParams& p, const Sums& s, int rank) {
  const int each = share(p.pages);
  int run = 0;
#pragma unroll
  for (int step = kAllWarps / 2; step; step >>= 1)
    if ((FORK ? s.a[run + step] : (int)min((long long)p.pages, (long long)each * (run + step)) - s.a[run + step]) <= rank) run += step;
  rank -= FORK ? s.a[run] : (int)min((long long)p.pages, (long long)each * run) - s.a[run];
  const int first = run * (each / 32);
  int low = 0, high = min(each / 32, (p.pages + 31) / 32 - first);
  while (high - low > 1) {  // (the last 32 with no more before them than the rank)
    const int mid = (low + high) / 2, before = __ldcg(&p.tallies[first + mid].before_a);
    if ((FORK ? before : 32 * mid - before) <= rank) low = mid;
    else high = mid;
  }
  const uint4 t = __ldcg(reinterpret_cast<const uint4*>(p.tallies + first + low));
  rank -= FORK ? (int)t.z : 32 * low - (int)t.z;
  return (first + low) * 32 + nth_bit(FORK ? t.x : ~t.x, rank);
}

__device__ __forceinline__ int pages_of(const PlanParams& p, int len) { return (int)(((long long)len + (1 << p.page_shift) - 1) >> p.page_shift); }
__device__ __forceinline__ int held_len(const PlanParams& p, int len, bool& bad) {
  const long long room = (long long)p.table_pages << p.page_shift;
  const int r = len < 0 ? 0 : len > room ? (int)room : len;
  bad |= r != len;
  return r;
}

// A child: its parent's row, how many of its entries it keeps, how many it needs, and whether it writes to the last.
struct Child {
  const int32_t* row;
  int have, need;
  bool writes;
};
__device__ __forceinline__ Child child_of(const PlanParams& p, int i, unsigned* bad) {
  Child c;
  const int parent = __ldg(p.parents + i);
  bool len_bad = false;
  const int wanted = held_len(p, __ldg(p.new_lens + i), len_bad);
  int had = 0;
  c.row = p.table;
  if (parent >= 0 && parent < p.sequences) {
    had = held_len(p, __ldg(p.lens + parent), len_bad);
    c.row = p.table + parent * p.table_stride;
  } else if (parent >= 0 && bad) {
    *bad |= kStatIndexBit;
  }
  if (len_bad && bad) *bad |= kStatRowLenBit;
  const int kept = min(had, wanted);
  c.have = pages_of(p, kept);
  c.need = pages_of(p, wanted);
  c.writes = (kept & ((1 << p.page_shift) - 1)) != 0 && wanted > kept;
  return c;
}

// What a warp does at once: a span of one row, kLanes entries a lane; where that left warps without a span (compact), fewer.
constexpr int kLanes = 8;
// The entry that a child writes to, or -1.
__device__ __forceinline__ int tail_of(const PlanParams& p, const Child& c) {
  const int e = c.writes ? __ldg(c.row + c.have - 1) : -1;
  return (unsigned)e < (unsigned)p.pages ? e : -1;
}

// Of a number of each thread of a block: the sum over the threads before it, and over all. (warps: for this call alone)
__device__ __forceinline__ int sum_before(int x, int (&warps)[kWarps], int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int end = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += y;
  }
  if (lane == 31) warps[warp] = end;
  __syncthreads();
  const int w = warps[lane];
  all = __reduce_add_sync(0xffffffffu, w);
  return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + end - x;
}

// Children that a thread block keeps in shared memory, looked up once (each look goes through three loads that wait for each
// other: parent, length, entry).
constexpr int kHeldChildren = 2048;
template <int N>
struct Children {
  int parent[N], have[N], need[N], tail[N], base[N], warps[kWarps];  // (tail: as above; later, the entry that is copied)
  __device__ __forceinline__ void look_up(const PlanParams& p, unsigned* bad) {
    for (int i = threadIdx.x; i < p.children; i += kThreads) {
      const Child c = child_of(p, i, bad);
      parent[i] = c.have > 0 ? __ldg(p.parents + i) : 0;
      have[i] = c.have;
      need[i] = c.need;
      tail[i] = tail_of(p, c);
    }
  }
  __device__ __forceinline__ Child child(const PlanParams& p, int i, int& written) const {
    written = tail[i];
    return Child{p.table + parent[i] * p.table_stride, have[i], need[i], written >= 0};
  }
  // Into base: whether a child before writes to the same page.
  __device__ __forceinline__ void look_for_writers(const PlanParams& p) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < p.children; i += kWarps) {
      const int e = tail[i];
      bool is = false;
      if (e >= 0)
        for (int j = lane; j < i; j += 32) is |= tail[j] == e;
      is = __any_sync(0xffffffffu, is);
      if (lane == 0) base[i] = is;
    }
  }
  // The pages that the children before each one want, and that all do; copied(i): whether child i's tail, which it has, is copied.
  template <typename F>
  __device__ __forceinline__ int sum_up(const PlanParams& p, F copied) {
    constexpr int kMine = (N + kThreads - 1) / kThreads;
    int n[kMine], sum = 0, all;
    bool copy[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = threadIdx.x * kMine + k;
      n[k] = 0;
      copy[k] = i < p.children && tail[i] >= 0 && copied(i);
      if (i < p.children) n[k] = need[i] - have[i] + (copy[k] ? 1 : 0);
      sum += n[k];
    }
    int at = sum_before(sum, warps, all);  // (all threads have looked at the tails)
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = threadIdx.x * kMine + k;
      if (i < p.children) {
        base[i] = at;
        if (!copy[k]) tail[i] = -1;
      }
      at += n[k];
    }
    __syncthreads();
    return all;
  }
};

__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const __grid_constant__ PlanParams p) {
  __shared__ Sums sums;
  const Cluster me;
  unsigned bad = 0;
  grid_wait();
  grid_launch_dependents();
  // who holds a page: nobody yet
  for (int i = me.thread; i < p.pages; i += me.kAllThreads) p.owner[i] = p.keep && p.keep[i] ? kShared : kFree;
  auto child = [&](int i, int& tail, unsigned* bad) -> Child {
    const Child c = child_of(p, i, bad);
    tail = tail_of(p, c);
    return c;
  };
  me.meet();
  constexpr int span = 32 * kLanes;
  const int spans = p.spans, units = p.children * spans;
  for (int u = me.warp; u < units; u += kAllWarps) {
    const int i = u / spans, j0 = (u - i * spans) * span;
    int tail;
    const Child c = child(i, tail, j0 == 0 ? &bad : nullptr);
    int e[kLanes];
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = j < c.have ? __ldg(c.row + j) : -1;
      if (j < c.have && (unsigned)e[k] >= (unsigned)p.pages) bad |= kStatIndexBit;
    }
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      if ((unsigned)e[k] >= (unsigned)p.pages) continue;
      // (a held page's word only ever falls: to kShared, or to the lowest of those who write to it)
      if (tail >= 0 && j0 + 32 * k + me.lane == c.have - 1) atomicMin(p.owner + e[k], i);
      else p.owner[e[k]] = kShared;
    }
  }
  me.meet();
  // how many pages each child wants, and how many are free
  auto wants = [&](int i, bool& copied) -> int {
    int tail;
    const Child c = child(i, tail, nullptr);
    copied = tail >= 0 && __ldcg(p.owner + tail) != i;
    return c.need - c.have + (copied ? 1 : 0);
  };
  int page0, page1, child0 = 0, child1 = 0;
  share(me, p.pages, page0, page1);
  int free = 0, wanted = 0;
#pragma unroll 4
  for (int i = page0; i < page1; i += 32) {
    const uint32_t m = __ballot_sync(0xffffffffu, i + me.lane < page1 && __ldcg(p.owner + i + me.lane) == kFree);
    if (me.lane == 0) p.tallies[i / 32] = Tally{m, 0, free, 0};
    free += __popc(m);
  }
  bool copied;
  share(me, p.children, child0, child1);
  for (int i = child0 + me.lane; i < child1; i += 32) wanted += wants(i, copied);
  sum_up(me, p, sums, free, __reduce_add_sync(0xffffffffu, wanted));
  int at = sums.b[me.warp];
  for (int i = child0; i < child1; i += 32) {
    const int n = i + me.lane < child1 ? wants(i + me.lane, copied) : 0;
    int end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (me.lane >= o) end += y;
    }
    if (i + me.lane < child1) p.base[i + me.lane] = at + end - n;
    at += __shfl_sync(0xffffffffu, end, 31);
  }
  wanted = sums.b[kAllWarps];
  me.meet();
  const int most = sums.a[kAllWarps];  // pages to hand out
  if (wanted > most) bad |= kStatNoPageBit;
  for (int u = me.warp; u < units; u += kAllWarps) {
    const int i = u / spans, j0 = (u - i * spans) * span;
    int tail;
    const Child c = child(i, tail, nullptr);
    const int base = __ldcg(p.base + i);
    const bool copy = tail >= 0 && __ldcg(p.owner + tail) != i;
    int32_t* to = p.out + (long long)i * p.table_pages;
    int e[kLanes];
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = j < c.have ? __ldg(c.row + j) : -1;
    }
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      const int j = j0 + 32 * k + me.lane;
      if (j >= p.table_pages) continue;
      if ((copy && j == c.have - 1) || (j >= c.have && j < c.need)) {
        const int rank = base + (j < c.have ? 0 : (copy ? 1 : 0) + j - c.have);
        const int got = rank < most ? free_page<true>(p, sums, rank) : -1;
        if (j < c.have) {
          p.src[i] = got < 0 ? -1 : e[k];
          p.dst[i] = got;
        }
        e[k] = got;
      }
      to[j] = e[k];
    }
    if (!copy && j0 == 0 && me.lane == 0) p.src[i] = p.dst[i] = -1;
  }
  if (bad) report(p.status, bad);
}

__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const __grid_constant__ PlanParams p) {
  __shared__ Sums sums;
  const Cluster me;
  unsigned bad = 0;
  grid_wait();
  grid_launch_dependents();
  auto pinned = [&](int i) { return p.keep && p.keep[i] != 0; };
  for (int i = me.thread; i < p.pages; i += me.kAllThreads) p.owner[i] = pinned(i) ? kShared : kFree;
  me.meet();
  const int lanes = p.lanes, span = 32 * lanes, spans = p.spans, units = p.sequences * spans;
  auto pages_held = [&](int s, bool tell) {
    bool len_bad = false;
    const int n = pages_of(p, held_len(p, __ldg(p.lens + s), len_bad));
    if (len_bad && tell) bad |= kStatRowLenBit;
    return n;
  };
  for (int u = me.warp; u < units; u += kAllWarps) {
    const int s = u / spans, j0 = (u - s * spans) * span;
    const int have = pages_held(s, j0 == 0);
    const int32_t* row = p.table + s * p.table_stride;
    int e[kLanes];
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = k < lanes && j < have ? row[j] : -1;
      if (k < lanes && j < have && (unsigned)e[k] >= (unsigned)p.pages) bad |= kStatIndexBit;
    }
#pragma unroll
    for (int k = 0; k < kLanes; ++k)
      if ((unsigned)e[k] < (unsigned)p.pages) p.owner[e[k]] = kShared;
  }
  me.meet();
  int page0, page1, held = 0, movable = 0;
  share(me, p.pages, page0, page1);
#pragma unroll 4
  for (int i0 = page0; i0 < page1; i0 += 32) {
    const int i = i0 + me.lane;
    const bool is = i < page1 && __ldcg(p.owner + i) != kFree;
    const uint32_t a = __ballot_sync(0xffffffffu, is), b = __ballot_sync(0xffffffffu, is && !pinned(i));
    if (me.lane == 0) p.tallies[i0 / 32] = Tally{a, b, held, movable};
    held += __popc(a);
    movable += __popc(b);
  }
  sum_up(me, p, sums, held, movable);
  const int used = sums.a[kAllWarps], each = share(p.pages);
  // movable pages before page i
  auto before = [&](int i, const uint4& t) { return sums.b[i / each] + (int)t.w + __popc(t.y & ((1u << (i & 31)) - 1u)); };
  auto tally = [&](int i) { return __ldcg(reinterpret_cast<const uint4*>(p.tallies + i / 32)); };
  const int below = used < p.pages ? before(used, tally(used)) : sums.b[kAllWarps];
  const int count = sums.b[kAllWarps] - below;
  if (me.thread == 0) {
    p.count[0] = count;
    p.count[1] = used;
  }
  for (int i = count + me.thread; i < p.pages / 2; i += me.kAllThreads) p.src[i] = p.dst[i] = -1;
  for (int i = used + me.thread; i < p.pages; i += me.kAllThreads) {
    const uint4 t = tally(i);
    if (!(t.y >> (i & 31) & 1u)) continue;
    const int rank = before(i, t) - below;
    p.src[rank] = i;
    p.dst[rank] = free_page<false>(p, sums, rank);
  }
  me.meet();
  for (int u = me.warp; u < units; u += kAllWarps) {
    const int s = u / spans, j0 = (u - s * spans) * span;
    const int have = pages_held(s, false);
    const int32_t* row = p.table + s * p.table_stride;
    int32_t* out = p.out + (long long)s * p.table_pages;
    int e[kLanes], to[kLanes];
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = k < lanes && j < have ? row[j] : -1;  // (out may be the table itself)
    }
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {  // which of the moves, or none
      to[k] = -1;
      if (e[k] >= used && e[k] < p.pages) {
        const uint4 t = tally(e[k]);
        if (t.y >> (e[k] & 31) & 1u) to[k] = before(e[k], t) - below;
      }
    }
#pragma unroll
    for (int k = 0; k < kLanes; ++k)
      if (to[k] >= 0) e[k] = __ldcg(p.dst + to[k]);
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      const int j = j0 + 32 * k + me.lane;
      if (k < lanes && j < p.table_pages) out[j] = e[k];
    }
  }
  if (bad) report(p.status, bad);
}

// ---------------------------------------------------------------------------
// By bits: larger tables, of pools whose pages' bits fit into shared memory. Every thread block of the cluster sets a bit for each
// page that its part of the rows holds, in its own shared memory, and after the only barrier reads the others' bits, all of
// them: so each knows by itself which pages are free, and how many are before each 32.
// ---------------------------------------------------------------------------
constexpr int kBitPages = 352 * 1024;           // (of compact, five arrays of that many bits)
// That look for others who write to the same page among all before them, instead of by a word for each page (64 beams over up to
// 65,536 positions 8.8 us so and 9.3 otherwise; 40 short ones 8.3 and 8.5, 100 8.9 and 8.8, 256 10.8 and 9.1).
constexpr int kFewChildren = 64;
constexpr int kOnePages = 8192, kOneRows = 32;  // of tables that a single thread block makes, at most (one_block)

__device__ __forceinline__ uint4 ld_peer(uint32_t addr, unsigned rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(of_rank(addr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 either(const uint4& a, const uint4& b) { return make_uint4(a.x | b.x, a.y | b.y, a.z | b.z, a.w | b.w); }
// All thread blocks' bits, four words at q.
template <bool ONE>
__device__ __forceinline__ uint4 all_bits(const uint32_t* bits, int q) {
  if (ONE) return reinterpret_cast<const uint4*>(bits)[q];
  const uint32_t own = smem_addr(bits);
  uint4 x[kBlocks];
#pragma unroll
  for (int r = 0; r < kBlocks; ++r) x[r] = ld_peer(own + 16 * q, r);
#pragma unroll
  for (int r = 1; r < kBlocks; ++r) x[0] = either(x[0], x[r]);
  return x[0];
}
template <bool ONE>
__device__ __forceinline__ void peers_read() { if (!ONE) asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
template <bool ONE>
__device__ __forceinline__ void peers_have_read() { if (!ONE) asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void set_bit(uint32_t* bits, int page) { atomicOr(bits + (page >> 5), 1u << (page & 31)); }
// The bits of pages [32 w, 32 w + 32) that there are, and of those that `keep` holds.
__device__ __forceinline__ uint32_t real_pages(const PlanParams& p, int w) {
  const int n = p.pages - 32 * w;
  return n >= 32 ? ~0u : n > 0 ? (1u << n) - 1u : 0u;
}
__device__ __forceinline__ uint32_t kept(const PlanParams& p, int w) {
  if (!p.keep) return 0;
  uint32_t bits = 0;
  const int n = min(32, p.pages - 32 * w);
  if (n == 32 && (reinterpret_cast<uintptr_t>(p.keep) & 3) == 0) {
    const uint32_t* at = reinterpret_cast<const uint32_t*>(p.keep) + 8 * w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = __vcmpne4(__ldg(at + i), 0u) & 0x01010101u;
      bits |= ((m | m >> 7 | m >> 14 | m >> 21) & 0xfu) << (4 * i);
    }
  } else {
    for (int i = 0; i < n; ++i) bits |= (p.keep[32 * w + i] != 0 ? 1u : 0u) << i;
  }
  return bits;
}
// The place of the rank-th of: bits (SET), or places without one. before: the bits before each word.
template <bool SET>
__device__ __forceinline__ int nth(const uint32_t* bits, const int* before, int words, int rank) {
  int low = 0, high = words;
  while (high - low > 1) {
    const int mid = (low + high) / 2;
    if ((SET ? before[mid] : 32 * mid - before[mid]) <= rank) low = mid;
    else high = mid;
  }
  return 32 * low + nth_bit(SET ? bits[low] : ~bits[low], rank - (SET ? before[low] : 32 * low - before[low]));
}

// LANES: the entries of a row that a lane takes.
template <int LANES, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) fork_bits_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ Children<ONE ? kOneRows : kHeldChildren> held;
  __shared__ int warps[kWarps];
  const Team<ONE> me;
  const int words = p.words;  // a multiple of four
  // the pages that this thread block's rows hold without writing to them; all tails; all pages that are held so, then those free
  uint32_t *own = bits, *written = bits + words, *free = bits + 2 * words;
  int* before = reinterpret_cast<int*>(bits + 3 * words);
  unsigned bad = 0;
  grid_wait();
  grid_launch_dependents();
  for (int q = threadIdx.x; q < words / 2; q += kThreads) reinterpret_cast<uint4*>(bits)[q] = make_uint4(0u, 0u, 0u, 0u);
  held.look_up(p, me.rank == 0 ? &bad : nullptr);
  __syncthreads();
  if (p.keep)
    for (int w = me.thread; 32 * w < p.pages; w += me.kAllThreads) atomicOr(own + w, kept(p, w));
  for (int i = threadIdx.x; i < p.children; i += kThreads)
    if (held.tail[i] >= 0) set_bit(written, held.tail[i]);
  const bool few = ONE || p.children <= kFewChildren;
  if (few) {
    held.look_for_writers(p);
  } else if (me.rank == 0) {
    // the lowest of those who write to a page
    for (int i = threadIdx.x; i < p.children; i += kThreads)
      if (held.tail[i] >= 0) p.owner[held.tail[i]] = kFree;
    __syncthreads();
    for (int i = threadIdx.x; i < p.children; i += kThreads)
      if (held.tail[i] >= 0) atomicMin(p.owner + held.tail[i], i);
  }
  constexpr int span = 32 * LANES;
  const int spans = p.spans, units = p.children * spans;
  for (int u = me.warp; u < units; u += me.kAllWarps) {
    const int i = u / spans, j0 = (u - i * spans) * span;
    int tail;
    const Child c = held.child(p, i, tail);
    int e[LANES];
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = j < c.have ? __ldg(c.row + j) : -1;
      if (j < c.have && (unsigned)e[k] >= (unsigned)p.pages) bad |= kStatIndexBit;
    }
#pragma unroll
    for (int k = 0; k < LANES; ++k)
      if ((unsigned)e[k] < (unsigned)p.pages && !(tail >= 0 && j0 + 32 * k + me.lane == c.have - 1)) set_bit(own, e[k]);
  }
  me.meet();
  for (int q = threadIdx.x; q < words / 4; q += kThreads) reinterpret_cast<uint4*>(free)[q] = all_bits<ONE>(own, q);
  peers_read<ONE>();
  __syncthreads();
  const int wanted = held.sum_up(p, [&](int i) {
    const int e = held.tail[i];
    if (free[e >> 5] >> (e & 31) & 1u) return true;
    return few ? held.base[i] != 0 : __ldcg(p.owner + e) != i;
  });
  const int each = (words / 4 + kThreads - 1) / kThreads, q0 = min(words / 4, (int)threadIdx.x * each), q1 = min(words / 4, q0 + each);
  int sum = 0, most;
  for (int w = 4 * q0; w < 4 * q1; ++w) {
    const uint32_t x = ~(free[w] | written[w]) & real_pages(p, w);
    free[w] = x;
    sum += __popc(x);
  }
  int at = sum_before(sum, warps, most);
  for (int w = 4 * q0; w < 4 * q1; ++w) {
    before[w] = at;
    at += __popc(free[w]);
  }
  __syncthreads();
  if (wanted > most) bad |= kStatNoPageBit;
  for (int u = me.warp; u < units; u += me.kAllWarps) {
    const int i = u / spans, j0 = (u - i * spans) * span;
    int tail;
    const Child c = held.child(p, i, tail);
    const int plain = tail >= 0 ? c.have - 1 : c.have;  // entries that stay
    int32_t* to = p.out + (long long)i * p.table_pages;
    int e[LANES];
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = j < plain ? __ldg(c.row + j) : -1;
    }
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
      const int j = j0 + 32 * k + me.lane;
      if (j < p.table_pages && (j < plain || j >= c.need)) to[j] = e[k];
    }
    // (a loop, not unrolled with the others: few entries are new, and a warp fetches the code that it runs once)
#pragma unroll 1
    for (int j = max(plain, j0) + me.lane; j < min(c.need, j0 + span); j += 32) {
      const int rank = held.base[i] + j - plain;
      const int got = rank < most ? nth<true>(free, before, words, rank) : -1;
      if (j < c.have) {
        p.src[i] = got < 0 ? -1 : __ldg(c.row + j);
        p.dst[i] = got;
      }
      to[j] = got;
    }
    if (tail < 0 && j0 == 0 && me.lane == 0) p.src[i] = p.dst[i] = -1;
  }
  if (bad) report(p.status, bad);
  peers_have_read<ONE>();
}

template <int LANES, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) compact_bits_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ int warps[2][kWarps];
  const Team<ONE> me;
  const int words = p.words;
  uint32_t *own = bits, *held = bits + words, *moving = bits + 2 * words;
  int *held_before = reinterpret_cast<int*>(bits + 3 * words), *moving_before = held_before + words;
  unsigned bad = 0;
  grid_wait();
  grid_launch_dependents();
  for (int q = threadIdx.x; q < words / 4; q += kThreads) reinterpret_cast<uint4*>(own)[q] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  constexpr int span = 32 * LANES;
  const int spans = p.spans, units = p.sequences * spans;
  auto pages_held = [&](int s, bool tell) {
    bool len_bad = false;
    const int n = pages_of(p, held_len(p, __ldg(p.lens + s), len_bad));
    if (len_bad && tell) bad |= kStatRowLenBit;
    return n;
  };
  for (int u = me.warp; u < units; u += me.kAllWarps) {
    const int s = u / spans, j0 = (u - s * spans) * span;
    const int have = pages_held(s, j0 == 0);
    const int32_t* row = p.table + s * p.table_stride;
    int e[LANES];
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = j < have ? row[j] : -1;
      if (j < have && (unsigned)e[k] >= (unsigned)p.pages) bad |= kStatIndexBit;
    }
#pragma unroll
    for (int k = 0; k < LANES; ++k)
      if ((unsigned)e[k] < (unsigned)p.pages) set_bit(own, e[k]);
  }
  me.meet();
  const int each = (words / 4 + kThreads - 1) / kThreads, q0 = min(words / 4, (int)threadIdx.x * each), q1 = min(words / 4, q0 + each);
  for (int q = threadIdx.x; q < words / 4; q += kThreads) reinterpret_cast<uint4*>(held)[q] = all_bits<ONE>(own, q);
  peers_read<ONE>();
  __syncthreads();
  int n_held = 0, n_moving = 0, used, movable;
  for (int w = 4 * q0; w < 4 * q1; ++w) {
    const uint32_t x = held[w], pinned = kept(p, w);
    held[w] = x | pinned;
    moving[w] = x & ~pinned;
    n_held += __popc(x | pinned);
    n_moving += __popc(x & ~pinned);
  }
  int at_held = sum_before(n_held, warps[0], used), at_moving = sum_before(n_moving, warps[1], movable);
  for (int w = 4 * q0; w < 4 * q1; ++w) {
    held_before[w] = at_held;
    moving_before[w] = at_moving;
    at_held += __popc(held[w]);
    at_moving += __popc(moving[w]);
  }
  __syncthreads();
  // moving pages before page i
  auto before = [&](int i) { return moving_before[i >> 5] + __popc(moving[i >> 5] & ((1u << (i & 31)) - 1u)); };
  const int below = used < p.pages ? before(used) : movable, count = movable - below;
  if (me.thread == 0) {
    p.count[0] = count;
    p.count[1] = used;
  }
  for (int i = count + me.thread; i < p.pages / 2; i += me.kAllThreads) p.src[i] = p.dst[i] = -1;
  for (int i = used + me.thread; i < p.pages; i += me.kAllThreads) {
    if (!(moving[i >> 5] >> (i & 31) & 1u)) continue;
    const int rank = before(i) - below;
    p.src[rank] = i;
    p.dst[rank] = nth<false>(held, held_before, words, rank);
  }
  for (int u = me.warp; u < units; u += me.kAllWarps) {
    const int s = u / spans, j0 = (u - s * spans) * span;
    const int have = pages_held(s, false);
    const int32_t* row = p.table + s * p.table_stride;
    int32_t* out = p.out + (long long)s * p.table_pages;
    int e[LANES];
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
      const int j = j0 + 32 * k + me.lane;
      e[k] = j < have ? row[j] : -1;  // (out may be the table itself)
    }
#pragma unroll
    for (int k = 0; k < LANES; ++k)
      if (e[k] >= used && e[k] < p.pages && (moving[e[k] >> 5] >> (e[k] & 31) & 1u)) e[k] = nth<false>(held, held_before, words, before(e[k]) - below);
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
      const int j = j0 + 32 * k + me.lane;
      if (j < p.table_pages) out[j] = e[k];
    }
  }
  if (bad) report(p.status, bad);
  peers_have_read<ONE>();
}

// By the entries of a lane, 1 << i, and by whether a single thread block makes the tables: it has kOneRows pieces at most, of
// kForkPiece or kCompactPiece entries (one_block), one for each of its warps, and so never needs more entries a lane than these.
constexpr int kBitKernels = 5, kForkPiece = 128, kCompactPiece = 64;
static_assert(kOneRows <= kWarps, "a piece each warp");
using PlanKernel = void (*)(const PlanParams);
constexpr PlanKernel kForkBits[kBitKernels] = {fork_bits_kernel<1, false>, fork_bits_kernel<2, false>, fork_bits_kernel<4, false>, fork_bits_kernel<8, false>,
                                               fork_bits_kernel<16, false>};
constexpr PlanKernel kForkOne[] = {fork_bits_kernel<1, true>, fork_bits_kernel<2, true>, fork_bits_kernel<4, true>};
constexpr PlanKernel kCompactBits[kBitKernels] = {compact_bits_kernel<1, false>, compact_bits_kernel<2, false>, compact_bits_kernel<4, false>,
                                                  compact_bits_kernel<8, false>, compact_bits_kernel<16, false>};
constexpr PlanKernel kCompactOne[] = {compact_bits_kernel<1, true>, compact_bits_kernel<2, true>};
static_assert(32 << (std::size(kForkOne) - 1) == kForkPiece && 32 << (std::size(kCompactOne) - 1) == kCompactPiece, "a kernel for every cut");
// As many as give every warp one piece of the tables at most (64 rows of 1040: 9.7 us with 16 entries, 10.4 with 8, of which some
// warps have two pieces).
int cut(PlanParams& p, int rows, bool one) {
  const int warps = one ? Team<true>::kAllWarps : Cluster::kAllWarps;
  int i = 0;
  while (i < kBitKernels - 1 && p.table_pages > 32 << i && rows * (((long long)p.table_pages + (32 << i) - 1) / (32 << i)) > warps) ++i;
  p.lanes = 1 << i;
  p.spans = std::max(1, (int)(((long long)p.table_pages + (32 << i) - 1) / (32 << i)));
  return i;
}

template <typename K>
cudaError_t launch_plan(K kernel, const PlanParams& p, bool one, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(one ? 1 : kBlocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute a[2] = {};
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, one ? 0 : kBlocks);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ---------------------------------------------------------------------------
// Copies.
// ---------------------------------------------------------------------------
struct CopyParams {
  unsigned char* base[4];  // keys, values, scales, bounds
  long long page_b, token_b, head_b;
  int pages, tokens, heads, run;       // run: contiguous 16-byte pieces; of which a page has tokens * heads
  long long page_words[2];             // scales and bounds: words of 8 bytes of a page
  int chunks[4];                       // of a page, and of the plane
  int scale_pieces, all_pieces;        // flat: of a page's scales, and of all
  int all_chunks;
  const int32_t *src, *dst, *count;
  int n;
  unsigned* status;
};

constexpr int kCopyThreads = 256, kPer = 4, kChunk = kCopyThreads * kPer;  // pieces (words) of a chunk

// A thread block takes one chunk of one plane of one pair after the other. FLAT: a page's keys are one run, and its values, and its
// scales and bounds are whole 16-byte pieces: the pieces of all planes are one axis, and their places need no divisions.
template <bool FLAT>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  grid_wait();
  grid_launch_dependents();
  const int n = p.count ? min(p.n, max(0, __ldg(p.count))) : p.n;
  const long long items = (long long)n * p.all_chunks;
  int next_src = -1, next_dst = -1;  // of the next item: looked up while this one's pieces are on their way
  auto look_up = [&](long long w) {
    if (w >= items) return;
    const int i = (int)(w / p.all_chunks);
    next_src = __ldg(p.src + i);
    next_dst = __ldg(p.dst + i);
  };
  look_up(blockIdx.x);
  for (long long w = blockIdx.x; w < items; w += gridDim.x) {
    int chunk = (int)(w % p.all_chunks);
    const int src = next_src, dst = next_dst;
    look_up(w + gridDim.x);
    if (src < 0 || dst < 0) continue;
    if (src >= p.pages || dst >= p.pages) {
      if (threadIdx.x == 0) report(p.status, kStatIndexBit);
      continue;
    }
    if (FLAT) {
      uint4 x[kPer];
      uint4* to[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        int v = chunk * kChunk + k * kCopyThreads + threadIdx.x;
        to[k] = nullptr;
        if (v >= p.all_pieces) continue;
        unsigned char* base = p.base[0];
        long long page = p.page_b;
        if (v >= p.run) {
          v -= p.run;
          base = p.base[1];
          if (v >= p.run) {
            v -= p.run;
            base = p.base[2];
            page = p.page_words[0] * 8;
            if (v >= p.scale_pieces) {
              v -= p.scale_pieces;
              base = p.base[3];
              page = p.page_words[1] * 8;
            }
          }
        }
        x[k] = __ldg(reinterpret_cast<const uint4*>(base + src * page) + v);
        to[k] = reinterpret_cast<uint4*>(base + dst * page) + v;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (to[k]) *to[k] = x[k];
      continue;
    }
    int plane = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (plane == k && chunk >= p.chunks[k]) {
        chunk -= p.chunks[k];
        ++plane;
      }
    if (plane < 2) {
      unsigned char* base = plane ? p.base[1] : p.base[0];
      const int pieces = p.tokens * p.heads * p.run;
      uint4 x[kPer];
      long long at[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int v = chunk * kChunk + k * kCopyThreads + threadIdx.x;
        at[k] = -1;
        if (v < pieces) {
          const int row = v / p.run, token = row / p.heads;
          at[k] = token * p.token_b + (row - token * p.heads) * p.head_b + (v - row * p.run) * 16LL;
          x[k] = __ldg(reinterpret_cast<const uint4*>(base + src * p.page_b + at[k]));
        }
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (at[k] >= 0) *reinterpret_cast<uint4*>(base + dst * p.page_b + at[k]) = x[k];
    } else {
      uint2* base = reinterpret_cast<uint2*>(plane == 2 ? p.base[2] : p.base[3]);
      const long long words = plane == 2 ? p.page_words[0] : p.page_words[1];
      uint2 x[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const long long v = (long long)chunk * kChunk + k * kCopyThreads + threadIdx.x;
        if (v < words) x[k] = __ldg(base + src * words + v);
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const long long v = (long long)chunk * kChunk + k * kCopyThreads + threadIdx.x;
        if (v < words) base[dst * words + v] = x[k];
      }
    }
  }
}

bool overlap(const int32_t* a, long long na, const int32_t* b, long long nb) { return a < b + nb && b < a + na; }

int check_plan(const int32_t* page_table, int64_t table_stride, int32_t table_pages, int32_t sequences, const int32_t* lens, int32_t pages,
               int32_t page_size) {
  if (pages < 1 || page_size < 1 || (page_size & (page_size - 1)) || (int64_t)pages * page_size > INT32_MAX) return TKS_E_INVAL;
  if (sequences < 0 || table_pages < 0 || table_stride < 0 || table_stride > ((int64_t)1 << 56) / (sequences > 0 ? sequences : 1)) return TKS_E_INVAL;
  if (!aligned(page_table, 4) || !aligned(lens, 4)) return TKS_E_INVAL;
  if (sequences > 0 && (!lens || (table_pages > 0 && !page_table))) return TKS_E_INVAL;
  return TKS_OK;
}

// A single thread block needs no cluster's barrier, as long as its warps have one short piece of the tables each, and (compact) no
// more pages each than a few. Forks of 8 rows of 64 pages 3.9 us so and 5.1 otherwise, of 500 4.7 and 5.5, of 1000 6.1 and 6.1;
// compactions of 8 rows of 64 pages in a pool of 1024 4.2 and 5.0, of 500 6.8 and 5.5, of 64 in 4096 6.9 and 5.7.
bool one_block(bool fork, int32_t pages, int32_t rows, int32_t table_pages) {
  const long long piece = fork ? kForkPiece : kCompactPiece;
  return pages <= (fork ? kOnePages : kOnePages / 8) && rows * std::max(1LL, (table_pages + piece - 1) / piece) <= kOneRows;
}

PlanParams plan_params(const int32_t* page_table, int64_t table_stride, int32_t table_pages, int32_t sequences, const int32_t* lens,
                       const uint8_t* keep, int32_t pages, int32_t page_size, int32_t* table, int32_t* src, int32_t* dst, int32_t* scratch, int rows, bool few) {
  PlanParams p{};
  p.table = page_table;
  p.table_stride = table_stride;
  p.table_pages = table_pages;
  p.sequences = sequences;
  p.lens = lens;
  p.keep = keep;
  p.pages = pages;
  p.page_shift = log2_of(page_size);
  p.out = table;
  p.src = src;
  p.dst = dst;
  p.lanes = kLanes;
  while (few && p.lanes > 1 && (long long)rows * (((long long)table_pages + 32 * p.lanes - 1) / (32 * p.lanes)) < kAllWarps) p.lanes /= 2;
  p.spans = std::max(1, (int)(((long long)table_pages + 32 * p.lanes - 1) / (32 * p.lanes)));
  p.words = (pages + 127) / 128 * 4;
  p.sums = scratch;
  p.tallies = reinterpret_cast<Tally*>(scratch + 1024);
  p.owner = scratch + 1024 + (pages + 31) / 32 * 4;
  p.base = p.owner + pages;
  return p;
}
static_assert(2 * kAllWarps <= 1024 && sizeof(Tally) == 16, "the scratch buffer's layout");

}  // namespace

cudaError_t setup_pages() {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < kBitKernels && e == cudaSuccess; ++i) {
    e = allow(kForkBits[i], 4 * kBitPages / 8);
    if (e == cudaSuccess) e = allow(kCompactBits[i], 5 * kBitPages / 8);
  }
  return e;
}

}  // namespace attn
}  // namespace tks

using namespace tks;
using namespace tks::attn;

extern "C" int tks_cache_fork(const int32_t* page_table, int64_t table_stride, int32_t table_pages, int32_t sequences, const int32_t* lens,
                              const int32_t* parents, const int32_t* new_lens, int32_t children, const uint8_t* keep, int32_t pages,
                              int32_t page_size, int32_t* table, int32_t* src, int32_t* dst, int32_t* scratch, void* stream) {
  if (check_plan(page_table, table_stride, table_pages, sequences, lens, pages, page_size) != TKS_OK || children < 0) return TKS_E_INVAL;
  if ((int64_t)children * table_pages + children > INT32_MAX - (1 << 16)) return TKS_E_TOO_LARGE;
  if (children == 0) return TKS_OK;
  if (!parents || !new_lens || !src || !dst || !scratch || (table_pages > 0 && !table)) return TKS_E_INVAL;
  if (!aligned(parents, 4) || !aligned(new_lens, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(scratch, 16) || !aligned(table, 4))
    return TKS_E_INVAL;
  const long long held = sequences > 0 ? (sequences - 1) * table_stride + table_pages : 0;
  if (table_pages > 0 && overlap(page_table, held, table, (long long)children * table_pages)) return TKS_E_INVAL;
  Place place;
  const int rc = place_of(stream, &place);
  if (rc != TKS_OK) return rc;
  const bool one = one_block(true, pages, children, table_pages);
  PlanParams p = plan_params(page_table, table_stride, table_pages, sequences, lens, keep, pages, page_size, table, src, dst, scratch, children, false);
  p.parents = parents;
  p.new_lens = new_lens;
  p.children = children;
  p.status = place.status;
  std::lock_guard<std::mutex> lock(*place.order);
  const bool bits = pages <= kBitPages && children <= kHeldChildren;
  const PlanKernel kernel = one ? kForkOne[cut(p, children, one)] : bits ? kForkBits[cut(p, children, one)] : fork_kernel;
  if (launch_plan(kernel, p, one, bits ? 4 * p.words * 4 : 0, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}

extern "C" int tks_cache_compact(const int32_t* page_table, int64_t table_stride, int32_t table_pages, int32_t sequences, const int32_t* lens,
                                 const uint8_t* keep, int32_t pages, int32_t page_size, int32_t* table, int32_t* src, int32_t* dst,
                                 int32_t* count, int32_t* scratch, void* stream) {
  if (check_plan(page_table, table_stride, table_pages, sequences, lens, pages, page_size) != TKS_OK) return TKS_E_INVAL;
  if ((int64_t)sequences * table_pages + sequences > INT32_MAX - (1 << 16)) return TKS_E_TOO_LARGE;
  if (!count || !scratch || (pages > 1 && (!src || !dst)) || (sequences > 0 && table_pages > 0 && !table)) return TKS_E_INVAL;
  if (!aligned(count, 4) || !aligned(scratch, 16) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(table, 4)) return TKS_E_INVAL;
  const long long held = sequences > 0 ? (sequences - 1) * table_stride + table_pages : 0;
  const bool in_place = table == page_table && (sequences <= 1 || table_stride == table_pages);
  if (held > 0 && table_pages > 0 && !in_place && overlap(page_table, held, table, (long long)sequences * table_pages)) return TKS_E_INVAL;
  Place place;
  const int rc = place_of(stream, &place);
  if (rc != TKS_OK) return rc;
  const bool one = one_block(false, pages, sequences, table_pages);
  PlanParams p = plan_params(page_table, table_stride, table_pages, sequences, lens, keep, pages, page_size, table, src, dst, scratch, sequences, true);
  p.count = count;
  p.status = place.status;
  std::lock_guard<std::mutex> lock(*place.order);
  const bool bits = pages <= kBitPages;
  const PlanKernel kernel = one ? kCompactOne[cut(p, sequences, one)] : bits ? kCompactBits[cut(p, sequences, one)] : compact_kernel;
  if (launch_plan(kernel, p, one, bits ? 5 * p.words * 4 : 0, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}

extern "C" int tks_cache_copy(const tks_cache* cache, const tks_bounds* bounds, const int32_t* src, const int32_t* dst, int32_t n,
                              const int32_t* count, void* stream) {
  if (check_cache(cache) != TKS_OK || n < 0) return TKS_E_INVAL;
  if (bounds && (check_bounds(bounds) != TKS_OK || !bounds_of(bounds, cache))) return TKS_E_INVAL;
  if (n == 0) return TKS_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4)) return TKS_E_INVAL;
  CopyParams p{};
  const long long size = cache->held == TKS_I8 ? 1 : 2, row = cache->head_dim * size;
  p.base[0] = static_cast<unsigned char*>(cache->k);
  p.base[1] = static_cast<unsigned char*>(cache->v);
  p.base[2] = reinterpret_cast<unsigned char*>(cache->scales);
  p.base[3] = bounds ? static_cast<unsigned char*>(bounds->bounds) : nullptr;
  p.page_b = cache->page_stride * size;
  p.token_b = cache->token_stride * size;
  p.head_b = cache->head_stride * size;
  p.pages = cache->pages;
  const __int128 pieces = (__int128)cache->page_size * cache->kv_heads * (row / 16);
  if (pieces > INT32_MAX / 2) return TKS_E_TOO_LARGE;
  p.tokens = cache->page_size;
  p.heads = cache->kv_heads;
  p.run = (int)(row / 16);
  // rows that follow each other without a gap are one
  if ((p.heads == 1 || p.head_b == row) && (p.tokens == 1 || p.token_b == row * p.heads)) {
    p.run = (int)pieces;
    p.tokens = p.heads = 1;
  }
  p.page_words[0] = cache->held == TKS_I8 ? (long long)cache->page_size * cache->kv_heads : 0;
  p.page_words[1] = bounds ? (long long)(bounds->page_size / bounds->block) * bounds->kv_heads * bounds->head_dim / 2 : 0;
  p.chunks[0] = p.chunks[1] = (int)((pieces + kChunk - 1) / kChunk);
  for (int i = 0; i < 2; ++i) p.chunks[2 + i] = (int)((p.page_words[i] + kChunk - 1) / kChunk);
  long long all = 2LL * p.chunks[0] + p.chunks[2] + p.chunks[3];
  const long long all_pieces = 2 * (long long)pieces + (p.page_words[0] + p.page_words[1]) / 2;
  const bool flat = p.tokens == 1 && p.heads == 1 && p.page_words[0] % 2 == 0 && aligned(p.base[2], 16) && all_pieces < INT32_MAX - kChunk;
  if (flat) {
    p.scale_pieces = (int)(p.page_words[0] / 2);
    p.all_pieces = (int)all_pieces;
    all = (all_pieces + kChunk - 1) / kChunk;
  }
  p.all_chunks = (int)all;
  p.src = src;
  p.dst = dst;
  p.count = count;
  p.n = n;
  Place place;
  const int rc = place_of(stream, &place);
  if (rc != TKS_OK) return rc;
  p.status = place.status;
  std::lock_guard<std::mutex> lock(*place.order);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(n * all, place.sms * 4LL));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute a[1] = {};
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, 0);
  if ((flat ? cudaLaunchKernelEx(&cfg, copy_kernel<true>, p) : cudaLaunchKernelEx(&cfg, copy_kernel<false>, p)) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}
