// Page tables of a step's new sequences, moving pages in use together, and
// copying pages.
//
// The two calls that make tables are a few passes over the tables and over one
// word for each page, with nothing between them but that all of one is done
// before the next begins: one thread-block cluster makes them, in one launch,
// its barrier between the passes. A pass is as long as the loads in it that wait
// for each other, so there are few: who holds which page; how many pages of each
// kind lie before each 32 (and their bits); and the tables, for which the r-th free
// page, or the number of moving pages before one, is looked up in those. What
// the passes leave for each other lies in the caller's scratch buffer, so that
// nothing is shared between calls. Small tables are made by a single thread block,
// which keeps it in shared memory.
//
// What bounds it: latency, of launch, barriers and loads that wait for each other; and,
// where rows are long, the scattered stores of who holds a page. Measured: 64 beams
// of 16 prompts over up to 65,536 positions in pages of 64: 12.4 us (launch 0.9, children
// looked up 0.8, marks 4, counts 2.8, tables 4); a pool of 8192 pages compacted 11.7 us; a
// few short beams 4.2 us (7.4 by a cluster), a pool of 639 pages compacted 5.5 (9.2).
// Copies: 2048 pages of 135 KB 92 us, 6.0 TB/s; more under way (five or six thread blocks
// an SM instead of four) 95.

#include <algorithm>

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
  // scratch: what the warps have counted, 32 pages' tallies, a word a page, a word a child
  int32_t* sums;
  Tally* tallies;
  int32_t *owner, *base;
  unsigned* status;
};

// Who makes the tables: a cluster, whose barrier also orders its accesses to global memory, or (ONE) a single thread block, which
// keeps what the passes leave for each other in shared memory.
constexpr int kOnePages = 4096, kOneRows = 32;  // at most
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
template <bool ONE>
struct Store {
  int32_t *owner, *dst;
  Tally* tallies;
  __device__ __forceinline__ Store(const PlanParams& p) : owner(p.owner), dst(p.dst), tallies(p.tallies) {}
  template <typename T>
  __device__ __forceinline__ T read(const T* at) const { return __ldcg(at); }
};
template <>
struct Store<true> {
  int32_t *owner, *dst;
  Tally* tallies;
  __device__ __forceinline__ Store(const PlanParams& p) {
    __shared__ int32_t words[kOnePages + kOnePages / 2];
    __shared__ Tally each32[kOnePages / 32];
    owner = words;
    dst = words + kOnePages;
    tallies = each32;
  }
  template <typename T>
  __device__ __forceinline__ T read(const T* at) const { return *at; }
};

// Of two numbers that each warp has counted: the sums over the warps before each one, in shared memory.
template <bool ONE>
struct Sums {
  static constexpr int kAllWarps = Team<ONE>::kAllWarps;
  int a[kAllWarps + 1], b[kAllWarps + 1], warps[2][kAllWarps / 32];
};
template <bool ONE>
__device__ __forceinline__ void sum_up(const Team<ONE>& me, const PlanParams& p, Sums<ONE>& s, int a, int b) {
  constexpr int kAllWarps = Team<ONE>::kAllWarps;
  if (me.lane == 0) {
    if (ONE) {
      s.a[me.warp + 1] = a;
      s.b[me.warp + 1] = b;
    } else {
      p.sums[me.warp] = a;
      p.sums[kAllWarps + me.warp] = b;
    }
  }
  me.meet();
  const int t = threadIdx.x, w = t >> 5;
  int x = 0, y = 0;
  if (t < kAllWarps) {
    x = ONE ? s.a[t + 1] : __ldcg(p.sums + t);
    y = ONE ? s.b[t + 1] : __ldcg(p.sums + kAllWarps + t);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (me.lane >= o) {
        x += u;
        y += v;
      }
    }
    if (!ONE && me.lane == 31) {
      s.warps[0][w] = x;
      s.warps[1][w] = y;
    }
  }
  if (!ONE) __syncthreads();
  if (t < kAllWarps) {
    if (!ONE)
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
template <bool ONE>
__device__ __forceinline__ int share(int n) {
  constexpr int kAllWarps = Team<ONE>::kAllWarps;
  return (int)((((long long)n + kAllWarps - 1) / kAllWarps + 31) / 32 * 32);
}
template <bool ONE>
__device__ __forceinline__ void share(const Team<ONE>& me, int n, int& begin, int& end) {
  const long long each = share<ONE>(n);
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
template <bool FORK, bool ONE>
__device__ __forceinline__ int free_page(const PlanParams& p, const Sums<ONE>& s, const Store<ONE>& store, int rank) {
  const int each = share<ONE>(p.pages);
  int run = 0;
#pragma unroll
  for (int step = Team<ONE>::kAllWarps / 2; step; step >>= 1)
    if ((FORK ? s.a[run + step] : (int)min((long long)p.pages, (long long)each * (run + step)) - s.a[run + step]) <= rank) run += step;
  rank -= FORK ? s.a[run] : (int)min((long long)p.pages, (long long)each * run) - s.a[run];
  const int first = run * (each / 32);
  int low = 0, high = min(each / 32, (p.pages + 31) / 32 - first);
  while (high - low > 1) {  // (the last 32 with no more before them than the rank)
    const int mid = (low + high) / 2, before = store.read(&store.tallies[first + mid].before_a);
    if ((FORK ? before : 32 * mid - before) <= rank) low = mid;
    else high = mid;
  }
  const uint4 t = store.read(reinterpret_cast<const uint4*>(store.tallies + first + low));
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
// Children that each thread block keeps in shared memory, looked up once (each look goes through three loads that wait for
// each other: parent, length, entry).
constexpr int kHeldChildren = 2048;

// HELD: all children fit there.
template <bool HELD, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const __grid_constant__ PlanParams p) {
  static_assert(HELD || !ONE, "a single thread block holds all children");
  constexpr int kHeld = ONE ? kOneRows : kHeldChildren, kMine = (kHeld + kThreads - 1) / kThreads, kAllWarps = Team<ONE>::kAllWarps;
  __shared__ struct {
    int parent[kHeld], have[kHeld], need[kHeld], tail[kHeld], base[kHeld];
    int warps[kWarps];
  } held;  // (tail: the entry that is going to be written to, or -1; later, the one that is copied)
  __shared__ Sums<ONE> sums;
  const Team<ONE> me;
  const Store<ONE> store(p);
  unsigned bad = 0;
  grid_wait();
  grid_launch_dependents();
  // the entry that child c writes to, or -1
  auto tail_of = [&](const Child& c) -> int {
    const int e = c.writes ? __ldg(c.row + c.have - 1) : -1;
    return (unsigned)e < (unsigned)p.pages ? e : -1;
  };
  // who holds a page: nobody yet
  for (int i = me.thread; i < p.pages; i += me.kAllThreads) store.owner[i] = p.keep && p.keep[i] ? kShared : kFree;
  if (HELD)
    for (int i = threadIdx.x; i < p.children; i += kThreads) {
      const Child c = child_of(p, i, me.rank == 0 ? &bad : nullptr);
      held.parent[i] = c.have > 0 ? __ldg(p.parents + i) : 0;
      held.have[i] = c.have;
      held.need[i] = c.need;
      held.tail[i] = tail_of(c);
    }
  auto child = [&](int i, int& tail, unsigned* bad) -> Child {
    if (!HELD) {
      const Child c = child_of(p, i, bad);
      tail = tail_of(c);
      return c;
    }
    tail = held.tail[i];
    return Child{p.table + held.parent[i] * p.table_stride, held.have[i], held.need[i], tail >= 0};
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
    if (HELD && i > 0) {
      // What the child before has in the same place, it marks: those that continue one prompt have its pages in common, and
      // scattered stores, of a few SMs only, are what this pass is bound by (16 groups of 4 beams over up to 65,536
      // positions: 14.0 us in all without, 12.4 so).
      int other;
      const Child o = child(i - 1, other, nullptr);
      const int same = o.have - (other >= 0 ? 1 : 0);
#pragma unroll
      for (int k = 0; k < kLanes; ++k) {
        const int j = j0 + 32 * k + me.lane;
        if (j < min(same, c.have) && __ldg(o.row + j) == e[k] && !(tail >= 0 && j == c.have - 1)) e[k] = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      if ((unsigned)e[k] >= (unsigned)p.pages) continue;
      // (a held page's word only ever falls: to kShared, or to the lowest of those who write to it)
      if (tail >= 0 && j0 + 32 * k + me.lane == c.have - 1) atomicMin(store.owner + e[k], i);
      else store.owner[e[k]] = kShared;
    }
  }
  me.meet();
  // how many pages each child wants, and how many are free
  auto wants = [&](int i, bool& copied) -> int {
    int tail;
    const Child c = child(i, tail, nullptr);
    copied = tail >= 0 && store.read(store.owner + tail) != i;
    return c.need - c.have + (copied ? 1 : 0);
  };
  int page0, page1, child0 = 0, child1 = 0;
  share(me, p.pages, page0, page1);
  int free = 0, wanted = 0;
#pragma unroll 4
  for (int i = page0; i < page1; i += 32) {
    const uint32_t m = __ballot_sync(0xffffffffu, i + me.lane < page1 && store.read(store.owner + i + me.lane) == kFree);
    if (me.lane == 0) store.tallies[i / 32] = Tally{m, 0, free, 0};
    free += __popc(m);
  }
  bool copied;
  if (HELD) {
    // every thread block for itself: the children's wishes before each child
    int n[kMine], sum = 0;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = threadIdx.x * kMine + k;
      n[k] = 0;
      if (i < p.children) {
        n[k] = wants(i, copied);
        if (!copied) held.tail[i] = -1;
      }
      sum += n[k];
    }
    int end = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (me.lane >= o) end += y;
    }
    if (me.lane == 31) held.warps[threadIdx.x >> 5] = end;
    __syncthreads();
    const int w = held.warps[me.lane], before = __reduce_add_sync(0xffffffffu, me.lane < (int)(threadIdx.x >> 5) ? w : 0);
    wanted = __reduce_add_sync(0xffffffffu, w);
    int at = before + end - sum;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = threadIdx.x * kMine + k;
      if (i < p.children) held.base[i] = at;
      at += n[k];
    }
    sum_up(me, p, sums, free, 0);
  } else {
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
  }
  const int most = sums.a[kAllWarps];  // pages to hand out
  if (wanted > most) bad |= kStatNoPageBit;
  for (int u = me.warp; u < units; u += kAllWarps) {
    const int i = u / spans, j0 = (u - i * spans) * span;
    int tail;
    const Child c = child(i, tail, nullptr);
    const int base = HELD ? held.base[i] : __ldcg(p.base + i);
    const bool copy = HELD ? tail >= 0 : tail >= 0 && store.read(store.owner + tail) != i;
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
        const int got = rank < most ? free_page<true>(p, sums, store, rank) : -1;
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

template <bool ONE>
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const __grid_constant__ PlanParams p) {
  __shared__ Sums<ONE> sums;
  const Team<ONE> me;
  const Store<ONE> store(p);
  unsigned bad = 0;
  grid_wait();
  grid_launch_dependents();
  constexpr int kAllWarps = Team<ONE>::kAllWarps;
  auto pinned = [&](int i) { return p.keep && p.keep[i] != 0; };
  for (int i = me.thread; i < p.pages; i += me.kAllThreads) store.owner[i] = pinned(i) ? kShared : kFree;
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
      if ((unsigned)e[k] < (unsigned)p.pages) store.owner[e[k]] = kShared;
  }
  me.meet();
  int page0, page1, held = 0, movable = 0;
  share(me, p.pages, page0, page1);
#pragma unroll 4
  for (int i0 = page0; i0 < page1; i0 += 32) {
    const int i = i0 + me.lane;
    const bool is = i < page1 && store.read(store.owner + i) != kFree;
    const uint32_t a = __ballot_sync(0xffffffffu, is), b = __ballot_sync(0xffffffffu, is && !pinned(i));
    if (me.lane == 0) store.tallies[i0 / 32] = Tally{a, b, held, movable};
    held += __popc(a);
    movable += __popc(b);
  }
  sum_up(me, p, sums, held, movable);
  const int used = sums.a[kAllWarps], each = share<ONE>(p.pages);
  // movable pages before page i
  auto before = [&](int i, const uint4& t) { return sums.b[i / each] + (int)t.w + __popc(t.y & ((1u << (i & 31)) - 1u)); };
  auto tally = [&](int i) { return store.read(reinterpret_cast<const uint4*>(store.tallies + i / 32)); };
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
    const int to = free_page<false>(p, sums, store, rank);
    p.dst[rank] = to;
    if (ONE) store.dst[rank] = to;
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
      if (to[k] >= 0) e[k] = store.read(store.dst + to[k]);
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
      const int j = j0 + 32 * k + me.lane;
      if (k < lanes && j < p.table_pages) out[j] = e[k];
    }
  }
  if (bad) report(p.status, bad);
}

template <typename K>
cudaError_t launch_plan(K kernel, const PlanParams& p, bool one, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(one ? 1 : kBlocks);
  cfg.blockDim = dim3(kThreads);
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
  int planes;              // (2 for keys and values without scales and bounds)
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

// A single thread block's passes are shorter, as long as no warp has more than one piece of the tables (16 rows of 256 pages, of
// 4096: forked in 4.9 us so and in 9.5 by a cluster, compacted in 5.8 and 8.9; 64 of 64: 7.6 and 9.0, 8.2 and 9.0; 256 of 16:
// 18.5 and 8.4, 22.5 and 8.8).
bool one_block(int32_t pages, int32_t rows, int32_t table_pages) {
  return pages <= kOnePages && rows * std::max(1LL, (table_pages + 32LL * kLanes - 1) / (32 * kLanes)) <= kOneRows;
}

PlanParams plan_params(const int32_t* page_table, int64_t table_stride, int32_t table_pages, int32_t sequences, const int32_t* lens,
                       const uint8_t* keep, int32_t pages, int32_t page_size, int32_t* table, int32_t* src, int32_t* dst, int32_t* scratch, int rows, bool few, bool one) {
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
  while (few && p.lanes > 1 && (long long)rows * (((long long)table_pages + 32 * p.lanes - 1) / (32 * p.lanes)) < (one ? Team<true>::kAllWarps : Team<false>::kAllWarps)) p.lanes /= 2;
  p.spans = std::max(1, (int)(((long long)table_pages + 32 * p.lanes - 1) / (32 * p.lanes)));
  p.sums = scratch;
  p.tallies = reinterpret_cast<Tally*>(scratch + 1024);
  p.owner = scratch + 1024 + (pages + 31) / 32 * 4;
  p.base = p.owner + pages;
  return p;
}
static_assert(2 * Team<false>::kAllWarps <= 1024 && sizeof(Tally) == 16, "the scratch buffer's layout");

}  // namespace
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
  const bool one = one_block(pages, children, table_pages);
  PlanParams p = plan_params(page_table, table_stride, table_pages, sequences, lens, keep, pages, page_size, table, src, dst, scratch, children, false, one);
  p.parents = parents;
  p.new_lens = new_lens;
  p.children = children;
  p.status = place.status;
  std::lock_guard<std::mutex> lock(*place.order);
  const bool fit = children <= kHeldChildren;
  const auto kernel = one ? fork_kernel<true, true> : fit ? fork_kernel<true, false> : fork_kernel<false, false>;
  if (launch_plan(kernel, p, one, (cudaStream_t)stream) != cudaSuccess) {
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
  const bool one = one_block(pages, sequences, table_pages);
  PlanParams p = plan_params(page_table, table_stride, table_pages, sequences, lens, keep, pages, page_size, table, src, dst, scratch, sequences, true, one);
  p.count = count;
  p.status = place.status;
  std::lock_guard<std::mutex> lock(*place.order);
  if (launch_plan(one ? compact_kernel<true> : compact_kernel<false>, p, one, (cudaStream_t)stream) != cudaSuccess) {
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
