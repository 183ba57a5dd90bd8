// Host side of the cache and attention calls (include/tks_attention.h), and
// the kernel that joins partial results.

#include <algorithm>
#include <atomic>
#include <cmath>
#include <exception>
#include <map>
#include <memory>
#include <mutex>
#include <tuple>

#include "tks_attention.h"
#include "tks_attn.cuh"

namespace tks {
namespace attn {
namespace {

// ---------------------------------------------------------------------------
// Joining the partial results of units that were split over blocks.
// A unit's partials are few (most units are whole, and return at once) or, for
// a lone long sequence, many; in the first case a warp takes a row (PER_BLOCK =
// 8), in the second the block's warps share one row's partials.
// ---------------------------------------------------------------------------
template <int ROWS, int D, int TK, bool SEL, int PER_BLOCK>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ Params p) {
  constexpr int kVec = D / 32;
  __shared__ struct {
    int c0, c1, slot0;
  } span;
  __shared__ float acc_s[8][D];
  __shared__ float2 ml_s[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = p.kv_heads * p.row_tiles;
  const int seq = blockIdx.x / per, in = blockIdx.x % per;
  const int head = in / p.row_tiles, row_tile = in % p.row_tiles;
  const int first = row_tile * ROWS + blockIdx.y * PER_BLOCK;
  grid_wait();
  grid_launch_dependents();
  if (first >= p.rows) return;
  const Split sp = SEL ? p.split : *p.plan;
  const int tiles = tiles_of<TK>(seq_of<SEL>(p, seq).len);
  if (sp.share) {
    if (threadIdx.x == 0) {
      span.c0 = blockIdx.x * sp.share;
      span.c1 = span.c0 + (int)min(sp.share, (unsigned)tiles) - 1;
      span.slot0 = 0;
    }
  } else if (warp == 0) {
    long long before = 0;  // tiles of a unit of each sequence before this one
    if (!SEL) {
      for (int s = lane; s < seq; s += 32) before += tiles_of<TK>(seq_of<SEL>(p, s).len);
#pragma unroll
      for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (lane == 0) {
      const long long w0 = (SEL ? (long long)tiles * seq : before) * per + (long long)in * tiles;
      span.c0 = sp.block_of(w0);
      span.c1 = sp.block_of(w0 + tiles - 1);  // (those between have tiles, too)
      span.slot0 = sp.start(span.c0) != w0 ? 1 : 0;
    }
  }
  __syncthreads();
  const int c0 = span.c0, c1 = span.c1, slot0 = span.slot0;
  if (c0 == c1) return;  // whole: its block has written the output

  const int r = first - row_tile * ROWS + (PER_BLOCK == 8 ? warp : 0);  // row in its tile
  const int R = row_tile * ROWS + r;
  const bool live = r < ROWS && R < p.rows;
  if (PER_BLOCK == 8) {
    if (!live) return;
    float m, l, acc[kVec];
    join_row<ROWS, D>(p.parts, c0, c1, slot0, r, 0, 1, acc, m, l);
    store_joined<D>(p, out_row<SEL>(p, seq, head, R), acc, m, l);
    return;
  }
  // (one row a block, and it is live)
  float m, l, acc[kVec];
  join_row<ROWS, D>(p.parts, c0, c1, slot0, r, warp, 8, acc, m, l);
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc_s[warp][lane * kVec + i] = acc[i];
  if (lane == 0) ml_s[warp] = make_float2(m, l);
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = fmaxf(top, ml_s[k].x);
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 q = ml_s[k];
    if (q.y == 0.f) continue;
    const float f = q.x == top ? 1.f : ex2(q.x - top);
    l += f * q.y;
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] += f * acc_s[k][lane * kVec + i];
  }
  store_joined<D>(p, out_row<SEL>(p, seq, head, R), acc, top, l);
}

template <int ROWS, int D, int TK, bool SEL, int PER_BLOCK>
cudaError_t combine(const Params& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int rows = p.rows < ROWS ? p.rows : ROWS;
  cfg.gridDim = dim3((unsigned)(p.seqs * p.kv_heads * p.row_tiles), (unsigned)((rows + PER_BLOCK - 1) / PER_BLOCK));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute a[1] = {};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<ROWS, D, TK, SEL, PER_BLOCK>, p);
}

template <int ROWS, int TK>
cudaError_t launch_combine(const Params& p, int head_dim, bool selected, int blocks, cudaStream_t s) {
  // Many partials for a unit, or few: one token over 1M positions of 4 heads (76 partials a unit) takes
  // 194 us with a block for each row and 207 with a warp; four of 64 heads over 2048 selected ones
  // (16) 12.4 and 15.2; 8 ragged sequences of 8 heads (2 or 3) 203 and 195.
  const bool many = (long long)p.seqs * p.kv_heads * p.row_tiles * 8 < blocks;
  if (head_dim == 64) {
    if (selected) return many ? combine<ROWS, 64, TK, true, 1>(p, s) : combine<ROWS, 64, TK, true, 8>(p, s);
    return many ? combine<ROWS, 64, TK, false, 1>(p, s) : combine<ROWS, 64, TK, false, 8>(p, s);
  }
  if (selected) return many ? combine<ROWS, 128, TK, true, 1>(p, s) : combine<ROWS, 128, TK, true, 8>(p, s);
  return many ? combine<ROWS, 128, TK, false, 1>(p, s) : combine<ROWS, 128, TK, false, 8>(p, s);
}

// ---------------------------------------------------------------------------
// Devices and workspaces
// ---------------------------------------------------------------------------
struct Device {
  int sms = 0;
  bool ok = false;
};
struct Workspace {
  unsigned char* ptr = nullptr;  // status word, the last call's split, then (at 256 bytes) partial slots
  // A call's two kernels follow each other on the stream, without another thread's call or a status
  // call's clear between them.
  std::shared_ptr<std::mutex> order;
};

constexpr size_t kPlanOffset = 64, kHeaderBytes = 256;

std::mutex g_mu;
std::map<int, Device> g_dev;

// Device, stream, and, where the handle stands for another stream in every host thread, the thread (by
// a number of its own: the system's are used again).
using Key = std::tuple<int, void*, unsigned long long>;
Key key_of(int dev, void* stream) {
  static std::atomic<unsigned long long> threads{0};
  thread_local unsigned long long mine = 0;
  if (stream != (void*)cudaStreamPerThread) return Key(dev, stream, 0);
  if (mine == 0) mine = ++threads;
  return Key(dev, stream, mine);
}
std::map<Key, Workspace> g_ws;

size_t part_bytes(const Device& d) {
  const size_t few = (size_t)d.sms * kRowsBlocksPerSm * 2 * kPartFloats<kRowsTile, 128>;
  const size_t many = (size_t)d.sms * 2 * kPartFloats<kTilesRows, 128>;
  return (few > many ? few : many) * sizeof(float);
}

// The current device and its workspace for `stream`, allocated on first use.
int prepare(void* stream, Device* dev, Workspace* ws) try {
  int id = 0;
  if (cudaGetDevice(&id) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_UNSUPPORTED;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  auto di = g_dev.find(id);
  if (di == g_dev.end()) {
    Device d;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, id) == cudaSuccess &&
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, id) == cudaSuccess &&
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, id) == cudaSuccess)
      d.ok = major == 10 && minor == 3 && setup_rows() == cudaSuccess && setup_tiles() == cudaSuccess;
    cudaGetLastError();
    di = g_dev.emplace(id, d).first;
  }
  if (!di->second.ok) return TKS_E_UNSUPPORTED;
  *dev = di->second;
  const Key key = key_of(id, stream);
  auto wi = g_ws.find(key);
  if (wi == g_ws.end()) {
    Workspace w;
    w.order = std::make_shared<std::mutex>();
    if (cudaMalloc(&w.ptr, kHeaderBytes + part_bytes(*dev)) != cudaSuccess) {
      cudaGetLastError();
      return TKS_E_CUDA;
    }
    if (cudaMemsetAsync(w.ptr, 0, kHeaderBytes, (cudaStream_t)stream) != cudaSuccess) {
      cudaGetLastError();
      cudaFree(w.ptr);
      return TKS_E_CUDA;
    }
    wi = g_ws.emplace(key, w).first;
  }
  *ws = wi->second;
  return TKS_OK;
} catch (const std::exception&) {  // (host memory ran out: no C++ exception leaves a C entry point)
  return TKS_E_CUDA;
}

// ---------------------------------------------------------------------------
// Argument checks (nothing is touched on the device)
// ---------------------------------------------------------------------------
bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// Strides in elements of `size` bytes (with the extents they step over): none is
// negative, all are whole 16-byte pieces, and every offset in bytes fits 60 bits.
bool strides_ok(int64_t size, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 0, int64_t s2 = 0) {
  const int64_t unit = 16 / size;
  if (s0 < 0 || s1 < 0 || s2 < 0 || s0 % unit || s1 % unit || s2 % unit) return false;
  const __int128 span = (__int128)n0 * s0 + (__int128)n1 * s1 + (__int128)n2 * s2;
  return span * size < ((__int128)1 << 60);
}

int check_cache(const tks_cache* c) {
  if (c == nullptr) return TKS_E_INVAL;
  if (c->held != TKS_BF16 && c->held != TKS_I8) return TKS_E_INVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return TKS_E_INVAL;
  if (c->kv_heads < 1 || c->pages < 1 || c->page_size < 1 || (c->page_size & (c->page_size - 1)))
    return TKS_E_INVAL;
  if ((int64_t)c->pages * c->page_size > INT32_MAX) return TKS_E_INVAL;
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return TKS_E_INVAL;
  const int64_t size = c->held == TKS_I8 ? 1 : 2;
  if (!strides_ok(size, c->pages, c->page_stride, c->page_size, c->token_stride, c->kv_heads, c->head_stride))
    return TKS_E_INVAL;
  if (c->held == TKS_I8 && (!c->scales || !aligned(c->scales, 8))) return TKS_E_INVAL;
  return TKS_OK;
}

int log2_of(int32_t n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

// What scores are scaled with, as powers of two.
float scale_log2(const tks_queries* q) { return (float)((double)q->softmax_scale * 1.4426950408889634); }

int check_queries(const tks_cache* c, const tks_queries* q) {
  if (q == nullptr) return TKS_E_INVAL;
  if (q->batch < 0 || q->tokens < 0 || q->q_heads < 1 || q->q_heads % c->kv_heads) return TKS_E_INVAL;
  if (!std::isfinite(scale_log2(q))) return TKS_E_INVAL;
  if (q->table_pages < 0 || q->table_stride < 0) return TKS_E_INVAL;
  if (q->batch == 0 || q->tokens == 0) return TKS_OK;
  if ((int64_t)q->batch * q->tokens > INT32_MAX / q->q_heads) return TKS_E_INVAL;
  if (!q->q || !q->out || !aligned(q->q, 16) || !aligned(q->out, 16) || !aligned(q->lse, 4)) return TKS_E_INVAL;
  if (!strides_ok(2, q->batch, q->q_batch_stride, q->tokens, q->q_token_stride, q->q_heads, q->q_head_stride))
    return TKS_E_INVAL;
  if (q->table_stride > ((int64_t)1 << 56) / (q->batch > 0 ? q->batch : 1)) return TKS_E_INVAL;
  if (q->table_pages > 0 && (!q->page_table || !aligned(q->page_table, 4))) return TKS_E_INVAL;
  return TKS_OK;
}

Params params_of(const tks_cache* c, const tks_queries* q) {
  Params p{};
  const long long size = c->held == TKS_I8 ? 1 : 2;
  p.k = static_cast<const unsigned char*>(c->k);
  p.v = static_cast<const unsigned char*>(c->v);
  p.scales = reinterpret_cast<const float2*>(c->scales);
  p.page_b = c->page_stride * size;
  p.token_b = c->token_stride * size;
  p.head_b = c->head_stride * size;
  p.pages = c->pages;
  p.page_shift = log2_of(c->page_size);
  p.kv_heads = c->kv_heads;
  p.q = static_cast<const __nv_bfloat16*>(q->q);
  p.q_batch = q->q_batch_stride;
  p.q_token = q->q_token_stride;
  p.q_head = q->q_head_stride;
  p.out = static_cast<__nv_bfloat16*>(q->out);
  p.lse = q->lse;
  p.batch = q->batch;
  p.tokens = q->tokens;
  p.q_heads = q->q_heads;
  p.group = q->q_heads / c->kv_heads;
  p.table = q->page_table;
  p.table_stride = q->table_stride;
  p.table_pages = q->table_pages;
  p.scale_log2 = scale_log2(q);
  return p;
}

// The cluster size that a unit of at most `tiles` tiles is split over, or 0. Clusters pay where the
// device holds all units at once and shares are short: up to 1024 keys where the blocks fill more
// than half of the device (4 sequences of 7000 positions, 8 heads: 19.3 us, 21.5 with a second
// kernel), up to 640 where more blocks would help (one sequence of 7000: 14.4 us in a cluster of 8,
// 13.1 over 304 blocks; of 2048: 9.3 and 12.1). Selected positions of many rows keep the second
// kernel: one query of 64 heads over 256 takes 11.6 us with a cluster and 9.5 without.
int cluster_of(long long units, int64_t tiles, int tile_keys, int blocks) {
  int n = 1;
  while (n < kClusterMax && 2 * n * units <= blocks && n < tiles) n *= 2;
  const int64_t keys = 2 * n * units > blocks ? 1024 : 640;
  return units <= blocks && tiles <= n * (keys / tile_keys) ? n : 0;
}

// Queues the attention kernel and the one that joins its partials. (A unit's last block joining
// them instead, by a count of the blocks that are done, saved 3 us of host time and cost more on
// the GPU: one token over 2048 selected positions 11.7 us against 10.5.)
int launch(Params& p, const tks_cache* c, bool selected, void* stream) {
  Device d;
  Workspace ws;
  const int rc = prepare(stream, &d, &ws);
  if (rc != TKS_OK) return rc;
  p.status = reinterpret_cast<unsigned*>(ws.ptr);
  p.parts = reinterpret_cast<float*>(ws.ptr + kHeaderBytes);
  const int64_t keys = selected ? p.k_sel : std::min((int64_t)p.table_pages << p.page_shift, (int64_t)kMaxPositions);
  const bool i8 = c->held == TKS_I8;
  const cudaStream_t s = (cudaStream_t)stream;
  p.spin_limit_ns = spin_limit_ns();
  p.test_skip_arrive = test_skip_arrive();
  cudaError_t e;
  // Few rows: mma.sync with 16, else tcgen05 with 128 of them. With the latter for few rows too, one token
  // over 1M positions takes 288 us instead of 194, 64 over 2048 selected ones of 2 heads 38.2 instead
  // of 30.6: the operands' way through shared memory is paid for rows that are not there. (More than
  // 16 would be read twice by the former.)
  const bool few = p.rows <= kRowsTile;
  const int tile = few ? kRowsTile : kTilesRows, tile_keys = few ? kRowsKeys : kTilesKeys;
  p.row_tiles = (p.rows + tile - 1) / tile;
  if ((keys / tile_keys + 1) * p.kv_heads * p.row_tiles > INT32_MAX) return TKS_E_TOO_LARGE;
  const long long units = (long long)p.seqs * p.kv_heads * p.row_tiles;
  if (units > INT32_MAX) return TKS_E_TOO_LARGE;
  int grid = few ? d.sms * kRowsBlocksPerSm : d.sms;
  p.plan = reinterpret_cast<Split*>(ws.ptr + kPlanOffset);
  if (selected) {
    const long long tiles = std::max(1, (p.k_sel + tile_keys - 1) / tile_keys);
    p.split.set(units * tiles, (unsigned)tiles, units, grid);
  }
  const int cluster = selected && !few ? 0 : cluster_of(units, (keys + tile_keys - 1) / tile_keys, tile_keys, grid);
  if (cluster > 0) {
    p.cluster = cluster;
    p.split.share = (unsigned)cluster;
    grid = (int)units * cluster;
  }
  std::lock_guard<std::mutex> lock(*ws.order);
  if (few) {
    e = launch_rows(p, c->head_dim, i8, selected, grid, s);
    if (e == cudaSuccess && !cluster) e = launch_combine<kRowsTile, kRowsKeys>(p, c->head_dim, selected, grid, s);
  } else {
    e = launch_tiles(p, c->head_dim, i8, selected, grid, s);
    if (e == cudaSuccess && !cluster) e = launch_combine<kTilesRows, kTilesKeys>(p, c->head_dim, selected, grid, s);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}

CacheParams cache_params(const tks_cache* c, const int32_t* slots, int32_t n, unsigned* status) {
  CacheParams p{};
  const long long size = c->held == TKS_I8 ? 1 : 2;
  p.k = static_cast<unsigned char*>(c->k);
  p.v = static_cast<unsigned char*>(c->v);
  p.scales = c->scales;
  p.page_b = c->page_stride * size;
  p.token_b = c->token_stride * size;
  p.head_b = c->head_stride * size;
  p.page_shift = log2_of(c->page_size);
  p.kv_heads = c->kv_heads;
  p.head_shift = (c->kv_heads & (c->kv_heads - 1)) == 0 ? log2_of(c->kv_heads) : -1;
  p.slots_held = c->pages * c->page_size;
  p.slots = slots;
  p.n = n;
  p.status = status;
  return p;
}

}  // namespace
}  // namespace attn

int attn_status(int dev, void* stream) {
  using namespace attn;
  Workspace w;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    const auto it = g_ws.find(key_of(dev, stream));
    if (it == g_ws.end()) return TKS_OK;
    w = it->second;
  }
  // Calls of other threads wait: none is queued between the read and the clear, which would lose its
  // report, and none has its first kernel before the clear and its second behind.
  std::lock_guard<std::mutex> lock(*w.order);
  unsigned st = 0;
  if (cudaMemcpyAsync(&st, w.ptr, sizeof st, cudaMemcpyDeviceToHost, (cudaStream_t)stream) != cudaSuccess ||
      cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  if (st == 0) return TKS_OK;
  // (the word alone: behind it lies the split that a call's second kernel reads)
  if (cudaMemsetAsync(w.ptr, 0, sizeof st, (cudaStream_t)stream) != cudaSuccess ||
      cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  if (st & kStatTimeoutBit) return TKS_E_TIMEOUT;
  return st & kStatIndexBit ? TKS_E_INDEX : TKS_E_ROW_LEN;
}

int attn_release() {
  using namespace attn;
  std::lock_guard<std::mutex> lock(g_mu);
  int rc = TKS_OK, cur = 0;
  cudaGetDevice(&cur);
  for (auto& kv : g_ws) {
    cudaSetDevice(std::get<0>(kv.first));
    if (cudaFree(kv.second.ptr) != cudaSuccess) rc = TKS_E_CUDA;
  }
  cudaSetDevice(cur);
  cudaGetLastError();
  g_ws.clear();
  return rc;
}

}  // namespace tks

using namespace tks;
using namespace tks::attn;

extern "C" int tks_cache_write(const tks_cache* cache, const void* k, const void* v, int32_t n,
                               int32_t dtype, int64_t k_token_stride, int64_t k_head_stride,
                               int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                               void* stream) {
  if (check_cache(cache) != TKS_OK || n < 0 || (dtype != TKS_BF16 && dtype != TKS_F32)) return TKS_E_INVAL;
  if (n == 0) return TKS_OK;
  const int64_t size = dtype == TKS_F32 ? 4 : 2;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return TKS_E_INVAL;
  if (!strides_ok(size, n, k_token_stride, cache->kv_heads, k_head_stride) ||
      !strides_ok(size, n, v_token_stride, cache->kv_heads, v_head_stride))
    return TKS_E_INVAL;
  if ((int64_t)n * cache->kv_heads > INT32_MAX) return TKS_E_INVAL;
  Device d;
  Workspace ws;
  const int rc = prepare(stream, &d, &ws);
  if (rc != TKS_OK) return rc;
  CacheParams p = cache_params(cache, slots, n, reinterpret_cast<unsigned*>(ws.ptr));
  p.src_k = k;
  p.src_v = v;
  p.k_token = k_token_stride;
  p.k_head = k_head_stride;
  p.v_token = v_token_stride;
  p.v_head = v_head_stride;
  std::lock_guard<std::mutex> lock(*ws.order);
  if (launch_cache_write(p, cache->head_dim, cache->held == TKS_I8, dtype == TKS_F32, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}

extern "C" int tks_cache_read(const tks_cache* cache, const int32_t* slots, int32_t n, void* k_out,
                              void* v_out, int32_t dtype, void* stream) {
  if (check_cache(cache) != TKS_OK || n < 0 || (dtype != TKS_BF16 && dtype != TKS_F32)) return TKS_E_INVAL;
  if (n == 0) return TKS_OK;
  if (!slots || !k_out || !v_out || !aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return TKS_E_INVAL;
  if ((int64_t)n * cache->kv_heads > INT32_MAX) return TKS_E_INVAL;
  Device d;
  Workspace ws;
  const int rc = prepare(stream, &d, &ws);
  if (rc != TKS_OK) return rc;
  CacheParams p = cache_params(cache, slots, n, reinterpret_cast<unsigned*>(ws.ptr));
  p.out_k = k_out;
  p.out_v = v_out;
  std::lock_guard<std::mutex> lock(*ws.order);
  if (launch_cache_read(p, cache->head_dim, cache->held == TKS_I8, dtype == TKS_F32, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return TKS_E_CUDA;
  }
  return TKS_OK;
}

extern "C" int tks_tree_attention(const tks_cache* cache, const tks_queries* queries,
                                  const int32_t* ctx_len, const int32_t* draft_len,
                                  const int32_t* tree, void* stream) {
  if (check_cache(cache) != TKS_OK || check_queries(cache, queries) != TKS_OK) return TKS_E_INVAL;
  if (queries->tokens > TKS_DRAFTS_MAX) return TKS_E_INVAL;
  if (queries->batch == 0 || queries->tokens == 0) return TKS_OK;
  if (!ctx_len || !aligned(ctx_len, 4) || !aligned(draft_len, 4) || !aligned(tree, 4)) return TKS_E_INVAL;
  Params p = params_of(cache, queries);
  p.ctx_len = ctx_len;
  p.draft_len = draft_len;
  p.tree = tree;
  p.tree_words = (queries->tokens + 31) / 32;
  p.seqs = queries->batch;
  p.rows = queries->tokens * p.group;
  return launch(p, cache, false, stream);
}

extern "C" int tks_selected_attention(const tks_cache* cache, const tks_queries* queries,
                                      const int32_t* indices, int32_t k, const int32_t* kv_len,
                                      void* stream) {
  if (check_cache(cache) != TKS_OK || check_queries(cache, queries) != TKS_OK) return TKS_E_INVAL;
  if (k < 0 || k > TKS_K_MAX) return TKS_E_INVAL;
  if (queries->batch == 0 || queries->tokens == 0) return TKS_OK;
  if ((k > 0 && !indices) || !aligned(indices, 4) || !aligned(kv_len, 4)) return TKS_E_INVAL;
  Params p = params_of(cache, queries);
  p.indices = indices;
  p.k_sel = k;
  p.kv_len = kv_len;
  p.seqs = queries->batch * queries->tokens;
  p.rows = p.group;
  return launch(p, cache, true, stream);
}
