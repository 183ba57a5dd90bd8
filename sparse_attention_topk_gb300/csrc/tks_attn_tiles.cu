// Attention over a paged cache for many query rows of each key/value head:
// trees, wide head groups and selected positions of many heads, on the
// tcgen05 tensor cores.
//
// Mathematics: that of tks_attn_rows.cu (running maximum and sum; codes of an
// 8-bit cache exact in half precision, both scales folded into one
// multiply-add per score, weights relative to the largest contribution).
// What weights are relative to follows only when a row's maximum has grown by
// more than 2^8, so the output in tensor memory is rarely rescaled. Over 8 bits
// each row's queries get their own power of two: a row whose largest element is
// in [2^-7, 2^14) goes as it is, another is brought to [1, 2). Elements more than
// 2^10 (2^17) below the largest may be off, by 2^-18 (2^-25) of it at most.
//
// Layout.  A block is one SM: 128 query rows (a lane of tensor memory each)
// against tiles of 128 keys. Warps 0-7 keep the rows: they take scores into
// registers and write the weights back over them, as the next product's
// operand, so neither touches shared memory. Warp 8 issues the products, S = Q K^T of tile i + 1 before O += P V
// of tile i, into two score buffers, so they run while tile i's weights are
// made. Warps 9-11 look up where the tile's keys lie (list, page table, scales)
// some tiles ahead. Warps 12-19 bring the rows: 16-byte loads, codes widened to
// halves, stored as 128-byte-swizzled operand tiles (keys K-major for the first
// product; values, in the same form, read transposed by the second); a
// bfloat16 cache goes there by cp.async. Rows are gathered one by one, so
// pages, lists and the order of positions do not matter.
//
// What bounds it: over bfloat16 and few rows the cache's bytes (64 KB a tile,
// 2800 cycles at the memory's rate, against 1536 of tensor work for a full 128
// rows). Over int8, whose tile memory delivers in 1400 cycles, and with many
// rows: the eight warps that make weights and the eight that widen rows, which
// share an SM's issue slots and take about as long as each other.
// Measured: 8 ragged trees of 8 drafts over up to 65,536 positions (32 rows a
// head) of bfloat16 (1.16 GB) 193-195 us, 5.9-6.0 TB/s, of int8 (0.6 GB) 181 us,
// 3.3 TB/s, a tile in some 3100 cycles; two trees of 64 drafts over 32,768
// positions (512 rows a head, 137 Gflop) of int8 196 us, 700 Tflop/s, a tile in
// some 3500 cycles (161 us without making weights, 178 without loading rows, 103
// without both), of bfloat16 230 us; 512 queries of 64 heads over 2048 selected
// positions each 103 us of int8, of which a block's four changes of segment take
// some 6 us each, and 114 us of bfloat16.
//
// Every wait is bounded: a wait that runs out reports TKS_E_TIMEOUT and ends its
// warp's role, which makes the waits on that warp run out; when all roles have
// ended the block frees its tensor memory and returns.

#include "tks_attn.cuh"
#include "tks_tensor.cuh"

namespace tks {
namespace attn {
namespace {

constexpr int kThreads = 640;
constexpr int kRowWarps = 8, kMulWarp = 8, kMetaWarp0 = 9;  // then the producers
constexpr int kKeys = kTilesKeys;  // keys of a tile
constexpr int kMetas = 6;          // tiles whose lookups may be ahead
constexpr int kProducers = 256, kProducer0 = 384;

// Where a tile's keys lie, and what their scores are scaled with.
struct Meta {
  long long off[kKeys];  // byte offset of the row in the cache, or -1
  // for each pair of keys: key scale * softmax scale * log2(e) of both (0 for no key),
  // and log2 of the value scale of both (-inf for no key)
  float kl[kKeys / 2][4];
  float inv[kKeys];      // 1 / value scale; 0 for no key
  unsigned valid[4];     // which keys there are
  int draft0;            // the first drafted token's place in the tile (kKeys: none)
  int pad[3];
};

template <int D, bool I8>
struct Shape {
  static constexpr int kBlock = kKeys * 128;              // 64 elements of every row
  static_assert(kBlock >> 4 == 1024 && 16 * 128 >> 4 == 128, "the steps of tc_scores and tc_outputs");
  static constexpr int kMat = (D / 64) * kBlock;          // a tile's keys, or its values
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kMetaOff = kStages * 2 * kMat;
  static constexpr int kBarOff = kMetaOff + kMetas * (int)sizeof(Meta);
  static constexpr int kSmem = kBarOff + 512 + 1024;      // and room to align the base
  static constexpr int kRow = D * (I8 ? 1 : 2);
  static constexpr int kPieces = kRow / 16;               // 16-byte pieces of a row in the cache
  static constexpr int kPer = kKeys * kPieces / kProducers;  // pieces of a matrix that a thread brings
  // tensor memory columns
  static constexpr int kS = 0, kO = 256, kQ = 384;
};

// Barriers, in 8-byte words behind the metas.
enum Bar { kMetaFull = 0, kMetaEmpty = kMetaFull + kMetas, kKFull = kMetaEmpty + kMetas, kVFull = kKFull + 6, kEmpty = kVFull + 6,
           kSFull = kEmpty + 6, kPReady = kSFull + 2, kPvDone = kPReady + 2, kQReady = kPvDone + 2, kFinal = kQReady + 1, kPair = kFinal + 1, kBars = kPair + 4 };
static_assert(kBars * 8 <= 400, "barriers fit");

// What every role of the block shares.
struct Block {
  unsigned char* smem;  // stages
  uint32_t stage, bars; // shared-memory addresses
  volatile unsigned* poisoned;
  unsigned* status;
  long long limit;
  Meta* metas;

  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  template <bool NAP = false>
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const { return bar_wait<NAP>(bar(i), parity, limit, status); }
};

// ---- products ---------------------------------------------------------------
// A tile's product, D (tensor memory) (+)= A (tensor memory) x B (shared memory), sixteen of the
// summed index an instruction, and the arrivals at barriers when it is done: one lane issues all of
// it in one go, so that the tensor cores do not run dry between instructions. Step j's operands
// lie ja columns of A and jb 16-byte pieces of B behind the first's.
#define TKS_MMA(ja, jb) \
  "add.s32 a, %1, " ja ";\n\tadd.s64 b, %2, " jb ";\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
#define TKS_COMMIT(n) "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%" n "];\n\t"
#define TKS_MMA_BEGIN \
  "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\t" \
  "setp.eq.u32 t, 0, 0;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
// S = Q K^T: K-major keys, 32 bytes of a 128-byte row a step, blocks of 64 elements 16 KB apart.
template <int D>
__device__ __forceinline__ void tc_scores(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t bar) {
  if (D == 128)
    asm volatile(TKS_MMA_BEGIN TKS_MMA("8", "2") TKS_MMA("16", "4") TKS_MMA("24", "6") TKS_MMA("32", "1024") TKS_MMA("40", "1026")
                     TKS_MMA("48", "1028") TKS_MMA("56", "1030") TKS_COMMIT("5") "}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(0), "r"(bar)
                 : "memory");
  else
    asm volatile(TKS_MMA_BEGIN TKS_MMA("8", "2") TKS_MMA("16", "4") TKS_MMA("24", "6") TKS_COMMIT("5") "}" ::"r"(d), "r"(a), "l"(b),
                 "r"(idesc), "r"(0), "r"(bar)
                 : "memory");
}
// O (+)= P V: 16 keys' rows a step; the weights of the second 64 keys lie 64 columns behind the first's.
__device__ __forceinline__ void tc_outputs(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(TKS_MMA_BEGIN TKS_MMA("8", "128") TKS_MMA("16", "256") TKS_MMA("24", "384") TKS_MMA("64", "512") TKS_MMA("72", "640")
                   TKS_MMA("80", "768") TKS_MMA("88", "896") "}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((unsigned)add)
               : "memory");
}
__device__ __forceinline__ void tc_outputs(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t bar0, uint32_t bar1, uint32_t bar2) {
  asm volatile(TKS_MMA_BEGIN TKS_MMA("8", "128") TKS_MMA("16", "256") TKS_MMA("24", "384") TKS_MMA("64", "512") TKS_MMA("72", "640")
                   TKS_MMA("80", "768") TKS_MMA("88", "896") TKS_COMMIT("5") TKS_COMMIT("6") TKS_COMMIT("7") "}" ::"r"(d), "r"(a), "l"(b),
               "r"(idesc), "r"((unsigned)add), "r"(bar0), "r"(bar1), "r"(bar2)
               : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// 16 lanes by 64 (32) columns: register 4j + 2i + e is lane n + 8i, column 8j + 2c + e, of
// thread 4n + c.
__device__ __forceinline__ void tc_ld_frag(uint32_t (&r)[32], uint32_t addr) {
#define TKS_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : TKS_R32(TKS_OUT) : "r"(addr) : "memory");
#undef TKS_OUT
}
// 16 lanes by 32 columns: register 2j + i is lane n + 8i, column 4j + c.
__device__ __forceinline__ void tc_st_frag(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// 16 lanes by 8 columns.
__device__ __forceinline__ void tc_ld_piece(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st_scores(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%4], {%0, %1, %2, %3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(addr)
               : "memory");
}

// ---- pairs of 32-bit floats ---------------------------------------------------
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------

// Warps 9-11: the lookups of every third tile.
template <int D, bool I8, bool SEL, bool BLK>
__device__ __forceinline__ void look_up(const Params& p, const Block& k, const Start& start, int who) {
  const int lane = threadIdx.x & 31;
  Segments<SEL, kKeys> it;
  it.begin(start);
  Segment s;
  unsigned g = 0;  // the tile's number in this block
  bool bad = false;
  while (uniform((int)it.next(p, s))) {
    const int32_t* table = p.table + s.b * p.table_stride;
    const int32_t* list = SEL ? list_of<BLK>(p, s.seq, s.head) : nullptr;
    const int limit = SEL ? kv_limit(p, kv_given<BLK>(p, s.b, s.seq)) : 0;
    const int end = (int)min((long long)s.len.len, (long long)s.t1 * kKeys);
    auto entry = [&](int t, int i) -> int {  // key i of tile t: its list entry, or its position
      const int j = t * kKeys + i;
      if (t >= s.t1 || j >= end) return -1;
      return SEL ? __ldg(list + list_entry<BLK>(p, j)) : j;
    };
    int t = uniform(s.t0 + (int)((who + 3u - g % 3u) % 3u));
    const int t1 = uniform(s.t1);
    int e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = entry(t, lane + 32 * i);
    for (; t < t1; t += 3) {
      int pos[4], pg[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pos[i] = SEL ? list_position<BLK>(p, e[i], t * kKeys + lane + 32 * i, limit, bad) : e[i];
        pg[i] = pos[i] < 0 ? -1 : __ldg(table + (pos[i] >> p.page_shift));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = entry(t + 3, lane + 32 * i);
      float2 sc[4];
      long long off[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = pos[i] >= 0 && (unsigned)pg[i] < (unsigned)p.pages;
        bad |= pos[i] >= 0 && !ok;
        const int in_page = pos[i] & ((1 << p.page_shift) - 1);
        off[i] = ok ? pg[i] * p.page_b + in_page * p.token_b + s.head * p.head_b : -1;
        sc[i] = make_float2(0.f, 1.f);
        if (I8 && ok) sc[i] = p.scales[(((long long)pg[i] << p.page_shift) + in_page) * p.kv_heads + s.head];
      }
      const unsigned tile = uniform(g + (unsigned)(t - s.t0)), slot = tile % kMetas;
      if (tile >= kMetas && !k.wait<true>(kMetaEmpty + slot, (tile / kMetas & 1) ^ 1)) return;
      Meta& m = k.metas[slot];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = lane + 32 * i;
        const bool ok = off[i] >= 0;
        const unsigned bits = __ballot_sync(0xffffffffu, ok);
        m.off[key] = off[i];
        if (I8) {
          const float lo = 7.105427357601002e-15f;  // 2^-47: a NaN stays one
          const float vs = sc[i].y < lo ? lo : sc[i].y;
          m.kl[key >> 1][key & 1] = ok ? sc[i].x * p.scale_log2 : 0.f;
          m.kl[key >> 1][2 + (key & 1)] = ok ? lg2(vs) : -INFINITY;
          m.inv[key] = !ok ? 0.f : vs == vs ? __fdividef(1.f, vs) : 1.f;  // (finite: a weight of 0 times it is 0)
        }
        if (lane == 0) m.valid[i] = bits;
      }
      if (lane == 0) {
        const long long d = SEL ? kKeys : (long long)s.len.ctx - (long long)t * kKeys;
        m.draft0 = d >= kKeys ? kKeys : (int)max(d, 0LL);
      }
      __syncwarp();
      if (!(p.test_skip_arrive && tile == 0)) bar_arrive(k.bar(kMetaFull + slot));
    }
    g += (unsigned)(s.t1 - s.t0);
  }
  if (bad) report(p.status, kStatIndexBit);
}

// Warps 12-19: the rows of every tile into its stage.
template <int D, bool I8>
__device__ __forceinline__ void produce(const Params& p, const Block& k, int tiles) {
  using S = Shape<D, I8>;
  const int t = threadIdx.x - kProducer0;
  constexpr int kRows = kProducers / S::kPieces;  // rows that a pass covers
  // A thread's piece of a row, and its first row. Eight neighbouring lanes take half of two rows
  // of int8 (two 16-byte stores a piece), or a row's half of bfloat16: no bank conflicts.
  const bool split = I8 && S::kPieces == 8;
  const int piece = split ? (t & 3) | (t >> 2 & 4) : t % S::kPieces;
  const int row0 = split ? (t >> 5) * 4 + (t >> 2 & 3) : t / S::kPieces;

  if (I8) {
    // A matrix's rows of the next tile are loaded as soon as this tile's have been stored.
    const int blk = (piece >> 2) * S::kBlock, first = (piece & 3) * 2;
    uint4 w[2][S::kPer];
    Ring<kMetas> meta;
    Ring<S::kStages> st;
#pragma unroll 1
    for (int g = -1; g < tiles; ++g) {  // (-1: only loads)
      const bool more = g + 1 < tiles;
      if (more && !k.wait(kMetaFull + meta.i, meta.parity)) return;
      if (g >= S::kStages && !k.wait<true>(kEmpty + st.i, st.parity ^ 1)) return;
      const Meta& m = k.metas[meta.i];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (g >= 0) {
          unsigned char* base = k.smem + (2 * st.i + kv) * S::kMat + blk;
#pragma unroll
          for (int i = 0; i < S::kPer; ++i) {
            const int r = row0 + i * kRows;
            const uint32_t a[4] = {w[kv][i].x ^ 0x80808080u, w[kv][i].y ^ 0x80808080u, w[kv][i].z ^ 0x80808080u, w[kv][i].w ^ 0x80808080u};
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<uint4*>(base + r * 128 + (((first + j) ^ (r & 7)) << 4)) =
                  make_uint4(codes_to_half2<0x4140>(a[2 * j]), codes_to_half2<0x4342>(a[2 * j]),
                             codes_to_half2<0x4140>(a[2 * j + 1]), codes_to_half2<0x4342>(a[2 * j + 1]));
          }
          __syncwarp();
          bar_arrive(k.bar((kv ? kVFull : kKFull) + st.i));
        }
        if (more) {
          const unsigned char* base = (kv ? p.v : p.k) + piece * 16;
#pragma unroll
          for (int i = 0; i < S::kPer; ++i) {
            const long long off = m.off[row0 + i * kRows];
            w[kv][i] = make_uint4(0u, 0u, 0u, 0u);
            if (off >= 0) w[kv][i] = __ldg(reinterpret_cast<const uint4*>(base + off));
          }
        }
      }
      if (more) {
        __syncwarp();
        bar_arrive(k.bar(kMetaEmpty + meta.i));
        meta.next();
      }
      if (g >= 0) st.next();
    }
    return;
  }

  // bfloat16: cp.async straight into the stage; a tile is announced when the next one's copies are under way.
  const int blk = (piece >> 3) * S::kBlock, at = piece & 7;
  auto announce = [&](int st) {
    __syncwarp();
    bar_arrive(k.bar(kKFull + st));
    bar_arrive(k.bar(kVFull + st));
  };
  Ring<kMetas> meta;
  Ring<S::kStages> ring;
  int last = 0;
  for (int g = 0; g < tiles; ++g) {
    const int st = ring.i;
    if (!k.wait(kMetaFull + meta.i, meta.parity) || (g >= S::kStages && !k.wait<true>(kEmpty + st, ring.parity ^ 1))) {
      cp_wait<0>();
      return;
    }
    const Meta& m = k.metas[meta.i];
    const int draft0 = m.draft0;
    const uint32_t kd = k.stage + 2 * st * S::kMat + blk, vd = kd + S::kMat;
#pragma unroll
    for (int i = 0; i < S::kPer; ++i) {
      const int r = row0 + i * kRows;
      const long long off = m.off[r];
      const long long src = off < 0 ? 0 : off + piece * 16;
      const int dst = r * 128 + ((at ^ (r & 7)) << 4);
      cp16(kd + dst, p.k + src, off < 0 ? 0 : 16);
      if (r < draft0) cp16(vd + dst, p.v + src, off < 0 ? 0 : 16);
    }
    if (draft0 < kKeys) {
      // drafted tokens: infinities and NaNs must not meet the zero weights of rows that do not see them
      bool bad = false;
#pragma unroll 1
      for (int i = 0; i < S::kPer; ++i) {
        const int r = row0 + i * kRows;
        if (r < draft0) continue;
        const long long off = m.off[r];
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (off >= 0) x = *reinterpret_cast<const uint4*>(p.v + off + piece * 16);
        uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((u[j] & 0x7f80u) == 0x7f80u) { u[j] &= 0xffff0000u; bad = true; }
          if ((u[j] & 0x7f800000u) == 0x7f800000u) { u[j] &= 0x0000ffffu; bad = true; }
        }
        *reinterpret_cast<uint4*>(k.smem + (2 * st + 1) * S::kMat + blk + r * 128 + ((at ^ (r & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      if (bad) *k.poisoned = 1;
    }
    cp_commit();
    __syncwarp();
    bar_arrive(k.bar(kMetaEmpty + meta.i));
    if (g > 0) {
      cp_wait<1>();
      announce(last);
    }
    last = st;
    meta.next();
    ring.next();
  }
  cp_wait<0>();
  if (tiles > 0) announce(last);
}

// Warp 8: the products.
template <int D, bool I8, bool SEL>
__device__ __forceinline__ void multiply(const Params& p, const Block& k, const Start& start, uint32_t tmem) {
  using S = Shape<D, I8>;
  constexpr uint32_t kQk = instr(I8, false, kKeys), kPv = instr(I8, true, D);
  Segments<SEL, kKeys> it;
  it.begin(start);
  Segment s;
  Ring<S::kStages> kr, vr;  // the stages of the first and of the second product
  Ring<kMetas> mr;          // the second's lookups, which are done with, too
  uint32_t gk = 0, gv = 0;  // their tiles, whose lowest bit is the score buffer
  uint32_t seg = 0;
  const uint64_t keys0 = operand(k.stage, 16), values0 = operand(k.stage + S::kMat, S::kBlock);
  bool ok = true;
  while (ok && uniform((int)it.next(p, s))) {
    if (!k.wait(kQReady, seg & 1)) break;
    const int n = uniform(s.t1 - s.t0);
#pragma unroll 1
    for (int i = 0; i <= n; ++i) {
      if (i < n) {  // S = Q K^T of tile i
        if (!k.wait(kKFull + kr.i, kr.parity)) { ok = false; break; }
        proxy_fence();
        tc_fence_after();
        const uint64_t b = keys0 + (uint32_t)(kr.i * (2 * S::kMat >> 4));
        const uint32_t d = tmem + S::kS + (gk & 1) * 128;
        tc_scores<D>(d, tmem + S::kQ, b, kQk, k.bar(kSFull + (gk & 1)));
        kr.next();
        ++gk;
      }
      if (i > 0) {  // O (+)= P V of tile i - 1
        if (!k.wait(kVFull + vr.i, vr.parity) || !k.wait(kPReady + (gv & 1), gv >> 1 & 1)) { ok = false; break; }
        proxy_fence();
        tc_fence_after();
        const uint64_t v = values0 + (uint32_t)(vr.i * (2 * S::kMat >> 4));
        const uint32_t a = tmem + S::kS + (gv & 1) * 128;
        if (!I8) tc_outputs(tmem + S::kO, a + 32, v, kPv, i > 1);  // the weights' second parts
        tc_outputs(tmem + S::kO, a, v, kPv, !I8 || i > 1, k.bar(kEmpty + vr.i), k.bar(kMetaEmpty + mr.i), k.bar(kPvDone + (gv & 1)));
        mr.next();
        vr.next();
        ++gv;
      }
    }
    ++seg;
  }
  // nothing may be under way when tensor memory is freed
  tc_commit(k.bar(kFinal));
  k.wait(kFinal, 0);
}

// What the two warps of a quarter of the rows tell each other, and themselves. Rows of a quarter
// are lanes: row 16h + n of it, and row 16h + n + 8, at [h][n].
struct PairRows {
  float2 top[2][2][2][8];    // a tile's maxima: [tile & 1][half of the keys]
  float2 sum[2][2][8];       // a segment's sums, by half of the keys
  float2 m[2][8];            // and maxima
  float2 before[2][32];      // maximum and sum of a run's pieces before this one, by row (a copy for each warp)
  float fac[2][32];          // what undoes the shifts of the rows' queries (a copy for each warp)
  unsigned seen[2][2][32];   // the keys that a row sees: [half of the keys][32 keys]
};
// Scales 16 lanes by 32 columns: lanes n by fa, lanes n + 8 by fb.
__device__ __forceinline__ void rescale(uint32_t addr, float fa, float fb) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * (i & 2 ? fb : fa));
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// The segments of a row warp, kept in shared memory: its registers hold scores.
template <bool SEL>
struct RowSegments {
  Segments<SEL, kKeys> it;
  Segment s[2];
};

// Warps 0-7: warps w and w + 4 have the rows of lanes 32w .. 32w + 31, warp w the first 64 keys of
// every tile, warp w + 4 the others. Scores come in the layout of matrix fragments, 16 rows a
// step (STEPS of them): thread 4n + c has rows n and n + 8 and keys 8j + 2c, 8j + 2c + 1, so the
// scales that it needs are an eighth of the tile's. What few tiles need (masks, shifted rows) is done in tensor
// memory ahead of the common way, which stays short: instructions not fetched in time bound a
// longer one. Queries and outputs go by whole rows, a thread each, and
// half the elements for each warp. Up to 64 rows lie in the first 16 lanes of each quarter, so
// that all the warps share them.
template <int D, bool I8, bool SEL, int STEPS>
__device__ __forceinline__ void rows(const Params& p, const Block& k, const Start& start, uint32_t tmem, RowSegments<SEL>& segs, PairRows& pr,
                                     const float4* plain_kl) {
  using S = Shape<D, I8>;
  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31, quarter = warp & 3, half = warp >> 2;
  const int n = lane >> 2, c = lane & 3;
  const int row_lane = lane < 16 * STEPS ? quarter * 16 * STEPS + lane : 1 << 20;  // this lane's row in the tile
  const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16);
  if (lane == 0) segs.it.begin(start);
  // the next segment, into place `at`
  auto advance = [&](int at) -> bool {
    int more = 0;
    if (lane == 0) more = segs.it.next(p, segs.s[at]) ? 1 : 0;
    __syncwarp();  // (a shuffle orders no memory: the other lanes read what lane 0 has written)
    return __shfl_sync(0xffffffffu, more, 0) != 0;
  };
  // Whether the second product of tile i is done. (That of tile i - 2, its barrier's phase
  // before, is: tile i's scores came after it.)
  auto outputs_done = [&](uint32_t i) -> bool {
    if (!k.wait(kPvDone + (i & 1), i >> 1 & 1)) return false;
    tc_fence_after();
    return true;
  };
  uint32_t meetings = 0;
  // Both warps of the quarter have come this far, their shared- and tensor-memory accesses done.
  auto meet = [&]() -> bool {
    tc_fence_before();
    __syncwarp();
    bar_arrive(k.bar(kPair + quarter));
    if (!k.wait(kPair + quarter, meetings++ & 1)) return false;
    tc_fence_after();
    return true;
  };
  bool shifted = false;   // some row's queries are not as they were
  float next_back = 1.f;  // what undoes the shift of this lane's row
  uint32_t g = 0;  // the tile's number in this block
  Ring<kMetas> mr;
  int at = 0;

  // Puts segment s's queries into tensor memory.
  auto queries = [&](const Segment& s) {
    const int R = s.row_tile * kTilesRows + row_lane;
    const __nv_bfloat16* q = R < p.rows ? q_row<SEL>(p, s.seq, s.head, R) : nullptr;
    float up = 1.f, back = 1.f;
    if (I8) {
      float top = 0.f;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 x = q ? __ldg(reinterpret_cast<const uint4*>(q + 8 * i)) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = fabsf(__uint_as_float(w[j] << 16)), b = fabsf(__uint_as_float(w[j] & 0xffff0000u));
          top = a < INFINITY ? fmaxf(top, a) : top;
          top = b < INFINITY ? fmaxf(top, b) : top;
        }
      }
      // a row whose largest finite magnitude is in [2^-7, 2^14) goes as it is, another is shifted to 1
      if (top > 0.f && (top < 0.0078125f || top >= 16384.f)) {
        const int shift = max(-120, min(120, -ilogbf(top)));
        up = __int_as_float((shift + 127) << 23);
        back = __int_as_float((127 - shift) << 23);
      }
    }
#pragma unroll 1
    for (int i = 0; i < D / 64; ++i) {  // 32 elements a step
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = q ? __ldg(reinterpret_cast<const uint4*>(q + half * (D / 2) + 32 * i + 8 * j)) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
      }
      if (I8)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[j] = pack_half(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
      __syncwarp();  // (tensor memory is accessed by whole warps; lanes have rows to load, or none)
      tc_st16(mine + S::kQ + half * (D / 4) + 16 * i, w);
    }
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    bar_arrive(k.bar(kQReady));
    shifted = __any_sync(0xffffffffu, back != 1.f);
    next_back = back;
  };

  // The scores, scaled, in pairs of keys: v[h][i][j] of row 16h + n + 8i, keys 8j + 2c, 8j + 2c + 1.
  auto scores = [&](uint32_t addr, const float4* kl, float f, uint64_t (&v)[STEPS][2][8]) {
    uint32_t x[STEPS][32];
#pragma unroll
    for (int h = 0; h < STEPS; ++h) tc_ld_frag(x[h], addr + ((uint32_t)(16 * h) << 16));
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const ulonglong2 e = I8 ? *reinterpret_cast<const ulonglong2*>(kl + 4 * j) : make_ulonglong2(pair(f, f), 0);
#pragma unroll
      for (int h = 0; h < STEPS; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t a = pair(__uint_as_float(x[h][4 * j + 2 * i]), __uint_as_float(x[h][4 * j + 2 * i + 1]));
          v[h][i][j] = I8 ? fma2(a, e.x, e.y) : mul2(a, e.x);
        }
    }
  };

  bool more = advance(0);
  if (more) queries(segs.s[0]);
  while (more) {
    const Segment& s = segs.s[at];
    const int R0 = s.row_tile * kTilesRows + quarter * 16 * STEPS;
    const float back = next_back;
    const bool warp_live = uniform((int)(R0 < p.rows)) != 0;
    float m[STEPS][2];
    uint64_t sum[STEPS][2];
#pragma unroll
    for (int h = 0; h < STEPS; ++h) {
      m[h][0] = m[h][1] = -INFINITY;
      sum[h][0] = sum[h][1] = 0;
    }

    const int t0 = uniform(s.t0), t1 = uniform(s.t1);
    // the next segment's queries are brought near while this one's tiles run
    more = advance(at ^ 1);
    if (more) {
      const Segment& next = segs.s[at ^ 1];
      const int Rn = next.row_tile * kTilesRows + row_lane;
      if (Rn < p.rows) prefetch_l2(q_row<SEL>(p, next.seq, next.head, Rn) + half * (D / 2));
    }
    for (int t = t0; t < t1; ++t, ++g) {
      const uint32_t sb = mine + S::kS + (g & 1) * 128 + half * 64;
      if (!warp_live) {
        if (!k.wait<true>(kSFull + (g & 1), g >> 1 & 1)) return;
      } else {
        if (!k.wait(kSFull + (g & 1), g >> 1 & 1)) return;
        tc_fence_after();
        // (scores exist, so the tile's lookups do)
        const Meta& meta = k.metas[mr.i];
        const uint4 all = *reinterpret_cast<const uint4*>(meta.valid);
        const bool plain = uniform((int)((all.x & all.y & all.z & all.w) == ~0u && meta.draft0 == kKeys)) != 0 && !shifted;
        const float4* kl = reinterpret_cast<const float4*>(meta.kl) + 32 * half + c;
        float f = p.scale_log2;
        if (!plain) {
          // Missing keys, drafted tokens, shifted rows: the scores are scaled and masked in tensor
          // memory first, and what follows takes them as they are.
          const int tr = SEL ? 0 : min((R0 + lane) / p.group, p.tokens - 1), j0 = t * kKeys + 64 * half - s.len.ctx;
          const bool drafts = !SEL && meta.draft0 < kKeys;
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < 2; ++i)
            pr.seen[half][i][lane] = meta.valid[2 * half + i] & (drafts ? draft_bits(p, s.b, tr, j0 + 32 * i) : ~0u);
          pr.fac[half][lane] = back;
          __syncwarp();
#pragma unroll 1
          for (int e = 0; e < 8 * STEPS; ++e) {
            const int h = e >> 3, j = e & 7;
            uint32_t x[4];
            tc_ld_piece(x, sb + 8 * j + ((uint32_t)(16 * h) << 16));
            tc_wait_ld();
            const float4 e4 = I8 ? kl[4 * j] : make_float4(f, f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = 16 * h + n + 8 * i;
              const unsigned bits = pr.seen[half][j >> 2][row] >> (8 * (j & 3) + 2 * c);
              const float b = pr.fac[half][row];
              x[2 * i] = __float_as_uint(bits & 1u ? fmaf(__uint_as_float(x[2 * i]) * b, e4.x, e4.z) : -INFINITY);
              x[2 * i + 1] = __float_as_uint(bits & 2u ? fmaf(__uint_as_float(x[2 * i + 1]) * b, e4.y, e4.w) : -INFINITY);
            }
            __syncwarp();
            tc_st_scores(sb + 8 * j + ((uint32_t)(16 * h) << 16), x);
          }
          tc_wait_st();
          kl = plain_kl + c;
          f = 1.f;
        }

        uint64_t v[STEPS][2][8];
        scores(sb, kl, f, v);
        float top[STEPS][2];
#pragma unroll
        for (int h = 0; h < STEPS; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2 a = unpair(v[h][i][0]), b = unpair(v[h][i][1]);
            float x0 = fmaxf(a.x, a.y), x1 = fmaxf(b.x, b.y);
#pragma unroll
            for (int j = 2; j < 8; j += 2) {
              a = unpair(v[h][i][j]);
              b = unpair(v[h][i][j + 1]);
              x0 = fmaxf(x0, fmaxf(a.x, a.y));
              x1 = fmaxf(x1, fmaxf(b.x, b.y));
            }
            top[h][i] = fmaxf(x0, x1);
          }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1)
#pragma unroll
          for (int h = 0; h < STEPS; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) top[h][i] = fmaxf(top[h][i], __shfl_xor_sync(0xffffffffu, top[h][i], o));
        if (c == 0)
#pragma unroll
          for (int h = 0; h < STEPS; ++h) pr.top[g & 1][half][h][n] = make_float2(top[h][0], top[h][1]);
        if (!meet()) return;

        // What the weights are relative to (kWeightLog2): -inf as long as a row has seen nothing.
        constexpr float kAbove = kWeightLog2<I8>;
        bool grow = false;
#pragma unroll
        for (int h = 0; h < STEPS; ++h) {
          const float2 y = pr.top[g & 1][half ^ 1][h][n];
          top[h][0] = fmaxf(top[h][0], y.x);
          top[h][1] = fmaxf(top[h][1], y.y);
          grow |= top[h][0] - m[h][0] > 8.f + kAbove || top[h][1] - m[h][1] > 8.f + kAbove;  // (both -inf: no; see tks_attn_rows.cu)
        }
        if (__any_sync(0xffffffffu, grow)) {
          if (t > t0 && !outputs_done(g - 1)) return;
#pragma unroll
          for (int h = 0; h < STEPS; ++h) {
            float back2[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool up = top[h][i] - m[h][i] > 8.f + kAbove;
              const float next = top[h][i] - kAbove;
              back2[i] = up ? ex2(m[h][i] - next) : 1.f;  // (m = -inf: 0)
              if (up) m[h][i] = next;
              sum[h][i] = mul2(sum[h][i], pair(back2[i], back2[i]));
            }
            if (t > t0)
#pragma unroll 1
              for (int i = 0; i < D / 64; ++i)
                rescale(mine + S::kO + half * (D / 2) + 32 * i + ((uint32_t)(16 * h) << 16), back2[0], back2[1]);
          }
        }

        // Weights and their sums. Rounded, they go over the scores' first 32 columns of these 64 keys
        // (bfloat16: their second parts over the other 32).
        uint32_t w[STEPS][16], rest[I8 ? 1 : STEPS][16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t inv = I8 ? *reinterpret_cast<const uint64_t*>(meta.inv + 64 * half + 8 * j + 2 * c) : 0;
#pragma unroll
          for (int h = 0; h < STEPS; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float u = m[h][i] == -INFINITY ? 0.f : -m[h][i];
              const float2 a = unpair(add2(v[h][i][j], pair(u, u)));
              const float e0 = ex2(a.x), e1 = ex2(a.y);
              sum[h][i] = I8 ? fma2(pair(e0, e1), inv, sum[h][i]) : add2(sum[h][i], pair(e0, e1));
              if (I8) w[h][2 * j + i] = pack_half(e0, e1);
              else split_bf16(e0, e1, w[h][2 * j + i], rest[I8 ? 0 : h][2 * j + i]);
            }
        }
#pragma unroll
        for (int h = 0; h < STEPS; ++h) {
          tc_st_frag(sb + ((uint32_t)(16 * h) << 16), w[h]);
          if (!I8) tc_st_frag(sb + 32 + ((uint32_t)(16 * h) << 16), rest[I8 ? 0 : h]);
        }
        tc_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      bar_arrive(k.bar(kPReady + (g & 1)));
      mr.next();
    }

    // The next segment's queries first (its scores can begin), then this one's output.
    const Segment& done = s;
    if (more) queries(segs.s[at ^ 1]);
    if (!outputs_done(g - 1)) return;
    if (warp_live) {
#pragma unroll
      for (int h = 0; h < STEPS; ++h) {
        float l[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 a = unpair(sum[h][i]);
          l[i] = a.x + a.y;
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        if (c == 0) {
          pr.sum[half][h][n] = make_float2(l[0], l[1]);
          if (half == 0) pr.m[h][n] = make_float2(m[h][0], m[h][1]);
        }
      }
      if (!meet()) return;
      const int R = done.row_tile * kTilesRows + row_lane, hl = lane >> 4, nl = lane & 7;
      const bool low = (lane & 8) == 0;
      const int t_row = SEL ? 0 : min(R / p.group, p.tokens - 1);
      const bool live = R < p.rows && (SEL || R / p.group < done.len.drafts);
      const float2 la = pr.sum[0][hl][nl], lb = pr.sum[1][hl][nl], mm = pr.m[hl][nl];
      float lr = low ? la.x + lb.x : la.y + lb.y, top = low ? mm.x : mm.y;
      bool empty = !live || lr == 0.f;
      // What this piece and those before count for in the run so far; theirs is in the slot, where this
      // thread has put it.
      float now = empty ? 0.f : 1.f, past = 0.f;
      if (done.goes_on()) {
        const float2 q = pr.before[half][lane];
        if (q.y != 0.f) {
          const float most = empty ? q.x : fmaxf(top, q.x);
          if (!empty) now = top == most ? 1.f : ex2(top - most);
          past = q.x == most ? 1.f : ex2(q.x - most);
          lr = (empty ? 0.f : now * lr) + past * q.y;
          top = most;
          empty = false;
        }
      }
      if (done.more) pr.before[half][lane] = make_float2(top, empty ? 0.f : lr);
      const float inv = empty ? 0.f : 1.f / lr;
      const bool fix = !I8 && !SEL && *k.poisoned != 0;
      const long long row = out_row<SEL>(p, done.seq, done.head, min(R, p.rows - 1));
      // (in a cluster, the block's one partial takes the place of its stages, which are done with)
      const bool whole = done.whole() && (SEL || !p.cluster);
      float* part = !SEL && p.cluster ? reinterpret_cast<float*>(k.smem) : p.parts + (2LL * blockIdx.x + (done.first ? 0 : 1)) * kPartFloats<kTilesRows, D>;
#pragma unroll 1
      for (int i = 0; i < D / 64; ++i) {
        const int d = half * (D / 2) + 32 * i;
        uint32_t o[32];
        tc_ld32(o, mine + S::kO + d);
        tc_wait_ld();
        if (R < p.rows) {
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = now == 0.f ? 0.f : __uint_as_float(o[j]);
          if (fix && now != 0.f) {  // infinities and NaNs of drafts that this row attends to
            const int32_t* table = p.table + done.b * p.table_stride;
            const int end = (int)min((long long)done.len.len, (long long)done.t1 * kKeys);
            for (int j = max(done.len.ctx, done.t0 * kKeys); j < end; ++j) {
              const int pg = table[j >> p.page_shift];
              if ((unsigned)pg >= (unsigned)p.pages || !sees_draft(p, done.b, t_row, j - done.len.ctx)) continue;
              const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(
                  p.v + pg * p.page_b + (j & ((1 << p.page_shift) - 1)) * p.token_b + done.head * p.head_b) + d;
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float y = __bfloat162float(v[c]);
                if (!(fabsf(y) < INFINITY)) f[c] += y;
              }
            }
          }
          if (past != 0.f) {
            const float4* was = reinterpret_cast<const float4*>(part + row_lane * D + d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 x = was[j];
              f[4 * j] = f[4 * j] * now + x.x * past;
              f[4 * j + 1] = f[4 * j + 1] * now + x.y * past;
              f[4 * j + 2] = f[4 * j + 2] * now + x.z * past;
              f[4 * j + 3] = f[4 * j + 3] * now + x.w * past;
            }
          }
          if (whole) {
            uint4* out = reinterpret_cast<uint4*>(p.out + row * D + d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              out[j] = make_uint4(pack_bf16(f[8 * j] * inv, f[8 * j + 1] * inv), pack_bf16(f[8 * j + 2] * inv, f[8 * j + 3] * inv),
                                  pack_bf16(f[8 * j + 4] * inv, f[8 * j + 5] * inv), pack_bf16(f[8 * j + 6] * inv, f[8 * j + 7] * inv));
          } else {
            float4* out = reinterpret_cast<float4*>(part + row_lane * D + d);
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
          }
        }
        __syncwarp();
      }
      if (R < p.rows && half == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(part + kTilesRows * D + 2 * row_lane) = make_float2(top, empty ? 0.f : lr);
        else if (p.lse)
          p.lse[row] = empty ? -INFINITY : (top + lg2(lr)) * 0.6931471805599453f;
      }
    }
    tc_fence_before();  // these reads come before the next segment's products (through kPReady)
    at ^= 1;
    __syncwarp();
  }
}

template <int D, bool I8, bool SEL, int STEPS, bool BLK>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, I8>;
  extern __shared__ unsigned char raw[];
  __shared__ Start start;
  __shared__ unsigned poisoned_s;
  __shared__ uint32_t tmem_s;
  __shared__ RowSegments<SEL> segs[kRowWarps];
  __shared__ __align__(16) PairRows pair_rows[4];
  __shared__ float4 plain_kl[32];  // the scales of scores that are scaled already

  unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  Block k;
  k.smem = smem;
  k.stage = smem_addr(smem);
  k.bars = smem_addr(smem + S::kBarOff);
  k.poisoned = &poisoned_s;
  k.status = p.status;
  k.limit = p.spin_limit_ns;
  k.metas = reinterpret_cast<Meta*>(smem + S::kMetaOff);
  const int warp = uniform((int)threadIdx.x >> 5);

  if (warp == kMulWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_s)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x < 32) plain_kl[threadIdx.x] = make_float4(1.f, 1.f, 0.f, 0.f);
  if (threadIdx.x == 0) {
    poisoned_s = 0;
    for (int i = 0; i < kMetas; ++i) {
      bar_init(k.bar(kMetaFull + i), 1);
      bar_init(k.bar(kMetaEmpty + i), 9);
    }
    for (int i = 0; i < S::kStages; ++i) {
      bar_init(k.bar(kKFull + i), 8);
      bar_init(k.bar(kVFull + i), 8);
      bar_init(k.bar(kEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(k.bar(kSFull + i), 1);
      bar_init(k.bar(kPReady + i), kRowWarps);
      bar_init(k.bar(kPvDone + i), 1);
    }
    for (int i = 0; i < 4; ++i) bar_init(k.bar(kPair + i), 2);
    bar_init(k.bar(kQReady), kRowWarps);
    bar_init(k.bar(kFinal), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  grid_wait();
  grid_launch_dependents();
  if (warp == kMetaWarp0) find_start<SEL, kKeys>(p, &start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tmem_s);
  const int tiles = uniform((int)start.left);

  // Registers, of the launch's 5 * 96: 2 * 128 + 64 + 2 * 80, or, where weights are split in two and
  // rows go straight to shared memory, 2 * 144 + 64 + 2 * 64.
  if (warp < kRowWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(I8 ? 128 : 144));
    rows<D, I8, SEL, STEPS>(p, k, start, tmem, segs[warp], pair_rows[warp & 3], plain_kl);
    if (!SEL && p.cluster) {  // (the other warps have given registers up)
      float2* ml = reinterpret_cast<float2*>(smem + kTilesRows * D * 4);
      if (start.left == 0 && threadIdx.x < kTilesRows) ml[threadIdx.x] = make_float2(-INFINITY, 0.f);
      join_cluster<kTilesRows, D, SEL>(p, smem_addr(smem), smem_addr(ml), kRowWarps * 32);
    }
  } else if (warp < kRowWarps + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == kMulWarp) {
      multiply<D, I8, SEL>(p, k, start, tmem);
    } else {
      look_up<D, I8, SEL, BLK>(p, k, start, warp - kMetaWarp0);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(I8 ? 80 : 64));
    produce<D, I8>(p, k, tiles);
  }
  if (!SEL && p.cluster && warp >= kRowWarps) {  // join_cluster's two meetings
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMulWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D, bool I8, bool SEL, int STEPS, bool BLK = false>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<D, I8>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute a[2] = {};
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, p.cluster);
  return cudaLaunchKernelEx(&cfg, tiles_kernel<D, I8, SEL, STEPS, BLK>, p);
}
template <bool I8>
cudaError_t launch_held(const Params& p, int head_dim, bool selected, int grid, cudaStream_t stream) {
  // Up to 64 rows lie in the first 16 lanes of each quarter, one step of 16 rows a warp instead of two
  // (8 ragged trees of 32 rows a head: 195 us so, 230 in two steps).
  const bool one = p.rows <= 64;
  if (p.blocks) {
    if (head_dim == 64) return one ? launch<64, I8, true, 1, true>(p, grid, stream) : launch<64, I8, true, 2, true>(p, grid, stream);
    return one ? launch<128, I8, true, 1, true>(p, grid, stream) : launch<128, I8, true, 2, true>(p, grid, stream);
  }
  if (head_dim == 64) {
    if (selected) return one ? launch<64, I8, true, 1>(p, grid, stream) : launch<64, I8, true, 2>(p, grid, stream);
    return one ? launch<64, I8, false, 1>(p, grid, stream) : launch<64, I8, false, 2>(p, grid, stream);
  }
  if (selected) return one ? launch<128, I8, true, 1>(p, grid, stream) : launch<128, I8, true, 2>(p, grid, stream);
  return one ? launch<128, I8, false, 1>(p, grid, stream) : launch<128, I8, false, 2>(p, grid, stream);
}

template <int D, bool I8, bool SEL, bool BLK = false>
cudaError_t opt_in() {
  const cudaError_t e = allow(tiles_kernel<D, I8, SEL, 1, BLK>, Shape<D, I8>::kSmem);
  return e != cudaSuccess ? e : allow(tiles_kernel<D, I8, SEL, 2, BLK>, Shape<D, I8>::kSmem);
}
template <bool I8>
cudaError_t setup_held() {
  cudaError_t e = opt_in<64, I8, false>();
  if (e == cudaSuccess) e = opt_in<64, I8, true>();
  if (e == cudaSuccess) e = opt_in<128, I8, false>();
  if (e == cudaSuccess) e = opt_in<128, I8, true>();
  if (e == cudaSuccess) e = opt_in<64, I8, true, true>();
  if (e == cudaSuccess) e = opt_in<128, I8, true, true>();
  return e;
}

}  // namespace

#ifdef TKS_TILES_BF16
cudaError_t setup_tiles_bf16() { return setup_held<false>(); }
cudaError_t launch_tiles_bf16(const Params& p, int head_dim, bool selected, int grid, cudaStream_t stream) {
  return launch_held<false>(p, head_dim, selected, grid, stream);
}
#else
cudaError_t setup_tiles() {
  const cudaError_t e = setup_held<true>();
  return e != cudaSuccess ? e : setup_tiles_bf16();
}
cudaError_t launch_tiles(const Params& p, int head_dim, bool i8, bool selected, int grid,
                         cudaStream_t stream) {
  return i8 ? launch_held<true>(p, head_dim, selected, grid, stream) : launch_tiles_bf16(p, head_dim, selected, grid, stream);
}
#endif

}  // namespace attn
}  // namespace tks
