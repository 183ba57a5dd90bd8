// Attention over a paged cache for few query rows of each key/value head: the
// decode step, small trees, and selected positions of small head groups.
//
// Mathematics.  For a row i and the keys j it attends to, with x_ij = q_i.k_j
// * scale * log2(e):
//     out_i = sum_j 2^(x_ij - m) v_j / sum_j 2^(x_ij - m),   m near the running
// maximum; all sums in 32 bits.  Of a cache in 8 bits, k_j = ks_j * a_j and
// v_j = vs_j * b_j with integer codes a, b; then
//     w_ij = 2^(q_i.a_j * ks_j * scale * log2(e) + log2(vs_j) - m'),
//     out_i = sum_j w_ij b_j / sum_j w_ij / vs_j,
// so the codes go into the matrix products as they are, exact in half
// precision, one multiply-add applies both scales to a score, and a weight is
// rounded to 11 bits of itself (a small one in steps of 2^-31 of the largest,
// which is the largest contribution to the output: kWeightLog2). That is an
// eighth of what the output's own rounding to bfloat16 may be; a second part of
// it would cost as many products of values again.
// Queries are bfloat16; they enter as halves, each row shifted by a power of
// two of its own that brings its largest element to [2^14, 2^15): exactly, but
// for elements more than 2^31 below that one.  (One shift for all 16 rows let a
// large one, or a padded row's contents, take the others' bits away.)  Over a
// bfloat16 cache, whose products want bfloat16 weights, a weight goes in as the
// sum of two (rounded to one, weights made outputs 1.4 times less exact).
//
// What bounds it: the cache's bytes, each read once.  One matrix instruction
// works on 16 rows, so up to 16 rows of a head cost the same; 16 keys of int8
// (4 KB) take 32 of them, a third of their rate at the memory's pace.
// Measured: one token over 1,048,576 positions of int8 (4 heads of 128, 1.11 GB)
// 179-195 us, 5.7-6.2 TB/s, of bfloat16 354 us, 6.1 TB/s; 8 ragged trees of 4
// drafts over up to 65,536 positions of int8 (16 rows a head, 0.6 GB) 122 us, 4.9
// TB/s; one token over 4096 (8 heads, 8.7 MB) 11.6 us, bound by the chain of
// lookups, copies and joins that a lone call cannot hide.
//
// Layout.  A block is four warps; each takes every fourth chunk of the block's
// segment (32 keys of int8, 16 of bfloat16: 8 KB), keeps its own maximum, sum and
// output in registers and its own ring of cp.async stages in shared memory, so
// warps meet only at a segment's end.  Where the keys lie is looked up (list, page
// table) for 1024 of them at once, the block's threads side by side, before their
// copies start (one chunk ahead, it bound a gather of rows: 64 tokens over 2048
// selected positions of bfloat16 took 35.0 us so, and 30.6 now, 4.4 TB/s); chunks
// that lie in one page each take one lookup, a chunk ahead (1M positions: 194 us so,
// 220 with the lookups of the others).  The order of the 16-wide k index inside
// a product is free as long as both operands agree, so a lane takes whole
// 16-byte pieces of its key's row for the first product and of its four
// value rows for the second; bytes are paired by byte permutes, and the rows'
// pieces are XOR-swizzled so that neither read has bank conflicts.

#include "tks_attn.cuh"

namespace tks {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int D, bool I8>
struct Shape {
  static constexpr int kElem = I8 ? 1 : 2;
  static constexpr int kRow = D * kElem;               // bytes of a row
  static constexpr int kPieces = kRow / 16;            // 16-byte pieces of a row
  static constexpr int kE = 16 / kElem;                // elements of a piece
  static constexpr int kKH = kPieces / 4;              // pieces a lane takes of a key
  static constexpr int kEV = (I8 && D == 64) ? 8 : kE; // elements a lane takes of a value at once
  static constexpr int kVH = D / (8 * kEV);            // how often
  static constexpr int kChunk = I8 ? 32 : 16;          // keys of a stage
  static constexpr int kOps = 2 * kChunk * kRow;       // keys, then values
  static constexpr int kScales = I8 ? kChunk * 8 : 0;
  static constexpr int kStage = kOps + kScales + 16;   // and the mask of valid keys
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr int kQs = D / 16 * 32 * 16;         // query fragments, behind the rings
  static constexpr int kConst = I8 ? kWarps * 32 * 16 : 0;  // and each warp's scales as they are used
  static constexpr int kRings = kWarps * kStages * kStage;
  static constexpr int kSlots = 1024 * 4;              // and where keys lie
  static constexpr int kSmem = kRings + kQs + kConst + kSlots;
  static_assert(kRings >= (kWarps + 1) * (16 * D * 4 + 16 * 8), "the merge fits the ring");
  // Piece swizzles: the eight lanes of a phase read pieces c..c+3 of rows n
  // and n+1 (keys), or pieces n, n+1 of rows 0, 2, 4, 6 (values).
  static __device__ __forceinline__ int ksw(int r) { return kPieces >= 8 ? (r & 1) << 2 : 0; }
  static __device__ __forceinline__ int vsw(int r) {
    return kPieces >= 8 ? ((r >> 1) & 3) << 1 : ((r >> 1) & 1) << 1;
  }
};

template <bool HALF>
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// The largest finite magnitude among two bfloat16 values and m.
__device__ __forceinline__ float finite_max(float m, uint32_t w) {
  const float2 f = bf16_pair(w);
  const float a = fabsf(f.x), b = fabsf(f.y);
  m = a < INFINITY ? fmaxf(m, a) : m;
  return b < INFINITY ? fmaxf(m, b) : m;
}
// Clears infinities and NaNs of two bfloat16 values; says whether there were any.
__device__ __forceinline__ bool clear_nonfinite(uint32_t& w) {
  const bool lo = (w & 0x7f80u) == 0x7f80u, hi = (w & 0x7f800000u) == 0x7f800000u;
  if (lo) w &= 0xffff0000u;
  if (hi) w &= 0x0000ffffu;
  return lo || hi;
}

// PAGED: every chunk lies in one page (positions in order, pages of at least a chunk).
template <int D, bool I8, bool SEL, bool PAGED>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, I8>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Start start;
  __shared__ float2 ml_s[kWarps + 1][16];  // maxima and sums: the warps', and those of a run's pieces before
  __shared__ float top_s[kWarps][16];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = lane >> 2, c = lane & 3;  // the lane's key, row or column, and its quarter
  constexpr int kChunk = S::kChunk, kNT = kChunk / 8;  // key columns of a chunk, in eights
  unsigned char* ring = smem + warp * S::kStages * S::kStage;
  uint4* qs = reinterpret_cast<uint4*>(smem + S::kRings);
  float4* consts = reinterpret_cast<float4*>(smem + S::kRings + S::kQs) + warp * 32;
  int* slots = reinterpret_cast<int*>(smem + S::kRings + S::kQs + S::kConst);
  constexpr int kSlots = S::kSlots / 4;
  // the lane's piece of a row, its first row, and where that goes in a stage
  constexpr int kPer = 32 / S::kPieces;  // rows that 32 lanes cover
  const int piece = lane % S::kPieces, row0 = lane / S::kPieces;
  const uint32_t k_dst = smem_addr(ring) + row0 * S::kRow + ((piece ^ S::ksw(row0)) << 4);
  const uint32_t v_dst = smem_addr(ring) + (kChunk + row0) * S::kRow;
  const int v_piece = piece ^ S::vsw(row0);  // (the swizzles of row0 and of i * kPer combine by XOR)

  grid_wait();
  grid_launch_dependents();
  if (warp == 0) find_start<SEL, kRowsKeys>(p, &start);
  __syncthreads();
  // clusters: this block's partial, behind the warps' outputs
  float* part_s = reinterpret_cast<float*>(smem) + kWarps * 16 * D;
  float2* part_ml = reinterpret_cast<float2*>(part_s + 16 * D);
  Segments<SEL, kRowsKeys> segments;
  segments.begin(start);
  Segment sg;

  while (segments.next(p, sg)) {
    // ---- the segment ------------------------------------------------------
    const Seq len = sg.len;
    const int seq = sg.seq, head = sg.head, row_tile = sg.row_tile, b = sg.b, t0 = sg.t0, t1 = sg.t1;
    const int k_beg = t0 * kRowsKeys;  // tiles * kRowsKeys stays below 2^31: len does, rounded up once
    const int k_end = (int)min((long long)len.len, (long long)t1 * kRowsKeys);
    const int32_t* table = p.table + b * p.table_stride;
    const int32_t* list = SEL ? p.indices + (long long)seq * p.k_sel : nullptr;
    const int given = SEL ? kv_given(p, b) : 0;
    const unsigned char* kb = p.k + head * p.head_b;
    const unsigned char* vb = p.v + head * p.head_b;

    // Query fragments: rows n and n + 8; for product step (h, j) of a lane, elements
    // kE * (c + 4h) + 4j + {0,1} and {2,3}. All warps have the same rows, and each brings every
    // fourth step.
    constexpr int kMySteps = D / 16 / kWarps;
    const int rows_left = p.rows - row_tile * kRowsTile;
    const float fac = p.scale_log2;
    float back0 = 1.f, back1 = 1.f;  // 8 bits: what undoes the shifts of rows n and n + 8
    uint2 qa[kMySteps], qe[kMySteps];
    {
      const bool in0 = n < rows_left, in1 = n + 8 < rows_left;
      const __nv_bfloat16* q0 = q_row<SEL>(p, seq, head, row_tile * kRowsTile + (in0 ? n : 0));
      const __nv_bfloat16* q1 = q_row<SEL>(p, seq, head, row_tile * kRowsTile + (in1 ? n + 8 : 0));
#pragma unroll
      for (int i = 0; i < kMySteps; ++i) {
        const int s = warp + i * kWarps, d = S::kE * (c + 4 * (s / (S::kE / 4))) + 4 * (s % (S::kE / 4));
        qa[i] = in0 ? __ldg(reinterpret_cast<const uint2*>(q0 + d)) : make_uint2(0u, 0u);
        qe[i] = in1 ? __ldg(reinterpret_cast<const uint2*>(q1 + d)) : make_uint2(0u, 0u);
      }
    }

    // The page of the warp's chunk that starts at key j.
    auto page = [&](int j) -> int { return PAGED && j < k_end ? table[j >> p.page_shift] : -1; };
    // Starts the copies of the chunk at key j into stage `st`; pg: its page; beg: the key of slots[0].
    auto issue = [&](int j, int st, int pg, int beg, int end) {
      if (j < end) {
        const uint32_t to = st * S::kStage;
        unsigned valid;
        if (PAGED) {
          const bool ok = (unsigned)pg < (unsigned)p.pages;
          if (!ok) report(p.status, kStatIndexBit);
          const int n_valid = ok ? min(kChunk, end - j) : 0, in_page = j & ((1 << p.page_shift) - 1);
          const long long off = ok ? pg * p.page_b + in_page * p.token_b : 0;
          const unsigned char* ks = kb + off + row0 * p.token_b + piece * 16;
          const unsigned char* vs = vb + off + row0 * p.token_b + piece * 16;
          const long long step = kPer * p.token_b;
#pragma unroll
          for (int i = 0; i < kChunk / kPer; ++i) {
            const int bytes = row0 + i * kPer < n_valid ? 16 : 0;
            cp16(k_dst + to + i * kPer * S::kRow, ks, bytes);
            cp16(v_dst + to + i * kPer * S::kRow + ((v_piece ^ S::vsw(i * kPer)) << 4), vs, bytes);
            ks += step;
            vs += step;
          }
          if (I8) {
            const long long row = ok ? (((long long)pg << p.page_shift) + in_page) * p.kv_heads + head : 0;
            cp8(smem_addr(ring) + to + S::kOps + lane * 8, p.scales + row + (lane < n_valid ? (long long)lane * p.kv_heads : 0), lane < n_valid ? 8 : 0);
          }
          valid = n_valid >= 32 ? ~0u : (1u << n_valid) - 1u;
        } else {
          const int* sl = slots + (j - beg);
          const int mine = lane < kChunk ? sl[lane] : -1;
          // all offsets before the first copy: the copies are not to be moved across
          long long at[kChunk / kPer];
#pragma unroll
          for (int i = 0; i < kChunk / kPer; ++i) {
            const int slot = sl[row0 + i * kPer];
            at[i] = slot < 0 ? -1 : (slot >> p.page_shift) * p.page_b + (slot & ((1 << p.page_shift) - 1)) * p.token_b + piece * 16;
          }
#pragma unroll
          for (int i = 0; i < kChunk / kPer; ++i) {
            const int bytes = at[i] >= 0 ? 16 : 0;
            const long long o = at[i] >= 0 ? at[i] : 0;
            cp16(k_dst + to + i * kPer * S::kRow, kb + o, bytes);
            cp16(v_dst + to + i * kPer * S::kRow + ((v_piece ^ S::vsw(i * kPer)) << 4), vb + o, bytes);
          }
          if (I8)
            cp8(smem_addr(ring) + to + S::kOps + lane * 8, p.scales + (mine >= 0 ? (long long)mine * p.kv_heads + head : 0), mine >= 0 ? 8 : 0);
          valid = __ballot_sync(0xffffffffu, mine >= 0);
        }
        if (lane == 0) *reinterpret_cast<unsigned*>(ring + to + S::kOps + S::kScales) = valid;
      }
      cp_commit();
    };
    constexpr int kAhead = S::kStages - 1, kStep = kWarps * kChunk;

    auto put_queries = [&] {
      float up0 = 1.f, up1 = 1.f;
      if (I8) {
        float a = 0.f, b = 0.f;  // the rows' largest finite magnitudes: this lane's, the warp's, the block's
#pragma unroll
        for (int i = 0; i < kMySteps; ++i) {
          a = finite_max(finite_max(a, qa[i].x), qa[i].y);
          b = finite_max(finite_max(b, qe[i].x), qe[i].y);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        if (c == 0) {
          top_s[warp][n] = a;
          top_s[warp][n + 8] = b;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          a = fmaxf(a, top_s[i][n]);
          b = fmaxf(b, top_s[i][n + 8]);
        }
        const int s0 = a > 0.f ? max(-120, min(120, 14 - ilogbf(a))) : 0, s1 = b > 0.f ? max(-120, min(120, 14 - ilogbf(b))) : 0;
        up0 = __int_as_float((s0 + 127) << 23);
        up1 = __int_as_float((s1 + 127) << 23);
        back0 = __int_as_float((127 - s0) << 23);
        back1 = __int_as_float((127 - s1) << 23);
      }
      auto held = [&](uint32_t w, float up) -> uint32_t {
        const float2 f = bf16_pair(w);
        return I8 ? pack_half(f.x * up, f.y * up) : w;
      };
#pragma unroll
      for (int i = 0; i < kMySteps; ++i)
        qs[(warp + i * kWarps) * 32 + lane] = make_uint4(held(qa[i].x, up0), held(qe[i].x, up1), held(qa[i].y, up0), held(qe[i].y, up1));
      __syncthreads();
    };

    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][r] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool poisoned = false;  // a draft's value held an infinity or NaN (bfloat16)

    // ---- the warp's chunks: of the whole segment, or of the keys looked up at once ----
    for (int beg = k_beg; beg < k_end; beg += PAGED ? k_end - k_beg : kSlots) {
    const int end = PAGED ? k_end : (int)min((long long)k_end, (long long)beg + kSlots);
    if (!PAGED) {
      // all list entries, then all pages: two waits, not one for each key
      constexpr int kMine = kSlots / kThreads;
      int pos[kMine], pg[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int j = beg + threadIdx.x + i * kThreads;
        pos[i] = j >= end ? -1 : SEL ? __ldg(list + j) : j;
      }
      bool bad = false;
      const int limit = SEL ? kv_limit(p, given) : 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        bad |= SEL && pos[i] >= limit;
        if (SEL && pos[i] >= limit) pos[i] = -1;
        pg[i] = pos[i] < 0 ? -1 : __ldg(table + (pos[i] >> p.page_shift));
      }
      __syncthreads();  // the previous keys' copies have started
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const bool ok = pos[i] >= 0 && (unsigned)pg[i] < (unsigned)p.pages;
        bad |= pos[i] >= 0 && !ok;
        slots[threadIdx.x + i * kThreads] = ok ? (int)(((unsigned)pg[i] << p.page_shift) + (pos[i] & ((1 << p.page_shift) - 1))) : -1;
      }
      if (bad) report(p.status, kStatIndexBit);
      __syncthreads();
    }
    // the first chunks' pages, a lane each (loops that run once or twice are not unrolled: a block
    // runs most of this code once, and fetches its instructions first)
    const int pgs = lane <= kAhead ? page(beg + warp * kChunk + lane * kStep) : -1;
    int pg_n = __shfl_sync(0xffffffffu, pgs, kAhead);
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i)
      issue(beg + warp * kChunk + i * kStep, i, __shfl_sync(0xffffffffu, pgs, i), beg, end);
    if (beg == k_beg) put_queries();
    int stage = 0, ahead = kAhead;  // of this chunk, and of the one whose copies start
    for (int j0 = beg + warp * kChunk; j0 < end; j0 += kStep) {  // (j0 + (kAhead + 1) * kStep stays below 2^31: kMaxPositions)
      cp_wait<kAhead - 1>();
      __syncwarp();
      // the next copies go into the stage that the previous chunk has left
      issue(j0 + kAhead * kStep, ahead, pg_n, beg, end);
      pg_n = page(j0 + (kAhead + 1) * kStep);
      const unsigned char* st = ring + stage * S::kStage;
      ahead = stage;
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
      const unsigned valid = *reinterpret_cast<const unsigned*>(st + S::kOps + S::kScales);
      if (I8) {  // the scales of key `lane` as they are used: a factor, a summand, and the sum's factor
        const float2 sc = *reinterpret_cast<const float2*>(st + S::kOps + lane * 8);
        const float lo = 7.105427357601002e-15f;  // 2^-47: a NaN stays one
        const float x = sc.y < lo ? lo : sc.y;
        // (the last is finite: a weight of 0 times it is 0)
        consts[lane] = make_float4(sc.x * fac, lg2(x), x == x ? __fdividef(1.f, x) : 1.f, 0.f);
      }

      float s[kNT][4];
#pragma unroll
      for (int t = 0; t < kNT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int h = 0; h < S::kKH; ++h) {
        uint4 kw[kNT];
#pragma unroll
        for (int t = 0; t < kNT; ++t)
          kw[t] = *reinterpret_cast<const uint4*>(st + (n + 8 * t) * S::kRow + (((c + 4 * h) ^ S::ksw(n)) << 4));
        if (I8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 q = qs[(h * 4 + j) * 32 + lane];
#pragma unroll
            for (int t = 0; t < kNT; ++t) {
              const uint32_t a = (j == 0 ? kw[t].x : j == 1 ? kw[t].y : j == 2 ? kw[t].z : kw[t].w) ^ 0x80808080u;
              mma<true>(s[t], q, codes_to_half2<0x4140>(a), codes_to_half2<0x4342>(a));
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 q = qs[(h * 2 + j) * 32 + lane];
#pragma unroll
            for (int t = 0; t < kNT; ++t) mma<false>(s[t], q, j ? kw[t].z : kw[t].x, j ? kw[t].w : kw[t].y);
          }
        }
      }

      // Scores: rows n (s[.][0..1]) and n + 8 (s[.][2..3]), keys 8t + 2c and the next.
      float inv[2 * kNT];
      if (I8) {
        __syncwarp();
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 k = consts[8 * t + 2 * c + e];
            s[t][e] = fmaf(s[t][e] * back0, k.x, k.y);
            s[t][2 + e] = fmaf(s[t][2 + e] * back1, k.x, k.y);
            inv[2 * t + e] = k.z;
          }
      } else {
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] *= fac;
      }
      const bool drafts = !SEL && j0 + kChunk > len.ctx;
      if (valid != (kChunk == 32 ? ~0u : 0xffffu) || drafts) {
        unsigned seen0 = valid, seen1 = valid;  // the keys that rows n and n + 8 see
        if (drafts) {
          const int R = row_tile * kRowsTile + n;
          seen0 &= draft_bits(p, b, min(R / p.group, p.tokens - 1), j0 - len.ctx);
          seen1 &= draft_bits(p, b, min((R + 8) / p.group, p.tokens - 1), j0 - len.ctx);
        }
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!(seen0 >> (8 * t + 2 * c + e) & 1u)) s[t][e] = -INFINITY;
            if (!(seen1 >> (8 * t + 2 * c + e) & 1u)) s[t][2 + e] = -INFINITY;
          }
      }

      // What weights are relative to (kWeightLog2) follows when a maximum has grown by more than 2^8: by
      // its difference, which weights are powers of. (Where 32 bits go in steps of 16, m + 8 can be m + 16.)
      float t0m = fmaxf(s[0][0], s[0][1]), t1m = fmaxf(s[0][2], s[0][3]);
#pragma unroll
      for (int t = 1; t < kNT; ++t) {
        t0m = fmaxf(t0m, fmaxf(s[t][0], s[t][1]));
        t1m = fmaxf(t1m, fmaxf(s[t][2], s[t][3]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        t0m = fmaxf(t0m, __shfl_xor_sync(0xffffffffu, t0m, o));
        t1m = fmaxf(t1m, __shfl_xor_sync(0xffffffffu, t1m, o));
      }
      constexpr float kAbove = kWeightLog2<I8>;
      const bool up0 = t0m - m[0] > 8.f + kAbove, up1 = t1m - m[1] > 8.f + kAbove;  // (both -inf: no)
      if (__any_sync(0xffffffffu, up0 || up1)) {
        t0m -= kAbove;
        t1m -= kAbove;
        const float f0 = up0 ? ex2(m[0] - t0m) : 1.f, f1 = up1 ? ex2(m[1] - t1m) : 1.f;
        if (up0) m[0] = t0m;
        if (up1) m[1] = t1m;
        l[0] *= f0; l[1] *= f1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          acc[i][0] *= f0; acc[i][1] *= f0;
          acc[i][2] *= f1; acc[i][3] *= f1;
        }
      }
      const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
      for (int t = 0; t < kNT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = ex2(s[t][e] - u0), d = ex2(s[t][2 + e] - u1);
          s[t][e] = a;
          s[t][2 + e] = d;
          l[0] = I8 ? fmaf(a, inv[2 * t + e], l[0]) : l[0] + a;
          l[1] = I8 ? fmaf(d, inv[2 * t + e], l[1]) : l[1] + d;
        }

      // Values, 16 keys at a time: keys 2c, 2c+1 (b0) and those + 8 (b1), element kEV * (n + 8h) + j in tile (h, j).
      const unsigned char* vst = st + kChunk * S::kRow;
#pragma unroll
      for (int g = 0; g < kNT / 2; ++g) {
        const float(&sa)[4] = s[2 * g];
        const float(&sb)[4] = s[2 * g + 1];
        uint4 pf, rest;
        if (I8) {
          pf = make_uint4(pack_half(sa[0], sa[1]), pack_half(sa[2], sa[3]), pack_half(sb[0], sb[1]), pack_half(sb[2], sb[3]));
        } else {
          split_bf16(sa[0], sa[1], pf.x, rest.x);
          split_bf16(sa[2], sa[3], pf.y, rest.y);
          split_bf16(sb[0], sb[1], pf.z, rest.z);
          split_bf16(sb[2], sb[3], pf.w, rest.w);
        }
#pragma unroll
        for (int h = 0; h < S::kVH; ++h) {
          constexpr int kW = S::kEV * S::kElem / 4;
          uint32_t vw[4][kW];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 16 * g + 2 * c + (e & 1) + 8 * (e >> 1);
            if (kW == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(vst + r * S::kRow + (((n + 8 * h) ^ S::vsw(r)) << 4));
              vw[e][0] = x.x; vw[e][1] = x.y; vw[e][2 % kW] = x.z; vw[e][3 % kW] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(vst + r * S::kRow + (((n >> 1) ^ S::vsw(r)) << 4) + (n & 1) * 8);
              vw[e][0] = x.x; vw[e][1] = x.y;
            }
          }
          if (!I8 && drafts) {
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j0 + 16 * g + 2 * c + (e & 1) + 8 * (e >> 1) >= len.ctx)
#pragma unroll
                for (int x = 0; x < kW; ++x) bad |= clear_nonfinite(vw[e][x]);
            poisoned |= __any_sync(0xffffffffu, bad);
          }
#pragma unroll
          for (int x = 0; x < kW; ++x) {
            if (I8) {
              const uint32_t a0 = vw[0][x] ^ 0x80808080u, a1 = vw[1][x] ^ 0x80808080u;
              const uint32_t a2 = vw[2][x] ^ 0x80808080u, a3 = vw[3][x] ^ 0x80808080u;
              const uint32_t lo0 = __byte_perm(a0, a1, 0x5140), hi0 = __byte_perm(a0, a1, 0x7362);
              const uint32_t lo1 = __byte_perm(a2, a3, 0x5140), hi1 = __byte_perm(a2, a3, 0x7362);
              const int i = h * S::kEV + 4 * x;
              mma<true>(acc[i], pf, codes_to_half2<0x4140>(lo0), codes_to_half2<0x4140>(lo1));
              mma<true>(acc[i + 1], pf, codes_to_half2<0x4342>(lo0), codes_to_half2<0x4342>(lo1));
              mma<true>(acc[i + 2], pf, codes_to_half2<0x4140>(hi0), codes_to_half2<0x4140>(hi1));
              mma<true>(acc[i + 3], pf, codes_to_half2<0x4342>(hi0), codes_to_half2<0x4342>(hi1));
            } else {
              const int i = h * S::kEV + 2 * x;
              const uint32_t a0 = __byte_perm(vw[0][x], vw[1][x], 0x5410), a1 = __byte_perm(vw[2][x], vw[3][x], 0x5410);
              const uint32_t b0 = __byte_perm(vw[0][x], vw[1][x], 0x7632), b1 = __byte_perm(vw[2][x], vw[3][x], 0x7632);
              mma<false>(acc[i], pf, a0, a1);
              mma<false>(acc[i + 1], pf, b0, b1);
              mma<false>(acc[i], rest, a0, a1);
              mma<false>(acc[i + 1], rest, b0, b1);
            }
          }
        }
      }
      __syncwarp();  // all lanes have read the stage before it is filled again
    }
    cp_wait<0>();
    }

    // Infinities and NaNs of drafted tokens' values reach only the rows that
    // attend to them (rare: the product above took them as zeros).
    if (!I8 && !SEL && poisoned) {
      for (int j0 = k_beg + warp * kChunk; j0 < k_end; j0 += kStep) {
        for (int j = max(j0, len.ctx); j < min(j0 + kChunk, k_end); ++j) {
          const int pg = table[j >> p.page_shift];
          if ((unsigned)pg >= (unsigned)p.pages) continue;
          const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(
              vb + pg * p.page_b + (j & ((1 << p.page_shift) - 1)) * p.token_b);
          const int R = row_tile * kRowsTile + n;
          const bool a0 = sees_draft(p, b, min(R / p.group, p.tokens - 1), j - len.ctx);
          const bool a1 = sees_draft(p, b, min((R + 8) / p.group, p.tokens - 1), j - len.ctx);
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = __bfloat162float(v[S::kEV * (2 * c + e + 8 * (i / S::kEV)) + i % S::kEV]);
              if (!(fabsf(x) < INFINITY)) {
                if (a0) acc[i][e] += x;
                if (a1) acc[i][2 + e] += x;
              }
            }
        }
      }
    }

    // ---- join the four warps ----------------------------------------------
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    __syncthreads();  // every warp's ring is done with
    float* om = reinterpret_cast<float*>(smem) + warp * 16 * D;
#pragma unroll
    for (int h = 0; h < S::kVH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < S::kEV; j += 4) {
          const int d = S::kEV * (2 * c + e + 8 * h) + j, i = h * S::kEV + j;
          *reinterpret_cast<float4*>(om + n * D + d) = make_float4(acc[i][e], acc[i + 1][e], acc[i + 2][e], acc[i + 3][e]);
          *reinterpret_cast<float4*>(om + (n + 8) * D + d) = make_float4(acc[i][2 + e], acc[i + 1][2 + e], acc[i + 2][2 + e], acc[i + 3][2 + e]);
        }
    if (c == 0) {
      ml_s[warp][n] = make_float2(m[0], l[0]);
      ml_s[warp][n + 8] = make_float2(m[1], l[1]);
    }
    __syncthreads();
    const bool whole = sg.whole() && !p.cluster;
    float* part = p.cluster ? part_s : p.parts + (2LL * blockIdx.x + (sg.first ? 0 : 1)) * kPartFloats<kRowsTile, D>;
    const float* om0 = reinterpret_cast<const float*>(smem);
#pragma unroll 1
    for (int x = threadIdx.x; x < min(rows_left, 16) * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4, R = row_tile * kRowsTile + r;
      float2 q[kWarps];
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        q[i] = ml_s[i][r];
        mm = fmaxf(mm, q[i].x);
      }
      float2 qb = make_float2(-INFINITY, 0.f);  // the run's pieces before
      if (sg.goes_on()) qb = ml_s[kWarps][r];
      mm = fmaxf(mm, qb.x);
      const bool active = SEL || R / p.group < len.drafts;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kWarps; ++i)
        if (active && q[i].y != 0.f) {  // (a warp whose keys are all unseen has a sum of zero)
          const float f = q[i].x == mm ? 1.f : ex2(q[i].x - mm);
          const float4 a = *reinterpret_cast<const float4*>(om0 + (i * 16 + r) * D + d);
          ll += f * q[i].y;
          o.x += f * a.x; o.y += f * a.y; o.z += f * a.z; o.w += f * a.w;
        }
      if (active && qb.y != 0.f) {  // (this thread has put them there)
        const float f = qb.x == mm ? 1.f : ex2(qb.x - mm);
        const float4 a = *reinterpret_cast<const float4*>(part + r * D + d);
        ll += f * qb.y;
        o.x += f * a.x; o.y += f * a.y; o.z += f * a.z; o.w += f * a.w;
      }
      if (whole) {
        const float g = ll == 0.f ? 0.f : 1.f / ll;
        const long long row = out_row<SEL>(p, seq, head, R);
        *reinterpret_cast<uint2*>(p.out + row * D + d) = make_uint2(pack_bf16(o.x * g, o.y * g), pack_bf16(o.z * g, o.w * g));
        if (p.lse && d == 0) p.lse[row] = ll == 0.f ? -INFINITY : (mm + lg2(ll)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(part + 16 * D + 2 * r) = make_float2(mm, ll);
      }
    }
    __syncthreads();  // the ring is free for the next segment
    if (sg.more && threadIdx.x < 16) {  // (read behind the next piece's barriers)
      const int r = threadIdx.x;
      float2 all = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i <= kWarps; ++i)
        if (i < kWarps || sg.goes_on()) all.x = fmaxf(all.x, ml_s[i][r].x);
#pragma unroll
      for (int i = 0; i <= kWarps; ++i) {
        if (i == kWarps && !sg.goes_on()) continue;
        const float2 q = ml_s[i][r];
        if (q.y != 0.f) all.y += (q.x == all.x ? 1.f : ex2(q.x - all.x)) * q.y;
      }
      ml_s[kWarps][r] = all;
    }
  }
  if (p.cluster) {
    if (start.left == 0 && threadIdx.x < 16) part_ml[threadIdx.x] = make_float2(-INFINITY, 0.f);
    join_cluster<kRowsTile, D, SEL>(p, smem_addr(part_s), smem_addr(part_ml), kThreads);
  }
}

template <int D, bool I8, bool SEL, bool PAGED>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<D, I8>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute a[2] = {};
  cfg.attrs = a;
  cfg.numAttrs = launch_attributes(a, p.cluster);
  return cudaLaunchKernelEx(&cfg, rows_kernel<D, I8, SEL, PAGED>, p);
}
template <int D, bool I8>
cudaError_t launch(const Params& p, bool selected, int grid, cudaStream_t stream) {
  if (selected) return launch<D, I8, true, false>(p, grid, stream);
  return (1 << p.page_shift) >= Shape<D, I8>::kChunk ? launch<D, I8, false, true>(p, grid, stream)
                                                     : launch<D, I8, false, false>(p, grid, stream);
}

template <int D, bool I8>
cudaError_t opt_in() {
  cudaError_t e = allow(rows_kernel<D, I8, true, false>, Shape<D, I8>::kSmem);
  if (e == cudaSuccess) e = allow(rows_kernel<D, I8, false, true>, Shape<D, I8>::kSmem);
  if (e == cudaSuccess) e = allow(rows_kernel<D, I8, false, false>, Shape<D, I8>::kSmem);
  return e;
}

}  // namespace

cudaError_t setup_rows() {
  cudaError_t e = opt_in<64, false>();
  if (e == cudaSuccess) e = opt_in<64, true>();
  if (e == cudaSuccess) e = opt_in<128, false>();
  if (e == cudaSuccess) e = opt_in<128, true>();
  return e;
}

cudaError_t launch_rows(const Params& p, int head_dim, bool i8, bool selected, int grid,
                        cudaStream_t stream) {
  if (head_dim == 64) return i8 ? launch<64, true>(p, selected, grid, stream) : launch<64, false>(p, selected, grid, stream);
  return i8 ? launch<128, true>(p, selected, grid, stream) : launch<128, false>(p, selected, grid, stream);
}

}  // namespace attn
}  // namespace tks
