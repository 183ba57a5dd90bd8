// Attention over a paged cache for few query rows of each key/value head: the
// decode step, small trees, and selected positions of small head groups.
//
// Mathematics.  For a row i and the keys j it attends to, with x_ij = q_i.k_j
// * scale * log2(e):
//     out_i = sum_j 2^(x_ij - m) v_j / sum_j 2^(x_ij - m),   m the running
// maximum; all sums in 32 bits.  Of a cache in 8 bits, k_j = ks_j * a_j and
// v_j = vs_j * b_j with integer codes a, b; then
//     w_ij = 2^(q_i.a_j * ks_j * scale * log2(e) + log2(vs_j) - m'),
//     out_i = sum_j w_ij b_j / sum_j w_ij / vs_j,
// so the codes go into the matrix products as they are, exact in half
// precision, one multiply-add applies both scales to a score, and the weights
// are rounded (to 11 bits) relative to the largest contribution to the output.
// Queries are bfloat16; they enter as halves, exactly, after a shift by a
// power of two that is common to the block's rows.  Over a bfloat16 cache the
// weights are rounded to bfloat16 (the products want one type).
//
// What bounds it: the cache's bytes, each read once.  One matrix instruction
// works on 16 rows, so up to 16 rows of a head cost the same; 16 keys of int8
// (4 KB) take 32 of them, a third of their rate at the memory's pace.
//
// Layout.  A block is four warps; each takes every fourth chunk of 16 keys of
// the block's segment, keeps its own maximum, sum and output in registers and
// its own ring of cp.async stages in shared memory, so warps meet only at a
// segment's end.  Key positions are looked up (list, page table) one and two
// chunks ahead of their copies.  The order of the 16-wide k index inside a
// product is free as long as both operands agree, so a lane takes whole
// 16-byte pieces of its key's row for the first product and of its four
// value rows for the second; bytes are paired by byte permutes, and the rows'
// pieces are XOR-swizzled so that neither read has bank conflicts.

#include "tks_attn.cuh"

namespace tks {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 16;  // keys of a stage

template <int D, bool I8>
struct Shape {
  static constexpr int kElem = I8 ? 1 : 2;
  static constexpr int kRow = D * kElem;               // bytes of a row
  static constexpr int kPieces = kRow / 16;            // 16-byte pieces of a row
  static constexpr int kE = 16 / kElem;                // elements of a piece
  static constexpr int kKH = kPieces / 4;              // pieces a lane takes of a key
  static constexpr int kEV = (I8 && D == 64) ? 8 : kE; // elements a lane takes of a value at once
  static constexpr int kVH = D / (8 * kEV);            // how often
  static constexpr int kOps = 2 * kChunk * kRow;       // keys, then values
  static constexpr int kScales = I8 ? kChunk * 8 : 0;
  static constexpr int kStage = kOps + kScales + 16;   // and the mask of valid keys
  static constexpr int kStages = I8 ? (D == 128 ? 5 : 6) : (D == 128 ? 3 : 5);
  static constexpr int kSmem = kWarps * kStages * kStage;
  static_assert(kSmem >= kWarps * (16 * D * 4 + 16 * 8), "the merge fits the ring");
  // Piece swizzles: the eight lanes of a phase read pieces c..c+3 of rows n
  // and n+1 (keys), or pieces n, n+1 of rows 0, 2, 4, 6 (values).
  static __device__ __forceinline__ int ksw(int r) { return kPieces >= 8 ? (r & 1) << 2 : 0; }
  static __device__ __forceinline__ int vsw(int r) {
    return kPieces >= 8 ? ((r >> 1) & 3) << 1 : ((r >> 1) & 1) << 1;
  }
};

template <bool HALF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <int D, bool I8, bool SEL>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, I8>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Start start;
  __shared__ float2 ml_s[kWarps][16];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = lane >> 2, c = lane & 3;  // the lane's key, row or column, and its quarter
  unsigned char* ring = smem + warp * S::kStages * S::kStage;
  const uint32_t ring_a = smem_addr(ring);

  grid_wait();
  grid_launch_dependents();
  if (warp == 0) find_start<SEL, kRowsKeys>(p, &start);
  __syncthreads();
  Segments<SEL, kRowsKeys> segments;
  segments.begin(start);
  Segment sg;

  while (segments.next(p, sg)) {
    // ---- the segment ------------------------------------------------------
    const Seq len = sg.len;
    const int seq = sg.seq, head = sg.head, row_tile = sg.row_tile, b = sg.b, t0 = sg.t0, t1 = sg.t1;
    const int k_beg = t0 * kRowsKeys;  // tiles * kRowsKeys stays below 2^31: len does, rounded up once
    const int k_end = (int)min((long long)len.len, (long long)t1 * kRowsKeys);
    const int chunks = (k_end - k_beg + kChunk - 1) / kChunk;
    const int iters = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
    const int32_t* table = p.table + b * p.table_stride;
    const int32_t* list = SEL ? p.indices + (long long)seq * p.k_sel : nullptr;
    const int limit = SEL ? kv_limit(p, b) : 0;
    const unsigned char* kb = p.k + head * p.head_b;
    const unsigned char* vb = p.v + head * p.head_b;

    // Position of this lane's key (lane & 15) of the warp's chunk `it`, or -1.
    auto position = [&](int it) -> int {
      const long long j = (long long)k_beg + ((long long)it * kWarps + warp) * kChunk + (lane & 15);
      if (j >= k_end) return -1;
      if (!SEL) return (int)j;
      const int idx = list[j];
      if (idx >= limit) report(p.status, kStatIndexBit);
      return idx < limit ? idx : -1;
    };
    auto page = [&](int pos) -> int { return pos < 0 ? -1 : table[pos >> p.page_shift]; };
    // Starts the copies of chunk `it` into its stage, given its lane's position and page.
    auto issue = [&](int it, int pos, int pg) {
      if (it < iters) {
        const bool ok = pos >= 0 && (unsigned)pg < (unsigned)p.pages;
        if (pos >= 0 && !ok) report(p.status, kStatIndexBit);
        const int in_page = pos & ((1 << p.page_shift) - 1);
        const long long off = ok ? pg * p.page_b + in_page * p.token_b : -1;
        const unsigned valid = __ballot_sync(0xffffffffu, ok) & 0xffffu;
        unsigned char* st = ring + (it % S::kStages) * S::kStage;
        const uint32_t st_a = ring_a + (it % S::kStages) * S::kStage;
        constexpr int kPer = 32 / S::kPieces;  // rows that 32 lanes cover
        const int piece = lane % S::kPieces;
#pragma unroll
        for (int i = 0; i < kChunk / kPer; ++i) {
          const int r = lane / S::kPieces + i * kPer;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const int bytes = o >= 0 ? 16 : 0;
          const long long at = (o >= 0 ? o : 0) + piece * 16;
          cp16(st_a + r * S::kRow + ((piece ^ S::ksw(r)) << 4), kb + (bytes ? at : 0), bytes);
          cp16(st_a + kChunk * S::kRow + r * S::kRow + ((piece ^ S::vsw(r)) << 4), vb + (bytes ? at : 0), bytes);
        }
        if (I8 && lane < kChunk) {
          const long long row = ok ? ((long long)(((long long)pg << p.page_shift) + in_page) * p.kv_heads + head) : 0;
          cp8(st_a + S::kOps + lane * 8, p.scales + row, ok ? 8 : 0);
        }
        if (lane == 0) *reinterpret_cast<unsigned*>(st + S::kOps + S::kScales) = valid;
      }
      cp_commit();
    };

    // ---- first copies; then the queries, while they are under way -----------
    constexpr int kAhead = S::kStages - 1;
    int pos_n, pg_n, pos_nn = -1;
    {
      int ps[kAhead], pg[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ps[i] = position(i);
      pos_n = position(kAhead);
      if (SEL) pos_nn = position(kAhead + 1);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) pg[i] = page(ps[i]);
      pg_n = page(pos_n);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) issue(i, ps[i], pg[i]);
    }

    // Query fragments: rows n and n + 8; for product step (h, j) of a lane,
    // elements kE * (c + 4h) + 4j + {0,1} and {2,3}.
    uint32_t qf[D / 16][4];
    const int rows_left = p.rows - row_tile * kRowsTile;
    float fac = p.scale_log2;
    {
      const bool in0 = n < rows_left, in1 = n + 8 < rows_left;
      const __nv_bfloat16* q0 = q_row<SEL>(p, seq, head, row_tile * kRowsTile + (in0 ? n : 0));
      const __nv_bfloat16* q1 = q_row<SEL>(p, seq, head, row_tile * kRowsTile + (in1 ? n + 8 : 0));
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < S::kKH; ++h)
#pragma unroll
        for (int j = 0; j < S::kE / 4; ++j) {
          const int d = S::kE * (c + 4 * h) + 4 * j, s = h * (S::kE / 4) + j;
          const uint2 a = in0 ? *reinterpret_cast<const uint2*>(q0 + d) : make_uint2(0u, 0u);
          const uint2 e = in1 ? *reinterpret_cast<const uint2*>(q1 + d) : make_uint2(0u, 0u);
          qf[s][0] = a.x; qf[s][1] = e.x; qf[s][2] = a.y; qf[s][3] = e.y;
          if (I8)
            top = finite_max(finite_max(finite_max(finite_max(top, a.x), a.y), e.x), e.y);
        }
      if (I8) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // the largest finite magnitude goes to [2^14, 2^15): halves keep 11 bits
        // over 2^28 below it
        const int shift = top > 0.f ? max(-120, min(120, 14 - ilogbf(top))) : 0;
        const float up = __int_as_float((shift + 127) << 23);
        fac *= __int_as_float((127 - shift) << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 f = bf16_pair(qf[s][r]);
            qf[s][r] = pack_half(f.x * up, f.y * up);
          }
      }
    }

    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][r] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool poisoned = false;  // a draft's value held an infinity or NaN (bfloat16)

    // ---- the warp's chunks ------------------------------------------------
    for (int it = 0; it < iters; ++it) {
      cp_wait<kAhead - 1>();
      __syncwarp();
      {  // the next copies go into the stage that the previous chunk has left
        issue(it + kAhead, pos_n, pg_n);
        if (SEL) {
          pos_n = pos_nn;
          pg_n = page(pos_n);
          pos_nn = position(it + kAhead + 2);
        } else {
          pos_n = position(it + kAhead + 1);
          pg_n = page(pos_n);
        }
      }
      const unsigned char* st = ring + (it % S::kStages) * S::kStage;
      const unsigned valid = *reinterpret_cast<const unsigned*>(st + S::kOps + S::kScales);

      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int h = 0; h < S::kKH; ++h) {
        const int piece = ((c + 4 * h) ^ S::ksw(n)) << 4;
        uint4 ka = *reinterpret_cast<const uint4*>(st + n * S::kRow + piece);
        uint4 kc = *reinterpret_cast<const uint4*>(st + (n + 8) * S::kRow + piece);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
        if (I8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a = wa[j] ^ 0x80808080u, e = wc[j] ^ 0x80808080u;
            mma<true>(s[0], qf[h * 4 + j], codes_to_half2<0x4140>(a), codes_to_half2<0x4342>(a));
            mma<true>(s[1], qf[h * 4 + j], codes_to_half2<0x4140>(e), codes_to_half2<0x4342>(e));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma<false>(s[0], qf[h * 2 + j], wa[2 * j], wa[2 * j + 1]);
            mma<false>(s[1], qf[h * 2 + j], wc[2 * j], wc[2 * j + 1]);
          }
        }
      }

      // Scores: rows n (s[.][0..1]) and n + 8 (s[.][2..3]), keys 2c, 2c+1 and those + 8.
      float inv[4];
      if (I8) {
        const float4 s0 = *reinterpret_cast<const float4*>(st + S::kOps + 16 * c);
        const float4 s1 = *reinterpret_cast<const float4*>(st + S::kOps + 64 + 16 * c);
        const float ks[4] = {s0.x * fac, s0.z * fac, s1.x * fac, s1.z * fac};
        const float vs[4] = {s0.y, s0.w, s1.y, s1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = 7.105427357601002e-15f;  // 2^-47: a NaN stays one
          const float x = vs[e] < lo ? lo : vs[e], lv = lg2(x);
          inv[e] = __fdividef(1.f, x);
          s[e >> 1][e & 1] = fmaf(s[e >> 1][e & 1], ks[e], lv);
          s[e >> 1][2 + (e & 1)] = fmaf(s[e >> 1][2 + (e & 1)], ks[e], lv);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[e >> 1][e & 1] *= fac;
          s[e >> 1][2 + (e & 1)] *= fac;
        }
      }
      const int j0 = k_beg + (it * kWarps + warp) * kChunk;  // the chunk's first key
      unsigned seen0 = 15u, seen1 = 15u;                      // of this lane's four keys
      const bool drafts = !SEL && j0 + kChunk > len.ctx;
      if (valid != 0xffffu || drafts) {
        seen0 = ((valid >> (2 * c)) & 3u) | (((valid >> (2 * c + 8)) & 3u) << 2);
        seen1 = seen0;
        if (drafts) {
          const int R = row_tile * kRowsTile + n;
          const int ta = min(R / p.group, p.tokens - 1), tc = min((R + 8) / p.group, p.tokens - 1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + 2 * c + (e & 1) + 8 * (e >> 1) - len.ctx;
            if (j >= 0 && j < len.drafts) {
              if (!sees_draft(p, b, ta, j)) seen0 &= ~(1u << e);
              if (!sees_draft(p, b, tc, j)) seen1 &= ~(1u << e);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!((seen0 >> e) & 1u)) s[e >> 1][e & 1] = -INFINITY;
          if (!((seen1 >> e) & 1u)) s[e >> 1][2 + (e & 1)] = -INFINITY;
        }
      }

      // Running maximum; the output is rescaled only when one has grown.
      float t0m = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float t1m = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        t0m = fmaxf(t0m, __shfl_xor_sync(0xffffffffu, t0m, o));
        t1m = fmaxf(t1m, __shfl_xor_sync(0xffffffffu, t1m, o));
      }
      if (__any_sync(0xffffffffu, t0m > m[0] || t1m > m[1])) {
        const float n0 = fmaxf(m[0], t0m), n1 = fmaxf(m[1], t1m);
        const float f0 = m[0] == n0 ? 1.f : ex2(m[0] - n0), f1 = m[1] == n1 ? 1.f : ex2(m[1] - n1);
        m[0] = n0; m[1] = n1;
        l[0] *= f0; l[1] *= f1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          acc[i][0] *= f0; acc[i][1] *= f0;
          acc[i][2] *= f1; acc[i][3] *= f1;
        }
      }
      const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = ex2(s[e >> 1][e & 1] - u0), d = ex2(s[e >> 1][2 + (e & 1)] - u1);
        s[e >> 1][e & 1] = a;
        s[e >> 1][2 + (e & 1)] = d;
        if (I8) {  // (an unseen key's scale may be NaN)
          l[0] += (seen0 >> e) & 1u ? a * inv[e] : 0.f;
          l[1] += (seen1 >> e) & 1u ? d * inv[e] : 0.f;
        } else {
          l[0] += a;
          l[1] += d;
        }
      }
      uint32_t pf[4];
      if (I8) {
        pf[0] = pack_half(s[0][0], s[0][1]); pf[1] = pack_half(s[0][2], s[0][3]);
        pf[2] = pack_half(s[1][0], s[1][1]); pf[3] = pack_half(s[1][2], s[1][3]);
      } else {
        pf[0] = pack_bf16(s[0][0], s[0][1]); pf[1] = pack_bf16(s[0][2], s[0][3]);
        pf[2] = pack_bf16(s[1][0], s[1][1]); pf[3] = pack_bf16(s[1][2], s[1][3]);
      }

      // Values: keys 2c, 2c+1 (b0) and those + 8 (b1), element kEV * (n + 8h) + j in tile (h, j).
      const unsigned char* vst = st + kChunk * S::kRow;
#pragma unroll
      for (int h = 0; h < S::kVH; ++h) {
        uint32_t vw[4][S::kEV * S::kElem / 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 2 * c + (e & 1) + 8 * (e >> 1);
          if (S::kEV * S::kElem == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(vst + r * S::kRow + (((n + 8 * h) ^ S::vsw(r)) << 4));
            vw[e][0] = x.x; vw[e][1] = x.y; vw[e][2 % (S::kEV * S::kElem / 4)] = x.z; vw[e][3 % (S::kEV * S::kElem / 4)] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vst + r * S::kRow + (((n >> 1) ^ S::vsw(r)) << 4) + (n & 1) * 8);
            vw[e][0] = x.x; vw[e][1] = x.y;
          }
        }
        if (!I8 && drafts) {
          bool bad = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 2 * c + (e & 1) + 8 * (e >> 1);
            if (j0 + r >= len.ctx)
#pragma unroll
              for (int x = 0; x < S::kEV * S::kElem / 4; ++x) bad |= clear_nonfinite(vw[e][x]);
          }
          poisoned |= __any_sync(0xffffffffu, bad);
        }
#pragma unroll
        for (int x = 0; x < S::kEV * S::kElem / 4; ++x) {
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
            mma<false>(acc[i], pf, __byte_perm(vw[0][x], vw[1][x], 0x5410), __byte_perm(vw[2][x], vw[3][x], 0x5410));
            mma<false>(acc[i + 1], pf, __byte_perm(vw[0][x], vw[1][x], 0x7632), __byte_perm(vw[2][x], vw[3][x], 0x7632));
          }
        }
      }
      __syncwarp();  // all lanes have read the stage before it is filled again
    }
    cp_wait<0>();

    // Infinities and NaNs of drafted tokens' values reach only the rows that
    // attend to them (rare: the product above took them as zeros).
    if (!I8 && !SEL && poisoned) {
      for (int it = 0; it < iters; ++it) {
        const int j0 = k_beg + (it * kWarps + warp) * kChunk;
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
    const bool whole = sg.whole();
    float* part = p.parts + (2LL * blockIdx.x + (sg.first ? 0 : 1)) * kPartFloats<kRowsTile, D>;
    const float* om0 = reinterpret_cast<const float*>(smem);
    for (int x = threadIdx.x; x < 16 * D / 4; x += kThreads) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4, R = row_tile * kRowsTile + r;
      if (r >= rows_left) continue;
      float2 q[kWarps];
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        q[i] = ml_s[i][r];
        mm = fmaxf(mm, q[i].x);
      }
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
  }
}

template <int D, bool I8, bool SEL>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<D, I8>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute a[1] = {};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rows_kernel<D, I8, SEL>, p);
}

template <int D, bool I8, bool SEL>
cudaError_t opt_in() {
  return cudaFuncSetAttribute(rows_kernel<D, I8, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Shape<D, I8>::kSmem);
}

}  // namespace

cudaError_t setup_rows() {
  cudaError_t e = opt_in<64, false, false>();
  if (e == cudaSuccess) e = opt_in<64, false, true>();
  if (e == cudaSuccess) e = opt_in<64, true, false>();
  if (e == cudaSuccess) e = opt_in<64, true, true>();
  if (e == cudaSuccess) e = opt_in<128, false, false>();
  if (e == cudaSuccess) e = opt_in<128, false, true>();
  if (e == cudaSuccess) e = opt_in<128, true, false>();
  if (e == cudaSuccess) e = opt_in<128, true, true>();
  return e;
}

cudaError_t launch_rows(const Params& p, int head_dim, bool i8, bool selected, int grid,
                        cudaStream_t stream) {
  if (head_dim == 64) {
    if (i8) return selected ? launch<64, true, true>(p, grid, stream) : launch<64, true, false>(p, grid, stream);
    return selected ? launch<64, false, true>(p, grid, stream) : launch<64, false, false>(p, grid, stream);
  }
  if (i8) return selected ? launch<128, true, true>(p, grid, stream) : launch<128, true, false>(p, grid, stream);
  return selected ? launch<128, false, true>(p, grid, stream) : launch<128, false, false>(p, grid, stream);
}

}  // namespace attn
}  // namespace tks
