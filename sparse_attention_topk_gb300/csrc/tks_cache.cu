// Writing the keys and values of new tokens into the paged cache, and reading
// rows of it back.
//
// Mathematics.  A row x of head_dim values (one token, one head) is held in 8
// bits as code_d = rint(x_d / scale) with scale = amax / 127, amax = max |x_d|
// held to [2^-40, 2^80]: the error of a value is at most scale / 2.  Both
// divisions are products with a correctly rounded reciprocal, in 32 bits.
//
// What bounds it: bytes.  Nothing is read twice: a row is split over
// head_dim / 16 neighbouring lanes, its maximum goes round them by shuffles, and
// a lane has kRowsPerLane rows in flight.  A lane has eight elements of either
// half of the row, so that a warp's accesses are whole 64- and 128-byte pieces,
// and what is done once a row (slot, address, scale) is done by half the lanes:
// with eight elements a lane, instructions were issued in 78 % of the cycles.
// Measured: 32,768 tokens of 8 heads of 128, bfloat16 to int8, written and read
// back, 406 MB moved in 63.6 us, 6.4 TB/s (73.5 with eight elements a lane; 64.7
// with four rows a lane, 66.6 with one); one token 2.5 us, two launches.

#include "tks_attn.cuh"

namespace tks {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerLane = 2;  // (of 5003 tokens: 8.0 us, 10.5 with four, 8.5 with one)

// Eight elements of a row as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint32_t u[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    u[0] = w.x; u[1] = w.y; u[2] = w.z; u[3] = w.w;
  }
  // The largest magnitude over the row's LANES lanes, two pieces each. Magnitudes are compared as unsigned
  // numbers, two at a time: their order, with NaN on top.
  template <int LANES>
  static __device__ __forceinline__ float amax(const Raw (&r)[2]) {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, r[h].u[i] & 0x7fff7fffu);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __uint_as_float(max(m & 0xffff0000u, m << 16));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  template <int LANES>
  static __device__ __forceinline__ float amax(const Raw (&r)[2]) {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(r[h].v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __uint_as_float(m);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
  }
};
// A row's token; rows are counted head fastest.
__device__ __forceinline__ unsigned token_of(const CacheParams& p, unsigned row) {
  return p.head_shift >= 0 ? row >> p.head_shift : row / (unsigned)p.kv_heads;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                            pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// Four values rounded to nearest even, as codes. Adding 1.5 * 2^23 leaves the rounded number in
// the low bits of the sum.
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  const float k = 12582912.f;
  const uint32_t x = __float_as_uint(__fadd_rn(a, k)), y = __float_as_uint(__fadd_rn(b, k));
  const uint32_t z = __float_as_uint(__fadd_rn(c, k)), w = __float_as_uint(__fadd_rn(d, k));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

// Rows are counted head fastest, then token; blockIdx.y is 0 for keys, 1 for values.
template <typename T, bool I8, int D>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ CacheParams p) {
  constexpr int kLanes = D / 16, kPerPass = kThreads / kLanes;
  const int g = threadIdx.x / kLanes, e = (threadIdx.x % kLanes) * 8;  // and e + D / 2
  const bool value = blockIdx.y != 0;
  const T* src = static_cast<const T*>(value ? p.src_v : p.src_k);
  const long long s_token = value ? p.v_token : p.k_token, s_head = value ? p.v_head : p.k_head;
  unsigned char* dst = value ? p.v : p.k;
  const unsigned total = (unsigned)p.n * (unsigned)p.kv_heads;
  const unsigned row0 = blockIdx.x * (kPerPass * kRowsPerLane) + g;
  grid_wait();
  grid_launch_dependents();

  Raw<T> raw[kRowsPerLane][2];
  int slot[kRowsPerLane];
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    const unsigned row = row0 + i * kPerPass;
    slot[i] = -1;
    if (row < total) {
      const unsigned token = token_of(p, row), head = row - token * p.kv_heads;
      slot[i] = __ldg(p.slots + token);
      const T* at = src + token * s_token + head * s_head + e;
      raw[i][0].load(at);
      raw[i][1].load(at + D / 2);
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    const unsigned row = row0 + i * kPerPass;
    const unsigned head = row - token_of(p, row) * p.kv_heads;
    const bool ok = slot[i] >= 0 && slot[i] < p.slots_held;
    if (slot[i] >= p.slots_held) report(p.status, kStatIndexBit);
    float amax = I8 ? Raw<T>::template amax<kLanes>(raw[i]) : 0.f;
    if (!ok) continue;
    unsigned char* at = dst + (slot[i] >> p.page_shift) * p.page_b + (slot[i] & ((1 << p.page_shift) - 1)) * p.token_b + head * p.head_b;
    if (!I8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[8];
        raw[i][h].get(x);
        store8(reinterpret_cast<__nv_bfloat16*>(at) + e + h * (D / 2), x);
      }
      continue;
    }
    const float lo = 9.094947017729282e-13f, hi = 1.2089258196146292e24f;  // 2^-40, 2^80
    const bool beyond = amax > hi;
    amax = amax < lo ? lo : beyond ? hi : amax;  // (a NaN stays one)
    const float scale = __fmul_rn(amax, 1.0f / 127.0f), inv = __frcp_rn(scale);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8];
      raw[i][h].get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], inv);
      if (beyond)  // (otherwise no value is beyond 127)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fminf(fmaxf(x[j], -127.f), 127.f);
      *reinterpret_cast<uint2*>(at + e + h * (D / 2)) = make_uint2(pack_codes(x[0], x[1], x[2], x[3]), pack_codes(x[4], x[5], x[6], x[7]));
    }
    if (e == 0) p.scales[2 * ((long long)slot[i] * p.kv_heads + head) + (value ? 1 : 0)] = scale;
  }
}

template <typename T, bool I8, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ CacheParams p) {
  constexpr int kLanes = D / 16, kPerPass = kThreads / kLanes;
  const int g = threadIdx.x / kLanes, e = (threadIdx.x % kLanes) * 8;
  const bool value = blockIdx.y != 0;
  T* dst = static_cast<T*>(value ? p.out_v : p.out_k);
  const unsigned char* src = value ? p.v : p.k;
  const unsigned total = (unsigned)p.n * (unsigned)p.kv_heads;
  const unsigned row0 = blockIdx.x * (kPerPass * kRowsPerLane) + g;
  grid_wait();
  grid_launch_dependents();

  int slot[kRowsPerLane];
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    const unsigned row = row0 + i * kPerPass;
    slot[i] = row < total ? __ldg(p.slots + token_of(p, row)) : -1;
    if (slot[i] >= p.slots_held) {
      report(p.status, kStatIndexBit);
      slot[i] = -1;
    }
  }
  uint4 w[kRowsPerLane][2];
  float scale[kRowsPerLane];
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    const unsigned row = row0 + i * kPerPass;
    const unsigned head = row - token_of(p, row) * p.kv_heads;
    w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0.f;
    if (slot[i] < 0) continue;
    const unsigned char* at = src + (slot[i] >> p.page_shift) * p.page_b +
                              (slot[i] & ((1 << p.page_shift) - 1)) * p.token_b + head * p.head_b;
    if (I8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 y = *reinterpret_cast<const uint2*>(at + e + h * (D / 2));
        w[i][h].x = y.x;
        w[i][h].y = y.y;
      }
      scale[i] = p.scales[2 * ((long long)slot[i] * p.kv_heads + head) + (value ? 1 : 0)];
    } else {
      w[i][0] = *reinterpret_cast<const uint4*>(at + 2 * e);
      w[i][1] = *reinterpret_cast<const uint4*>(at + 2 * e + D);
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    const unsigned row = row0 + i * kPerPass;
    if (row >= total) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t u[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (I8)
          x[j] = (float)(int)(signed char)(u[j >> 2] >> (8 * (j & 3))) * scale[i];
        else
          x[j] = __uint_as_float(j & 1 ? u[j >> 1] & 0xffff0000u : u[j >> 1] << 16);
      }
      store8(dst + (long long)row * D + e + h * (D / 2), x);
    }
  }
}

template <typename K>
cudaError_t run(K kernel, const CacheParams& p, int head_dim, cudaStream_t stream) {
  const unsigned per = kThreads / (head_dim / 16) * kRowsPerLane;
  const unsigned long long rows = (unsigned long long)p.n * p.kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + per - 1) / per), 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute a[1] = {};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheParams& p, int head_dim, bool i8, bool f32, cudaStream_t s) {
  if (head_dim == 64) {
    if (i8) return f32 ? run(write_kernel<float, true, 64>, p, 64, s) : run(write_kernel<__nv_bfloat16, true, 64>, p, 64, s);
    return f32 ? run(write_kernel<float, false, 64>, p, 64, s) : run(write_kernel<__nv_bfloat16, false, 64>, p, 64, s);
  }
  if (i8) return f32 ? run(write_kernel<float, true, 128>, p, 128, s) : run(write_kernel<__nv_bfloat16, true, 128>, p, 128, s);
  return f32 ? run(write_kernel<float, false, 128>, p, 128, s) : run(write_kernel<__nv_bfloat16, false, 128>, p, 128, s);
}

cudaError_t launch_cache_read(const CacheParams& p, int head_dim, bool i8, bool f32, cudaStream_t s) {
  if (head_dim == 64) {
    if (i8) return f32 ? run(read_kernel<float, true, 64>, p, 64, s) : run(read_kernel<__nv_bfloat16, true, 64>, p, 64, s);
    return f32 ? run(read_kernel<float, false, 64>, p, 64, s) : run(read_kernel<__nv_bfloat16, false, 64>, p, 64, s);
  }
  if (i8) return f32 ? run(read_kernel<float, true, 128>, p, 128, s) : run(read_kernel<__nv_bfloat16, true, 128>, p, 128, s);
  return f32 ? run(read_kernel<float, false, 128>, p, 128, s) : run(read_kernel<__nv_bfloat16, false, 128>, p, 128, s);
}

}  // namespace attn
}  // namespace tks
