// E4M3 with one fp32 scale for each block of 128 along K: pieces of 1 x 128 of
// a row (activations) or blocks of 128 x 128 (weights).
//   scale = max(absmax(block) / 448, 2^-126), 1 for an all-zero block
//   code  = E4M3(x / scale), round to nearest even, saturating
// (DeepSeek-V3's FP8 format; jacopoparretti "Mixture of experts, token by
// token", "Memory".) A block that holds a NaN comes out as NaN; one that holds
// an infinity has an infinite scale, finite elements 0 and infinite ones NaN.
//
// Bound: memory (bf16: 3 bytes an element, read and written once), close to
// issue: 8192 x 7168 rows 34 us (5.2 TB/s, 0.80 of the measured copy; issue 76%
// of active cycles), weights 8 x 14336 x 4096 244 us (5.8 TB/s, 0.88); fp32 in: 44 us
// back to back (6.7 TB/s, part from L2) and, 2 x 14336 x 4096, 101 us (5.8 TB/s).
// The dequantiser writes four bytes a code: 8192 x 7168 64 us (4.6 TB/s). The block stays in registers between
// its maximum and its codes. The quotient is the one of an fp32 division: q = x y
// corrected once by its remainder, q + (x - q scale) y with y = 1 / scale
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), three fused operations where a division of its own for each element would make these
// kernels bound by arithmetic. Outside 2^-80 .. 2^100 the remainder could
// underflow or the reciprocal vanish: such blocks divide.
#pragma once
#include "quant_formats.cuh"
#include <float.h>

namespace moe {
namespace f8b {

constexpr int BLK = 128;

// NaN-propagating maximum of magnitudes.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float block_scale(float absmax) {
  return absmax == 0.f ? 1.f : (absmax != absmax ? absmax : fmaxf(absmax / 448.0f, FLT_MIN));
}

// Two fp32 -> two E4M3 codes (a in the low byte), round to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __noinline__ uint32_t e4m3x4_by_division(float a, float b, float c, float d, float s) {
  return e4m3x2(__fdiv_rn(a, s), __fdiv_rn(b, s)) |
         e4m3x2(__fdiv_rn(c, s), __fdiv_rn(d, s)) << 16;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

struct Divisor {
  float scale;
  uint64_t neg_inv2, scale2;  // -1 / scale and scale, twice each
  bool fast;
  __device__ __forceinline__ explicit Divisor(float s) : scale(s) {
    fast = s > 0x1p-80f && s < 0x1p100f;
    const float inv = fast ? __frcp_rn(s) : 0.f;
    neg_inv2 = pack2(-inv, -inv);
    scale2 = pack2(s, s);
  }
  // Codes of -a / scale and -b / scale: fp32 rounds both signs alike, and the negated
  // form keeps a zero's sign (+0 gives -0 + -0 = -0, and -0 gives +0 + -0 = +0), where
  // q + r y itself makes +0 of both.
  __device__ __forceinline__ uint32_t neg_codes2(float a, float b) const {
    const uint64_t x = pack2(a, b);
    uint64_t q;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(neg_inv2));
    q = fma2(fma2(q, scale2, x), neg_inv2, q);
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(q));
    return e4m3x2(lo, hi);
  }
};

__device__ __forceinline__ uint32_t encode4(const float* f, const Divisor& d) {
  if (d.fast)
    return (d.neg_codes2(f[0], f[1]) | d.neg_codes2(f[2], f[3]) << 16) ^ 0x80808080u;
  return e4m3x4_by_division(f[0], f[1], f[2], f[3], d.scale);
}

// Row blocks a lane has in flight: 64 (bf16) or 128 (fp32) bytes of loads.
template <typename TX> constexpr int ROW_UNITS = 2;

// Sixteen consecutive elements held as raw 16-byte vectors.
template <typename TX> struct Vec16E {
  static constexpr int NVEC = 16 * sizeof(TX) / 16;
  uint4 u[NVEC];
  __device__ __forceinline__ void load(const TX* p) {
#pragma unroll
    for (int i = 0; i < NVEC; ++i) u[i] = ld_nc_v4(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NVEC; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(int i, float* f) const { Vec16<TX>::unpack(u[i], f); }
  // Largest magnitude. The bits of magnitudes order as integers do, NaNs above
  // infinity: bf16 pairs are compared as two 16-bit integers at once.
  __device__ __forceinline__ float absmax() const {
    if (sizeof(TX) == 2) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NVEC; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
      }
      return __uint_as_float(max(m << 16, m & 0xffff0000u));
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NVEC; ++i)
      m = max(max(max(m, u[i].x & 0x7fffffffu), max(u[i].y & 0x7fffffffu, u[i].z & 0x7fffffffu)),
              u[i].w & 0x7fffffffu);
    return __uint_as_float(m);
  }
  __device__ __forceinline__ uint4 codes(const Divisor& d) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
      float f[Vec16<TX>::N];
      values(i, f);
#pragma unroll
      for (int j = 0; j < Vec16<TX>::N / 4; ++j)
        w[i * (Vec16<TX>::N / 4) + j] = encode4(f + 4 * j, d);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// 1 x 128 blocks: eight lanes a block, sixteen elements a lane, UNITS blocks a
// lane whose loads are all in flight before the first is used.
template <typename TX>
__global__ void __launch_bounds__(256) quantize_row_blocks_kernel(
    const TX* __restrict__ x, int64_t rows, int cols, int64_t ld, int step_r, int step_b,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int UNITS = ROW_UNITS<TX>;
  const int kb = (cols + BLK - 1) / BLK;
  const int64_t units = rows * kb;  // blocks
  const int sub = threadIdx.x & 7;
  const int64_t u0 = (int64_t)blockIdx.x * (32 * UNITS) + (threadIdx.x >> 3);
  Vec16E<TX> v[UNITS];
  int64_t at[UNITS];  // where this lane's codes go, -1 behind the last column or block
  int64_t r;
  int b;
  if (units <= 0x7fffffff) {
    r = (uint32_t)u0 / (uint32_t)kb;
    b = (int)((uint32_t)u0 - (uint32_t)r * (uint32_t)kb);
  } else {
    r = u0 / kb;
    b = (int)(u0 - r * kb);
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int c = b * BLK + sub * 16;
    at[i] = r < rows && c < cols ? r * cols + c : -1;
    if (at[i] >= 0) v[i].load(x + r * ld + c); else v[i].zero();
    r += step_r;  // 32 blocks on: 32 = step_r kb + step_b
    b += step_b;
    if (b >= kb) {
      b -= kb;
      ++r;
    }
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    float m = v[i].absmax();
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = block_scale(m);
    if (at[i] >= 0) {
      st_v4(codes + at[i], v[i].codes(Divisor(s)));
      if (sub == 0) scales[u0 + 32 * i] = s;
    }
  }
}

// The layer's permute step on this format: token rows quantised in 1 x 128 blocks
// and their codes and scales stored at each kept assignment's row (the positions
// are those of scatter_kernel in permute.cuh). One warp a token and 512 columns:
// eight lanes a block, sixteen elements a lane.
template <typename TX>
__global__ void __launch_bounds__(256) quantize_scatter_kernel(
    const TX* __restrict__ x, int d, int T, int k, int E, int64_t C,
    const int32_t* __restrict__ idx, const float* __restrict__ gate,
    const int32_t* __restrict__ lrank, const int32_t* __restrict__ base,
    const int32_t* __restrict__ tile_start, int32_t* __restrict__ slot_pos,
    float* __restrict__ row_gate, uint8_t* __restrict__ codes, float* __restrict__ scales,
    int64_t rows_max) {
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= T) return;  // warp-uniform
  int mypos = -1;
  if (lane < k) {
    const size_t a = (size_t)t * k + lane;
    const int e = idx[a];
    const int rank = base[(size_t)(t / ROUTE_CHUNK) * E + e] + lrank[a];
    if (C < 0 || (int64_t)rank < C) mypos = tile_start[e] * ROW_TILE + rank;
#if defined(MOE_DEBUG)
    if (mypos >= 0 && ((int64_t)mypos >= rows_max || mypos >= tile_start[e + 1] * ROW_TILE ||
                       e < 0 || e >= E)) {
      flag_bounds();
      mypos = -1;
    }
#else
    (void)rows_max;
#endif
    if (blockIdx.y == 0) {
      if (mypos >= 0) row_gate[mypos] = gate[a];
      slot_pos[a] = mypos;
    }
  }
  const int kb = (d + BLK - 1) / BLK;
  const int c = blockIdx.y * 512 + lane * 16, b = c / BLK;
  Vec16E<TX> v;
  if (c < d) v.load(x + (size_t)t * d + c); else v.zero();
  float m = v.absmax();
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float s = block_scale(m);
  const uint4 q = v.codes(Divisor(s));
  for (int i = 0; i < k; ++i) {
    const int64_t row = __shfl_sync(0xffffffffu, mypos, i);
    if (row < 0) continue;
    if (c < d) {
      st_v4(codes + row * d + c, q);
      if ((lane & 7) == 0) scales[row * kb + b] = s;
    }
  }
}

// 128 x 128 blocks: one block of 256 threads each, 64 elements a thread; four
// (fp32: two) blocks an SM, so that one's loads cover another's arithmetic.
template <typename TX>
__global__ void __launch_bounds__(256, sizeof(TX) == 2 ? 4 : 2) quantize_square_blocks_kernel(
    const TX* __restrict__ x, int64_t rows, int cols, int64_t ld, int nb, int kb,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float red[8];
  const int64_t tile = blockIdx.x;
  const int64_t e = tile / ((int64_t)nb * kb);
  const int in_e = (int)(tile - e * nb * kb);
  const int rb = in_e / kb, cb = in_e - rb * kb;
  const int c = cb * BLK + (threadIdx.x & 7) * 16;
  const TX* src = x + e * rows * ld;
  uint8_t* dst = codes + e * rows * cols;
  Vec16E<TX> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = (int64_t)rb * BLK + i * 32 + (threadIdx.x >> 3);
    if (r < rows && c < cols) v[i].load(src + r * ld + c); else v[i].zero();
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_nan(m, v[i].absmax());
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max_nan(m, red[w]);
  const float s = block_scale(m);
  const Divisor d(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = (int64_t)rb * BLK + i * 32 + (threadIdx.x >> 3);
    if (r < rows && c < cols) st_v4(dst + r * cols + c, v[i].codes(d));
  }
  if (threadIdx.x == 0) scales[tile] = s;
}

// out = value(code) * scale of its block, rounded once to fp32. Sixteen codes a thread.
__global__ void __launch_bounds__(256) dequantize_blocks_kernel(
    const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t stack,
    int64_t rows, int cols, int block_rows, float* __restrict__ out) {
  pdl_wait();
  pdl_launch_dependents();
  const int vpr = cols / 16, kb = (cols + BLK - 1) / BLK;
  const int64_t nb = (rows + block_rows - 1) / block_rows, n = stack * rows * vpr;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / vpr, e = row / rows, r = row - e * rows;
    const int c = (int)(i - row * vpr) * 16;
    const float s = scales[(e * nb + r / block_rows) * kb + c / BLK];
    const uint4 v = ld_nc_v4(codes + i * 16);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    float4* o = reinterpret_cast<float4*>(out + i * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t lo, hi;
      tcf8::e4m3x4_to_f16x4(in[j], lo, hi);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      o[j] = make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
    }
  }
}

}  // namespace f8b
}  // namespace moe
