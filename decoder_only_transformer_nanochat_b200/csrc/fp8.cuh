// 8-bit (e4m3) operands with a scale per block: the row kernels that make
// them.  A block of values v with largest magnitude a is held as
//   q = round_e4m3(448 v / a),   s = a / 448   (v ~ q s; a = 0: q = 0, s = 0)
// with fp32 scales.  Activation rows are cut into 1 x 128 blocks along the
// contraction, their scales stored k-block-major (s[kb * lds + row]: the
// scales that a GEMM tile needs for one K block are contiguous); weights
// into 128 x 128 blocks, s[nb * lds + kb].
//
// Which code a value gets is decided exactly for bf16 inputs: z = 448 v / a is
// the quotient of integers below 2^11 and 2^8 times a power of two, so it is
// either a rounding border of e4m3 (at most 5 significant bits) or at least
// 2^-13 away from every one, relatively.  v * RN(448 / a) is within 2^-23 of
// z, so rounding it to 16 significant bits first puts every border case back
// on the border and moves no other value across one: the result is the
// round-to-nearest-even of the exact quotient, without a division per value.
// fp32 inputs take RN(RN(448 v) / a), one IEEE division per value.
#pragma once

#include "elementwise.cuh"

namespace nc {
namespace fp8 {

constexpr float kMax = 448.f;   // largest e4m3 value
constexpr int kBlock = 128;     // values per scale along a row

// two fp32 to two e4m3 (nearest even, saturating): lo in the low byte
__device__ __forceinline__ uint32_t cvt2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  return cvt2(a, b) | (cvt2(c, d) << 16);
}

// What turns a block's values into codes, from the block's largest magnitude
// a.  Blocks below 2^-100 are scaled up by 2^100 first (exact), because
// 448 / a would overflow.
struct Quant {
  float a, inv, pre;
  __device__ __forceinline__ explicit Quant(float amax) {
    pre = amax < 0x1p-100f ? 0x1p100f : 1.f;
    a = amax * pre;
    inv = a > 0.f ? __fdiv_rn(kMax, a) : 0.f;
  }
};

// to the nearest value of 16 significant bits (the split of Veltkamp, "ALGOL
// procedures voor het rekenen in dubbele lengte"); NaN stays NaN
__device__ __forceinline__ uint64_t round16(uint64_t y) {
  const uint64_t k = f2(257.f, 257.f), m1 = f2(-1.f, -1.f);
  const uint64_t t = mul2(y, k);
  const uint64_t d = fma2(y, m1, t);
  return fma2(d, m1, t);
}

template <typename T> __device__ __forceinline__ uint2 quant8(const float (&v)[8], const Quant &z);
template <> __device__ __forceinline__ uint2 quant8<bf16>(const float (&v)[8], const Quant &z) {
  const uint64_t f = f2(z.inv, z.inv), p = f2(z.pre, z.pre);
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t y = round16(mul2(mul2(f2(v[2 * j], v[2 * j + 1]), p), f));
    float lo, hi;
    f2split(y, lo, hi);
    h[j] = cvt2(lo, hi);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
template <> __device__ __forceinline__ uint2 quant8<float>(const float (&v)[8], const Quant &z) {
  uint32_t h[4];
  // above 2^100 the product 448 v could overflow: scaled down instead (exact)
  const float pre = z.a > 0x1p100f ? 0x1p-100f : z.pre;
  const float a = z.a > 0x1p100f ? z.a * 0x1p-100f : z.a;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      y[i] = a != 0.f ? __fdiv_rn(__fmul_rn(v[2 * j + i] * pre, kMax), a) : v[2 * j + i];  // 0 or NaN
    h[j] = cvt2(y[0], y[1]);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
  return a;
}
// over the 16 lanes that hold one block of 128
__device__ __forceinline__ float max16(float a) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// ---------------------------------------------------------------------------
// x' = x + res (rounded to T);  r = 1/sqrt(mean(x'^2) + eps);  y = r x' held in
// e4m3 by blocks: since y / max|y| = x' / max|x'|, the codes come from x'
// alone and only the scale, r max|x'| / 448, carries the norm.
// One warp per row: the row is read once and stays in registers, in its
// storage type until it is used, so that all of its loads are in flight.
template <typename T> struct Raw8;  // eight values as loaded
template <> struct Raw8<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16 *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p + 4));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

template <typename T, int NV, bool kRes>
__global__ void __launch_bounds__(256) add_rmsnorm_fp8_kernel(const T *x, const T *res, T *x_out, uint8_t *__restrict__ q,
                                                              float *__restrict__ s, int64_t lds,
                                                              float *__restrict__ r_out, int M, int C) {
  const int row = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= M) return;
  const int nv = C >> 3;
  const size_t base = (size_t)row * C;
  Raw8<T> xr[NV], rr[kRes ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + 32 * i;
    if (c < nv) {
      xr[i].load(x + base + c * 8);
      if (kRes) rr[i].load(res + base + c * 8);
    }
  }
  float v[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + 32 * i;
    if (c < nv) {
      xr[i].get(v[i]);
      if (kRes) {
        float w[8];
        rr[i].get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = to_f(from_f<T>(v[i][j] + w[j]));
      }
      if (kRes || x_out != x) Vec8<T>::store(x_out + base + c * 8, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  ss = warp_sum(ss);
  const float r = rsqrtf(ss / (float)C + kEps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + 32 * i;
    const float a = max16(amax8(v[i]));
    if (c < nv) {
      const Quant z(a);
      *reinterpret_cast<uint2 *>(q + base + c * 8) = quant8<T>(v[i], z);
      if ((lane & 15) == 0) s[(int64_t)(c >> 4) * lds + row] = __fdiv_rn(a * r, kMax);
    }
  }
  if (r_out && lane == 0) r_out[row] = r;
}

// ---------------------------------------------------------------------------
// 1 x 128 blocks: a warp takes 256 columns of one row, 16 lanes to a block.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T *__restrict__ x, int64_t ldx, uint8_t *__restrict__ q,
                                                         int64_t ldq, float *__restrict__ s, int64_t lds, int rows,
                                                         int cols) {
  const int lane = threadIdx.x & 31;
  const int segs = (cols + 255) >> 8;
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t row = unit / segs;
  if (row >= rows) return;
  const int col = (int)(unit % segs) * 256 + lane * 8;
  float v[8] = {};
  if (col < cols) Vec8<T>::load(x + row * ldx + col, v);
  const float a = max16(amax8(v));
  if (col >= cols) return;
  *reinterpret_cast<uint2 *>(q + row * ldq + col) = quant8<T>(v, Quant(a));
  if ((lane & 15) == 0) s[(int64_t)(col >> 7) * lds + row] = __fdiv_rn(a, kMax);
}

// 128 x 128 blocks: one CTA per block, held in registers between the
// reduction and the codes (16 lanes across, 16 rows per pass, 8 passes).
template <typename T>
__global__ void __launch_bounds__(256) quant_tiles_kernel(const T *__restrict__ x, int64_t ldx, uint8_t *__restrict__ q,
                                                          int64_t ldq, float *__restrict__ s, int64_t lds, int rows,
                                                          int cols) {
  __shared__ float sh[32];
  const int kbs = (cols + kBlock - 1) / kBlock;
  const int nb = blockIdx.x / kbs, kb = blockIdx.x % kbs;
  const int col = kb * kBlock + (threadIdx.x & 15) * 8;
  float v[8][8];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = (int64_t)nb * kBlock + (threadIdx.x >> 4) + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (row < rows && col < cols) Vec8<T>::load(x + row * ldx + col, v[i]);
    a = fmaxf(a, amax8(v[i]));
  }
  a = block_max(a, sh);
  const Quant z(a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = (int64_t)nb * kBlock + (threadIdx.x >> 4) + 16 * i;
    if (row < rows && col < cols) *reinterpret_cast<uint2 *>(q + row * ldq + col) = quant8<T>(v[i], z);
  }
  if (threadIdx.x == 0) s[(int64_t)nb * lds + kb] = __fdiv_rn(a, kMax);
}

// ------------------------------- host side -------------------------------

template <typename T>
inline cudaError_t launch_add_rmsnorm(const T *x, const T *res, T *x_out, uint8_t *q, float *s, int64_t lds, float *r,
                                      int M, int C, cudaStream_t st) {
  const unsigned grid = rows_grid(M, 8);
  if (res)
    NC_DISPATCH_NV(C, (add_rmsnorm_fp8_kernel<T, NV, true><<<grid, 256, 0, st>>>(x, res, x_out, q, s, lds, r, M, C)));
  else
    NC_DISPATCH_NV(C, (add_rmsnorm_fp8_kernel<T, NV, false><<<grid, 256, 0, st>>>(x, res, x_out, q, s, lds, r, M, C)));
  return cudaGetLastError();
}

template <typename T>
inline cudaError_t launch_quant(const T *x, int64_t ldx, uint8_t *q, int64_t ldq, float *s, int64_t lds, int rows,
                                int cols, int block_rows, cudaStream_t st) {
  const int64_t units = block_rows == 1 ? ((int64_t)rows * ((cols + 255) / 256) + 7) / 8
                                        : (((int64_t)rows + 127) / 128) * ((cols + 127) / 128);
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  if (block_rows == 1) quant_rows_kernel<T><<<(unsigned)units, 256, 0, st>>>(x, ldx, q, ldq, s, lds, rows, cols);
  else quant_tiles_kernel<T><<<(unsigned)units, 256, 0, st>>>(x, ldx, q, ldq, s, lds, rows, cols);
  return cudaGetLastError();
}

}  // namespace fp8
}  // namespace nc
