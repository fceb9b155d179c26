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
// 2^-13 away from every one, relatively.  v times an approximate 448 / a is
// within 2^-20 of z, so rounding it to 16 significant bits first puts every border case back
// on the border and moves no other value across one: the result is the
// round-to-nearest-even of the exact quotient, without a division per value.
// fp32 inputs take RN(RN(448 v) / a): the same approximate product decides, but
// for the one value in 2^14 so close to a border that the division has to.
#pragma once

#include "elementwise.cuh"

namespace nc {
namespace fp8 {

constexpr float kMax = 448.f;   // largest e4m3 value
constexpr int kBlock = 128;     // values per scale along a row

// These kernels are launched so that they may start while the kernel before
// them in the stream still runs (programmatic stream serialization): each lets
// its own successor start as soon as all of its CTAs have set up, and touches global
// memory only after pdl_wait(), which returns when the kernel before has
// completed and its writes are visible.  Launch and set-up then overlap the
// predecessor's end (calls in a row, us: 16 x 65,536 x 1280 GEMM 20.5 -> 17.7,
// 1001 x 1003 x 1040 14.3 -> 12.7, an 8192 x 2048 weight's codes 20.3 -> 17.7).
// So what the kernel before may have written is not read-only while these run:
// inputs carry no const __restrict__, under which a load could be taken through
// the read-only path or moved above the wait.
__device__ __forceinline__ void pdl_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch(void (*kernel)(P...), unsigned grid, int threads, int smem, int cluster, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

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
// a: the factor 448 / a to 2^-21 (the approximate reciprocal is within one
// unit).  Blocks below 2^-100 are scaled up by 2^100 first (exact), because
// 448 / a would overflow.
struct Quant {
  float a, inv, pre;
  __device__ __forceinline__ explicit Quant(float amax) {
    pre = amax < 0x1p-100f ? 0x1p100f : 1.f;
    a = amax * pre;
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(a));
    inv = a > 0.f ? kMax * r : 0.f;
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
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t w = f2(v[2 * j], v[2 * j + 1]);
    if (z.pre != 1.f) w = mul2(w, p);
    f2split(round16(mul2(w, f)), y[2 * j], y[2 * j + 1]);
  }
  return make_uint2(cvt4(y[0], y[1], y[2], y[3]), cvt4(y[4], y[5], y[6], y[7]));
}
template <> __device__ __forceinline__ uint2 quant8<float>(const float (&v)[8], const Quant &z) {
  // v times the approximate 448 / a is within 2^-20 of RN(RN(448 v) / a).  Only
  // where it lies that close to a value of six significant bits, which every
  // border is, can the two get different codes: those (one value in 2^14) take
  // the division.
  const uint64_t f = f2(z.inv, z.inv), p = f2(z.pre, z.pre), k = f2(262145.f, 262145.f), m1 = f2(-1.f, -1.f);
  float y[8];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t q = mul2(mul2(f2(v[2 * j], v[2 * j + 1]), p), f);
    const uint64_t t = mul2(q, k);
    const uint64_t h = fma2(fma2(q, m1, t), m1, t);  // q to six bits
    float e0, e1;
    f2split(fma2(h, m1, q), e0, e1);
    f2split(q, y[2 * j], y[2 * j + 1]);
    near |= fabsf(e0) < fabsf(y[2 * j]) * 0x1p-20f || fabsf(e1) < fabsf(y[2 * j + 1]) * 0x1p-20f;  // not for 0
  }
  if (near && z.a > 0.f) {
    // above 2^100 the product 448 v could overflow: scaled down instead (exact)
    const float pre = z.a > 0x1p100f ? 0x1p-100f : z.pre;
    const float a = z.a > 0x1p100f ? z.a * 0x1p-100f : z.a;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(__fmul_rn(v[j] * pre, kMax), a);
  }
  return make_uint2(cvt4(y[0], y[1], y[2], y[3]), cvt4(y[4], y[5], y[6], y[7]));
}

// The codes of fp32 values that stand in f32x2 pairs, as an epilogue has them,
// by the same rule, RN_e4m3(RN(RN(448 v) / a)), without a division or a branch
// per value: n = RN(448 v) times 1 / a held as two floats, rh + rl, each rounded
// to nearest, as RN(n rh + RN(n rl)) (Brisebarre and Muller, "Correctly rounded
// multiplication by arbitrary precision constants").  That is off by less than
// 2^-47 before its rounding, for a in [1, 2) and n / a around 1; and n / a, as a
// quotient of 24-bit numbers beside a border of 5 bits, stays that far from the
// middle between two floats unless a's 24-bit significand is within 4 of a
// multiple of 2^20.  All of those (and 40 to each side) give the right code for
// every border and every n around it.  v and a are scaled by one power of two,
// exactly, so that a is in [1, 4) (or, for a < 2^-119, at least 2^-30): nothing
// overflows, and nothing that a code but 0 comes from is subnormal.  Against one
// product with an approximate 448 / a this costs 8 us of 228 at 32,768 x 5120 x
// 1280 (a residual step, y + (n - y a) / a, 14; two bracketing products and
// that step only where their codes differ, 12).
struct Ratio {
  uint64_t k, rh, rl;  // 448 scaled; 1 / a scaled
  __device__ __forceinline__ explicit Ratio(float a) {
    const int e = min(max((int)(__float_as_uint(a) >> 23), 8), 253);  // exponent field
    const float s = __uint_as_float((uint32_t)(254 - e) << 23), kf = kMax * s;
    const bool any = a > 0.f && a < INFINITY;  // else codes are 0, but for what is not finite
    const float af = any ? a * s : 1.f, h = __frcp_rn(af), l = __fdiv_rn(fmaf(-h, af, 1.f), af);  // 1 - h a is exact
    k = f2(kf, kf);
    rh = any ? f2(h, h) : 0;
    rl = any ? f2(l, l) : 0;
  }
  __device__ __forceinline__ uint32_t codes4(uint64_t v0, uint64_t v1) const {
    const uint64_t n0 = mul2(v0, k), n1 = mul2(v1, k);
    float a, b, c, d;
    f2split(fma2(n0, rh, mul2(n0, rl)), a, b);
    f2split(fma2(n1, rh, mul2(n1, rl)), c, d);
    return cvt4(a, b, c, d);
  }
};

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
// Bandwidth-bound: 32,768 x 1280 bf16 rows 46 us, 6.4 TB/s; one row 1.9 us.
// WPR warps per row (one where there are rows enough to fill the SMs, four
// otherwise): the row is read once and stays in registers, in its storage type
// until it is used, so that all of its loads are in flight.
template <typename T> struct Raw8;  // eight values as loaded
template <> struct Raw8<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ float amax() const {  // largest magnitude, two at a time
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    return fmaxf(__low2float(m), __high2float(m));
  }
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
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ float amax() const {
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                 fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

template <typename T, int NV, int WPR, bool kRes>
__global__ void __launch_bounds__(256) add_rmsnorm_fp8_kernel(const T *x, const T *res, T *x_out, uint8_t *__restrict__ q,
                                                              float *__restrict__ s, int64_t lds,
                                                              float *__restrict__ r_out, int M, int C) {
  constexpr int T_ROW = 32 * WPR;  // threads per row
  pdl_start();
  pdl_wait();
  const int row = blockIdx.x * (256 / T_ROW) + threadIdx.x / T_ROW;
  const int lane = threadIdx.x % T_ROW;
  if (WPR == 1 && row >= M) return;  // with more, whole warps of a missing row take part in the barrier
  const bool in = row < M;
  const int nv = C >> 3;
  const size_t base = (size_t)row * C;
  Raw8<T> xr[NV], rr[kRes ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + T_ROW * i;
    if (in && c < nv) {
      xr[i].load(x + base + c * 8);
      if (kRes) rr[i].load(res + base + c * 8);
    }
  }
  float v[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + T_ROW * i;
    if (in && c < nv) {
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
  if constexpr (WPR > 1) {
    __shared__ float part[8];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    const int w0 = threadIdx.x / T_ROW * WPR;
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) ss += part[w0 + w];
  }
  const float r = rsqrtf(ss / (float)C + kEps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + T_ROW * i;
    const float a = max16(amax8(v[i]));
    if (in && c < nv) {
      const Quant z(a);
      *reinterpret_cast<uint2 *>(q + base + c * 8) = quant8<T>(v[i], z);
      if ((lane & 15) == 0) s[(int64_t)(c >> 4) * lds + row] = __fdiv_rn(a * r, kMax);
    }
  }
  if (r_out && in && lane == 0) r_out[row] = r;
}

// ---------------------------------------------------------------------------
// 1 x 128 blocks: a warp takes 256 columns of four rows, 16 lanes to a block,
// a CTA 32 rows of the same columns.  Lanes 0..3 and 16..19 then hold one
// row's maximum each, so the four rows' scales take one division and one store.
// 16,384 x 2048 bf16: 24 us, 4.2 TB/s: instruction issue (72 % of the slots, the
// integer pipe 55 %, at 65,536 x 1280), in CTAs whose loads, arithmetic and
// stores follow one another, five to an SM by their registers.
// (Measured against CTAs that walk several units with the next one's loads in
// flight: 23.9 against 26.8 us at 16,384 x 2048 bf16.)
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T *x, int64_t ldx, uint8_t *__restrict__ q,
                                                         int64_t ldq, float *__restrict__ s, int64_t lds, int rows,
                                                         int cols, unsigned segs) {
  pdl_start();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int col = (int)(blockIdx.x % segs) * 256 + lane * 8;
  const int64_t row0 = (int64_t)(blockIdx.x / segs) * 32 + (threadIdx.x >> 5) * 4;
  Raw8<T> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + i < rows && col < cols) raw[i].load(x + (row0 + i) * ldx + col);
  float mine = 0.f;  // the maximum whose scale this lane stores
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row0 + i >= rows) break;
    const float a = max16(col < cols ? raw[i].amax() : 0.f);
    if ((lane & 15) == i) mine = a;
    if (col < cols) {
      float v[8];
      raw[i].get(v);
      *reinterpret_cast<uint2 *>(q + (row0 + i) * ldq + col) = quant8<T>(v, Quant(a));
    }
  }
  const int kb = (int)(blockIdx.x % segs) * 2 + (lane >> 4), i = lane & 15;
  if (i < 4 && row0 + i < rows && kb * kBlock < cols) s[(int64_t)kb * lds + row0 + i] = __fdiv_rn(mine, kMax);
}

// 128 x 128 blocks: one CTA per block, held in registers as loaded between the
// reduction and the codes (16 lanes across, 32 rows per pass, 4 passes).
// 8192 x 2048 fp32: 18 to 19 us, 4.5 TB/s; the block's maximum stands between its
// loads and its stores, and two or three CTAs per SM hide that in part.
template <typename T>
__global__ void __launch_bounds__(512, sizeof(T) == 2 ? 3 : 2)
    quant_tiles_kernel(const T *x, int64_t ldx, uint8_t *__restrict__ q, int64_t ldq,
                       float *__restrict__ s, int64_t lds, int rows, int cols, unsigned kbs) {
  __shared__ float sh[16];
  pdl_start();
  pdl_wait();
  const unsigned nb = blockIdx.x / kbs, kb = blockIdx.x % kbs;
  const int col = (int)kb * kBlock + (threadIdx.x & 15) * 8;
  const int64_t row0 = (int64_t)nb * kBlock + (threadIdx.x >> 4);
  Raw8<T> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + 32 * i < rows && col < cols) raw[i].load(x + (row0 + 32 * i) * ldx + col);
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + 32 * i < rows && col < cols) a = fmaxf(a, raw[i].amax());
  a = warp_max(a);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
  __syncthreads();
  a = warp_max(sh[threadIdx.x & 15]);
  const Quant z(a);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + 32 * i < rows && col < cols) {
      float v[8];
      raw[i].get(v);
      *reinterpret_cast<uint2 *>(q + (row0 + 32 * i) * ldq + col) = quant8<T>(v, z);
    }
  if (threadIdx.x == 0) s[(int64_t)nb * lds + kb] = __fdiv_rn(a, kMax);
}

// ------------------------------- host side -------------------------------

template <typename T, bool kRes>
inline cudaError_t launch_norm(const T *x, const T *res, T *x_out, uint8_t *q, float *s, int64_t lds, float *r, int M,
                               int C, cudaStream_t st) {
  // bf16 rows of up to 2048 values take a warp each once there are enough of
  // them to fill the SMs (1280 wide, us: 2048 rows 5.9 against 6.6 with four
  // warps, 32,768 rows 49.1 against 54.9; 256 rows 4.6 against 3.6).  fp32 rows
  // do not fit one warp's registers as well (4096 x 2048: 39.7 against 21.7).
  if constexpr (sizeof(T) == 2) {
    if (M >= 2048 && C <= 2048) {
      const unsigned grid = rows_grid(M, 8);
      switch ((C / 8 + 31) / 32) {
        case 1: return launch(add_rmsnorm_fp8_kernel<T, 1, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
        case 2: return launch(add_rmsnorm_fp8_kernel<T, 2, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
        case 3: return launch(add_rmsnorm_fp8_kernel<T, 3, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
        case 4: return launch(add_rmsnorm_fp8_kernel<T, 4, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
        case 5: return launch(add_rmsnorm_fp8_kernel<T, 5, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
        case 6: return launch(add_rmsnorm_fp8_kernel<T, 6, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
        case 7: return launch(add_rmsnorm_fp8_kernel<T, 7, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
        default: return launch(add_rmsnorm_fp8_kernel<T, 8, 1, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
      }
    }
  }
  const unsigned grid = rows_grid(M, 2);
  switch ((C / 8 + 127) / 128) {
    case 1: return launch(add_rmsnorm_fp8_kernel<T, 1, 4, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
    case 2: return launch(add_rmsnorm_fp8_kernel<T, 2, 4, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
    case 3: return launch(add_rmsnorm_fp8_kernel<T, 3, 4, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
    default: return launch(add_rmsnorm_fp8_kernel<T, 4, 4, kRes>, grid, 256, 0, 1, st, x, res, x_out, q, s, lds, r, M, C);
  }
}

template <typename T>
inline cudaError_t launch_add_rmsnorm(const T *x, const T *res, T *x_out, uint8_t *q, float *s, int64_t lds, float *r,
                                      int M, int C, cudaStream_t st) {
  return res ? launch_norm<T, true>(x, res, x_out, q, s, lds, r, M, C, st)
             : launch_norm<T, false>(x, res, x_out, q, s, lds, r, M, C, st);
}

// CTAs of a quantiser's grid: 32 x 256 values each, or a block
inline int64_t quant_units(int rows, int cols, int block_rows) {
  const int across = block_rows == 1 ? 256 : 128, down = block_rows == 1 ? 32 : 128;
  return ((int64_t)rows + down - 1) / down * ((cols + across - 1) / across);
}

template <typename T>
inline cudaError_t launch_quant(const T *x, int64_t ldx, uint8_t *q, int64_t ldq, float *s, int64_t lds, int rows,
                                int cols, int block_rows, cudaStream_t st) {
  const unsigned units = (unsigned)quant_units(rows, cols, block_rows);
  if (block_rows == 1)
    return launch(quant_rows_kernel<T>, units, 256, 0, 1, st, x, ldx, q, ldq, s, lds, rows, cols, (cols + 255) / 256);
  return launch(quant_tiles_kernel<T>, units, 512, 0, 1, st, x, ldx, q, ldq, s, lds, rows, cols, (cols + 127) / 128);
}

}  // namespace fp8
}  // namespace nc
