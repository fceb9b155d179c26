// e4m3 GEMM with block scales on the 5th-generation tensor cores:
//   D[m, n] = epilogue( sum_kb sa[kb, m] sb[n / 128, kb] sum_{k in block kb} A[m, k] B[n, k] )
// A: activations [M, K] with a scale per 1 x 128 block, B: weights [N, K]
// with a scale per 128 x 128 block, both K-major (y = x W^T).  One K block is
// 128 bytes of a row: the width of a 128-byte-swizzled tile and four
// tcgen05.mma kind::f8f6f4 steps of K = 32.
//
// The tensor core sums one K block into a fresh TMEM accumulator; the
// epilogue warps read it back, scale it and add it to fp32 sums in registers
// while the next block is multiplied (the scales differ per block, so the
// tensor core's own accumulator cannot run over the whole K).
#pragma once

#include "fp8.cuh"
#include "gemm_tc.cuh"

namespace nc {

// epilogue that leaves relu(acc)^2 in e4m3 with 1 x 128 scales: the next GEMM's A operand
constexpr int EPI_RELU2_FP8 = 7;

struct GemmFp8Problem {
  int M, N, K;
  const void *A;
  int64_t lda;
  const float *sa;
  int64_t lsa;
  const void *B;
  int64_t ldb;
  const float *sb;
  int64_t lsb;
  void *D;
  int64_t ldd;
  float *sd;
  int64_t lsd;
  int epi;
};

namespace tc8 {

using namespace tc;

constexpr int BK = 128;  // one scale block of K

// kind::f8f6f4: fp32 accumulate, e4m3 A and B (type codes 0), both K-major
__host__ __device__ constexpr uint32_t idesc8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_nw(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 15 tanh(z / 15) from one exponential: t = (1 - E) / (1 + E), E = exp(-2 |z| / 15)
__device__ __forceinline__ float softcap8(float z) {
  const float e = __expf(-2.f / kSoftcap * fabsf(z));
  return copysignf(kSoftcap * __fdividef(1.f - e, 1.f + e), z);
}

// ===========================================================================
// Few rows: the weights are the M = 128 operand of the tensor core and TN
// activation rows the N operand, so one decoded token costs an N = 16 tile
// instead of a 128-row one.
//
// Roles: warp 0 TMA, warp 1 MMA, the others add up (thread = weight row, up
// to 64 activation rows in registers).
template <int TN> struct RowsCfg {
  static constexpr int kEpiWarps = TN > 64 ? 8 : 4;        // 4 cover the 128 TMEM lanes; 8: two column halves
  static constexpr int kCols = TN * 4 / kEpiWarps;         // activation rows per thread
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kStageBytes = (128 + TN) * BK;
  static constexpr int kStages = TN == 16 ? 6 : TN == 32 ? 5 : TN == 64 ? 4 : 3;
  static constexpr int kAccs = TN > 64 ? 2 : 4;            // TMEM accumulators in flight
  static constexpr int kTmemCols = kAccs * TN;             // 64, 128, 256, 256: a power of two
  static constexpr int kScaleBytes = kEpiWarps * kCols * 4;
  static constexpr int kSmem = kStages * kStageBytes + kScaleBytes + 256 + 1024;
  static_assert(TN * 128 * 4 <= kStages * kStageBytes, "the sums of a tile fit the ring");
  // two CTAs share an SM and no third fits, so their TMEM always does
  static_assert(2 * kSmem <= 232448 && 3 * kSmem > 232448 && 2 * kTmemCols <= 512, "two CTAs per SM");
};

struct RowsParams {
  int M, N, kblocks;
  int n_m, n_n;
  const float *sa, *sb;
  int64_t lsa, lsb;
  void *D;
  int64_t ldd;
  float *sd;
  int64_t lsd;
  int epi;
  int *status;
};

// One activation row m, this lane's four weight rows [n, n + 4): v = sums
__device__ __forceinline__ void rows_store(const RowsParams &p, int m, int n, float (&v)[4], int lane) {
  const int left = p.N - n;  // <= 0: nothing to store (the lane still takes part in the block's maximum)
  if (p.epi == EPI_STORE_F32) {
    float *d = reinterpret_cast<float *>(p.D) + (int64_t)m * p.ldd + n;
    if (left >= 4) *reinterpret_cast<float4 *>(d) = make_float4(v[0], v[1], v[2], v[3]);
    else
      for (int j = 0; j < left; ++j) d[j] = v[j];
    return;
  }
  if (p.epi == EPI_RELU2 || p.epi == EPI_RELU2_FP8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = v[j] < 0.f ? 0.f : v[j];  // NaN stays
      v[j] = t * t;
    }
  } else if (p.epi == EPI_SOFTCAP) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = softcap8(v[j]);
  }
  if (p.epi == EPI_RELU2_FP8) {
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) a = fmaxf(a, v[j]);
    a = warp_max(a);
    const fp8::Quant z(a);
    const float f = z.inv, pre = z.pre;
    const uint32_t c = fp8::cvt2(v[0] * pre * f, v[1] * pre * f) | (fp8::cvt2(v[2] * pre * f, v[3] * pre * f) << 16);
    uint8_t *d = reinterpret_cast<uint8_t *>(p.D) + (int64_t)m * p.ldd + n;
    if (left >= 4) *reinterpret_cast<uint32_t *>(d) = c;
    else
      for (int j = 0; j < left; ++j) d[j] = (uint8_t)(c >> (8 * j));
    if (lane == 0) p.sd[(int64_t)(n >> 7) * p.lsd + m] = __fdiv_rn(a, fp8::kMax);
    return;
  }
  bf16 *d = reinterpret_cast<bf16 *>(p.D) + (int64_t)m * p.ldd + n;
  if (left >= 4) {
    if (p.epi == EPI_ADD) {
      float old[4];
      Vec4<bf16>::load(d, old);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += old[j];
    }
    Vec4<bf16>::store(d, v);
  } else {
    for (int j = 0; j < left; ++j)
      d[j] = __float2bfloat16_rn(p.epi == EPI_ADD ? __bfloat162float(d[j]) + v[j] : v[j]);
  }
}

template <int TN>
__global__ void __launch_bounds__(RowsCfg<TN>::kThreads, 2)
    gemm_fp8_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                         const RowsParams p) {
  using Cfg = RowsCfg<TN>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs, COLS = Cfg::kCols;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *scales = reinterpret_cast<float *>(smem + S * Cfg::kStageBytes);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S * Cfg::kStageBytes + Cfg::kScaleBytes);
  // bars: full[S], empty[S], tfull[NA], tempty[NA], drain
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 2 * NA + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert((2 * S + 2 * NA + 1) * 8 + 8 <= 256, "barriers, TMEM slot and abort flag fit their 256 bytes");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + S + s); };
  auto tfull_bar = [&](int a) { return smem_u32(bars + 2 * S + a); };
  auto tempty_bar = [&](int a) { return smem_u32(bars + 2 * S + NA + a); };
  const uint32_t drain_bar = smem_u32(bars + 2 * S + 2 * NA);
  const int m0 = (int)(blockIdx.x % p.n_m) * TN;
  const int nb = blockIdx.x / p.n_m;
  const int n0 = nb * 128;
  const int kb0 = 0, kb1 = p.kblocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < NA; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), Cfg::kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait<true>(empty_bar(stage), phase ^ 1, abort_flag, p.status)) break;
        const uint32_t sw = smem_u32(smem + stage * Cfg::kStageBytes);
        mbar_expect_tx(full_bar(stage), Cfg::kStageBytes);
        tma_load_2d(sw, &map_w, kb * BK, n0, full_bar(stage));
        tma_load_2d(sw + 128 * BK, &map_x, kb * BK, m0, full_bar(stage));
        ++issued;
        if (++stage == S) { stage = 0; phase ^= 1; }
      }
      // no copy of ours may still be landing when the CTA exits (bounded)
      for (int i = 0; i < min(issued, S); ++i) {
        if (--stage < 0) { stage = S - 1; phase ^= 1; }
        const uint64_t t0 = globaltimer();
        while (!mbar_try(full_bar(stage), phase) && globaltimer() - t0 < kWaitNs) {}
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      const uint32_t idesc = idesc8(128, TN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait<true>(tempty_bar(acc), acc_phase ^ 1, abort_flag, p.status)) break;
        if (!mbar_wait<true>(full_bar(stage), phase, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t sw = smem_u32(smem + stage * Cfg::kStageBytes);
        const uint32_t sx = sw + 128 * BK;
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          mma8(tmem_base + acc * TN, smem_desc(sw + kk * 32, 16, 1024), smem_desc(sx + kk * 32, 16, 1024), idesc, kk > 0);
        tc_commit(empty_bar(stage));
        tc_commit(tfull_bar(acc));
        if (++stage == S) { stage = 0; phase ^= 1; }
        if (++acc == NA) { acc = 0; acc_phase ^= 1; }
      }
      // every MMA this thread issued has completed once the drain barrier flips
      tc_commit(drain_bar);
      const uint64_t t0 = globaltimer();
      while (!mbar_try(drain_bar, 0) && globaltimer() - t0 < kWaitNs) {}
    }
  } else {
    // ---------------- sums over the K blocks ----------------
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;         // weight row of the tile
    const int c0 = ((warp - 2) >> 2) * COLS;     // first activation row of this warp
    float *sw = scales + (warp - 2) * COLS;      // this warp's copy of its rows' scales
    uint64_t sum[COLS / 2];
#pragma unroll
    for (int i = 0; i < COLS / 2; ++i) sum[i] = 0;
    // lane l fetches the scales of activation rows l, l + 32, one K block ahead
    constexpr int NS = (COLS + 31) / 32;
    auto fetch = [&](int kb, float (&f)[NS]) {
      const float wb = kb < kb1 ? p.sb[(int64_t)nb * p.lsb + kb] : 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int c = lane + 32 * i, m = m0 + c0 + c;
        f[i] = (kb < kb1 && c < COLS && m < p.M) ? p.sa[(int64_t)kb * p.lsa + m] * wb : 0.f;
      }
    };
    float next[NS];
    fetch(kb0, next);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      __syncwarp();  // the previous block's scales have been read
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (lane + 32 * i < COLS) sw[lane + 32 * i] = next[i];
      __syncwarp();
      fetch(kb + 1, next);
      const bool ok = mbar_wait<true>(tfull_bar(acc), acc_phase, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t t = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * TN + c0;
#pragma unroll
      for (int c = 0; c < COLS; c += 16) {
        uint32_t v[16];
        tmem_ld16_nw(t + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(sw + c + j);
          sum[(c + j) / 2] = fma2(f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2(f.x, f.y), sum[(c + j) / 2]);
          sum[(c + j) / 2 + 1] =
              fma2(f2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), f2(f.z, f.w), sum[(c + j) / 2 + 1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
      if (++acc == NA) { acc = 0; acc_phase ^= 1; }
    }
    // The last accumulator is complete, so every MMA has read the ring and
    // every copy has landed: the ring's memory takes the sums, [activation
    // row][weight row].  After an abort a copy may still land: no sums then.
    if (!*abort_flag) {
      float *red = reinterpret_cast<float *>(smem);
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) {
        float lo, hi;
        f2split(sum[i], lo, hi);
        red[(c0 + 2 * i) * 128 + row] = lo;
        red[(c0 + 2 * i + 1) * 128 + row] = hi;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::kTmemCols);
  // one warp per activation row: 128 weight rows are one 1 x 128 output block
  for (int c = warp; c < TN && m0 + c < p.M; c += Cfg::kThreads / 32) {
    const float4 f = *reinterpret_cast<const float4 *>(smem + (c * 128 + lane * 4) * 4);
    float v[4] = {f.x, f.y, f.z, f.w};
    rows_store(p, m0 + c, n0 + lane * 4, v, lane);
  }
}

// ------------------------------- host side -------------------------------

// 2D map over row-major bytes [rows, cols] with row stride ld, 128-byte swizzle
inline bool make_map8(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN>
inline cudaError_t launch_rows(const GemmFp8Problem &g, int *status, cudaStream_t st) {
  using Cfg = RowsCfg<TN>;
  CUtensorMap mw, mx;
  if (!make_map8(&mw, g.B, g.N, g.K, g.ldb, 128) || !make_map8(&mx, g.A, g.M, g.K, g.lda, TN)) return cudaErrorInvalidValue;
  RowsParams p;
  p.M = g.M; p.N = g.N; p.kblocks = (g.K + BK - 1) / BK;
  p.n_m = (g.M + TN - 1) / TN;
  p.n_n = (g.N + 127) / 128;
  p.sa = g.sa; p.lsa = g.lsa; p.sb = g.sb; p.lsb = g.lsb;
  p.D = g.D; p.ldd = g.ldd; p.sd = g.sd; p.lsd = g.lsd; p.epi = g.epi; p.status = status;
  if ((int64_t)p.n_m * p.n_n > INT32_MAX) return cudaErrorInvalidValue;
  gemm_fp8_rows_kernel<TN><<<p.n_m * p.n_n, Cfg::kThreads, Cfg::kSmem, st>>>(mw, mx, p);
  return cudaGetLastError();
}

inline cudaError_t init() {
  cudaError_t e = tc_init();
  auto big = [&](auto *k, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  big(gemm_fp8_rows_kernel<16>, RowsCfg<16>::kSmem);
  big(gemm_fp8_rows_kernel<32>, RowsCfg<32>::kSmem);
  big(gemm_fp8_rows_kernel<64>, RowsCfg<64>::kSmem);
  big(gemm_fp8_rows_kernel<128>, RowsCfg<128>::kSmem);
  return e;
}

}  // namespace tc8

inline cudaError_t launch_gemm_fp8(const GemmFp8Problem &g, int num_sms, int *status, cudaStream_t st) {
  (void)num_sms;
  if (g.M <= 16) return tc8::launch_rows<16>(g, status, st);
  if (g.M <= 32) return tc8::launch_rows<32>(g, status, st);
  if (g.M <= 64) return tc8::launch_rows<64>(g, status, st);
  return tc8::launch_rows<128>(g, status, st);
}

}  // namespace nc
