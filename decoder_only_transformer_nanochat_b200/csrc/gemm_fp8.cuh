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
#include "fp8_plan.h"
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
// Bounded wait for barriers that are handed over every K block: a count of
// tries is the limit, which costs the callers one register where a clock would
// cost several.  A try gives up after 4 us (measured: 50,176 of them in 200 ms), so
// 2^20 of them are four seconds without progress.
constexpr uint32_t kTries = 1u << 20;
__device__ __forceinline__ bool wait8(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status,
                                      uint32_t tries = kTries) {
  for (uint32_t i = 1; !mbar_try(bar, parity); ++i) {
    if ((i & 255) == 0 && (*abort_flag || i > tries)) {
      if (!*abort_flag) {
        *abort_flag = 1;
        set_status(status, kStatusTimeout);
      }
      return false;
    }
  }
  return true;
}

// The warps that issue TMA and MMAs stay converged and one elected lane
// issues, so descriptors and addresses are computed in uniform registers: four
// MMAs then issue in 58 cycles, against 310 from a branch that one lane took alone.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}
__device__ __forceinline__ void tmem_ld16_nw(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// the wait for those loads; the registers pass through it, so nothing that uses them can move above
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// relu that keeps a NaN
__device__ __forceinline__ float relu_nan(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// 15 tanh(z / 15) to 2^-15 of its value: t = (1 - E) / (1 + E), E = exp(-2 |z| / 15),
// off by the error of E, up to 2^-22, against 1 - E; z itself up to |z| = 0.09,
// where tanh's next term is 2^-16.3 and 1 - E has fallen to 2^-6.4.  (tanh's
// series to 2^-21 below 15 / 4 instead: 265 us against 238 at 2048 x 65,536 x 1280.)
__device__ __forceinline__ float softcap8(float z) {
  const float e = __expf(-2.f / kSoftcap * fabsf(z));
  const float t = copysignf(kSoftcap * __fdividef(1.f - e, 1.f + e), z);
  return fabsf(z) < 0.09f ? z : t;
}

// ===========================================================================
// Few rows (or few tiles): the weights are the M = 128 operand of the tensor core and TN
// activation rows the N operand, so one decoded token costs an N = 16 tile
// instead of a 128-row one.
//
// Roles: warp 0 TMA, warp 1 MMA, the others add up (thread = weight row, up
// to 64 activation rows in registers).
//
// Few tiles leave SMs idle, so K is cut over a cluster of 1, 2, 4 or 8 CTAs.
// Each owns TN / splits of the activation rows and receives the others' sums
// for them in its shared memory; after one cluster barrier it adds them in
// rank order (the bits do not depend on which CTA ends first) and stores.
//
// Measured: one row x 1536 x 1280 3.4 us in a graph (launch, set-up, one load and
// one cluster barrier; the weights alone would take 0.3); 16 rows x 65,536 x
// 1280 17.7 us in a row of calls, 4.9 TB/s.  The sums are 4-byte stores to the owner because a
// pull needs a second cluster barrier (one row 6.5 us, pushed 5.4).
//
// kMany: more tiles than two CTAs per SM hold at once (the logits of a few
// rows), so K is not cut; four smaller CTAs per SM then keep every tile's
// loads in flight from the start.
template <int TN, bool kMany> struct RowsCfg {
  static constexpr int kEpiWarps = TN > 64 ? 8 : 4;        // 4 cover the 128 TMEM lanes; 8: two column halves
  static constexpr int kCols = TN * 4 / kEpiWarps;         // activation rows per thread
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kStageBytes = (128 + TN) * BK;
  static constexpr int kCtas = rows_ctas(TN, kMany);       // per SM
  static constexpr int kStages = kMany ? 3 : TN == 16 ? 5 : TN == 64 ? 3 : 4;
  static constexpr int kAccs = 4;                          // TMEM accumulators in flight
  static constexpr int kTmemCols = kAccs * TN;             // 64, 128, 256, 512: a power of two
  static constexpr int kScaleBytes = kEpiWarps * kCols * 4;
  // the cluster's sums of this CTA's activation rows; without a cluster they take the ring's memory
  static constexpr int kSumBytes = kMany ? 0 : TN * 128 * 4;
  static constexpr int kSmem = kStages * kStageBytes + kSumBytes + kScaleBytes + 256 + 1024;
  static_assert(!kMany || TN * 128 * 4 <= kStages * kStageBytes, "the sums fit the ring");
  // no more CTAs fit an SM than its TMEM serves: an allocation never waits for another CTA's
  static_assert(kCtas * (kSmem + 1024) <= 233472 && (kCtas + 1) * (kSmem + 1024) > 233472 && kCtas * kTmemCols <= 512,
                "CTAs per SM");
};

// Where a product goes
struct Out {
  int M, N;
  void *D;
  int64_t ldd;
  float *sd;
  int64_t lsd;
};

struct RowsParams {
  Out out;
  int kblocks;
  int n_m, splits;      // CTAs per cluster
  const float *sa, *sb;
  int64_t lsa, lsb;
  int epi;
  int *status;
};

// Epilogue of a warp that holds one row m of a 128-column block, four columns
// [n, n + 4) a lane: v = sums
__device__ __forceinline__ void store_block_row(const Out &p, int epi, int m, int n, float (&v)[4], int lane) {
  const int left = p.N - n;  // <= 0: nothing to store (the lane still takes part in the block's maximum)
  if (epi == EPI_STORE_F32) {
    float *d = reinterpret_cast<float *>(p.D) + (int64_t)m * p.ldd + n;
    if (left >= 4) *reinterpret_cast<float4 *>(d) = make_float4(v[0], v[1], v[2], v[3]);
    else
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < left) d[j] = v[j];
    return;
  }
  if (epi == EPI_RELU2 || epi == EPI_RELU2_FP8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = relu_nan(v[j]);
      v[j] *= v[j];
    }
  } else if (epi == EPI_SOFTCAP) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = softcap8(v[j]);
  }
  if (epi == EPI_RELU2_FP8) {
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) a = fmaxf(a, v[j]);
    a = warp_max(a);
    const uint32_t c = fp8::Ratio(a).codes4(f2(v[0], v[1]), f2(v[2], v[3]));
    uint8_t *d = reinterpret_cast<uint8_t *>(p.D) + (int64_t)m * p.ldd + n;
    if (left >= 4) *reinterpret_cast<uint32_t *>(d) = c;
    else
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < left) d[j] = (uint8_t)(c >> (8 * j));
    if (lane == 0) p.sd[(int64_t)(n >> 7) * p.lsd + m] = __fdiv_rn(a, fp8::kMax);
    return;
  }
  bf16 *d = reinterpret_cast<bf16 *>(p.D) + (int64_t)m * p.ldd + n;
  if (left >= 4) {
    if (epi == EPI_ADD) {
      float old[4];
      Vec4<bf16>::load(d, old);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += old[j];
    }
    Vec4<bf16>::store(d, v);
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < left) d[j] = __float2bfloat16_rn(epi == EPI_ADD ? __bfloat162float(d[j]) + v[j] : v[j]);
  }
}

__device__ __forceinline__ void cluster_started(int splits) {
  if (splits > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <int TN, bool kMany>
__global__ void __launch_bounds__(RowsCfg<TN, kMany>::kThreads, RowsCfg<TN, kMany>::kCtas)
    gemm_fp8_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                         const RowsParams p) {
  using Cfg = RowsCfg<TN, kMany>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs, COLS = Cfg::kCols;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *sums = reinterpret_cast<float *>(smem + (kMany ? 0 : S * Cfg::kStageBytes));  // [splits][TN / splits][128]
  float *scales = reinterpret_cast<float *>(smem + S * Cfg::kStageBytes + Cfg::kSumBytes);
  uint64_t *bars = reinterpret_cast<uint64_t *>(scales + Cfg::kScaleBytes / 4);
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
  // tiles of one weight row block are neighbours, so its panel is read from L2 after the first
  const int rank = (int)(blockIdx.x % p.splits), tile = blockIdx.x / p.splits;
  const int m0 = tile % p.n_m * TN;
  const int nb = tile / p.n_m;
  const int n0 = nb * 128;
  const int kb0 = (int)((int64_t)p.kblocks * rank / p.splits), kb1 = (int)((int64_t)p.kblocks * (rank + 1) / p.splits);
  const uint32_t elected = warp < 2 ? elect_one() : 0;

  // waited for before the first store to another CTA: it has started by then
  if (p.splits > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (warp == 0) {
    if (elected) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
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
      // the ring's first loads need nothing that the other warps set up
      fp8::pdl_wait();
      for (int s = 0; s < min(S, kb1 - kb0); ++s) {
        const uint32_t sw = smem_u32(smem + s * Cfg::kStageBytes);
        mbar_expect_tx(full_bar(s), Cfg::kStageBytes);
        tma_load_2d(sw, &map_w, (kb0 + s) * BK, n0, full_bar(s));
        tma_load_2d(sw + 128 * BK, &map_x, (kb0 + s) * BK, m0, full_bar(s));
      }
    }
    __syncwarp();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  fp8::pdl_start();  // only now: a successor's CTA that waits for this grid must not hold the TMEM that this one needs
  fp8::pdl_wait();

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    int stage = 0, issued = min(S, kb1 - kb0);
    uint32_t phase = 1;
    if (issued < S) { stage = issued; phase = 0; }
    for (int kb = kb0 + S; kb < kb1; ++kb) {
      const bool ok = wait8(empty_bar(stage), phase ^ 1, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t sw = smem_u32(smem + stage * Cfg::kStageBytes);
      if (elected) {
        mbar_expect_tx(full_bar(stage), Cfg::kStageBytes);
        tma_load_2d(sw, &map_w, kb * BK, n0, full_bar(stage));
        tma_load_2d(sw + 128 * BK, &map_x, kb * BK, m0, full_bar(stage));
      }
      __syncwarp();
      if (++stage == S) { stage = 0; phase ^= 1; }
    }
    cluster_started(p.splits);
    // no copy of ours may still be landing when the CTA exits (bounded)
    for (int i = 0; i < issued; ++i) {
      if (--stage < 0) { stage = S - 1; phase ^= 1; }
      const uint64_t t0 = globaltimer();
      while (!mbar_try(full_bar(stage), phase) && globaltimer() - t0 < kWaitNs) {}
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    const uint32_t idesc = idesc8(128, TN);
    const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      const bool ok = wait8(tempty_bar(acc), acc_phase ^ 1, abort_flag, p.status) &&
                      wait8(full_bar(stage), phase, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint64_t wd = desc0 + (uint64_t)(stage * (Cfg::kStageBytes >> 4)), xd = wd + (128 * BK >> 4);
      if (elected) {
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) mma8(tmem_base + acc * TN, wd + 2 * kk, xd + 2 * kk, idesc, kk > 0);
        tc_commit(tfull_bar(acc));
        tc_commit(empty_bar(stage));
      }
      __syncwarp();
      if (++stage == S) { stage = 0; phase ^= 1; }
      if (++acc == NA) { acc = 0; acc_phase ^= 1; }
    }
    cluster_started(p.splits);
    // every MMA issued has completed once the drain barrier flips
    if (elected) {
      tc_commit(drain_bar);
      const uint64_t t0 = globaltimer();
      while (!mbar_try(drain_bar, 0) && globaltimer() - t0 < kWaitNs) {}
    }
    __syncwarp();
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
    float fa[NS], fb = 0.f;
    auto fetch = [&](int kb) {
      fb = p.sb[(int64_t)nb * p.lsb + kb];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int c = lane + 32 * i, m = m0 + c0 + c;
        fa[i] = (c < COLS && m < p.out.M) ? p.sa[(int64_t)kb * p.lsa + m] : 0.f;
      }
    };
    if (kb0 < kb1) fetch(kb0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      __syncwarp();  // the previous block's scales have been read
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (lane + 32 * i < COLS) sw[lane + 32 * i] = fa[i] * fb;
      __syncwarp();
      if (kb + 1 < kb1) fetch(kb + 1);
      const bool ok = wait8(tfull_bar(acc), acc_phase, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t t = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * TN + c0;
      uint32_t v[COLS / 16][16];
#pragma unroll
      for (int c = 0; c < COLS / 16; ++c) tmem_ld16_nw(t + 16 * c, v[c]);
#pragma unroll
      for (int c = 0; c < COLS / 16; ++c) tmem_wait16(v[c]);  // the first waits for all
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
#pragma unroll
      for (int c = 0; c < COLS / 16; ++c)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(sw + 16 * c + j);
          uint64_t *o = sum + 8 * c + j / 2;
          o[0] = fma2(f2(__uint_as_float(v[c][j]), __uint_as_float(v[c][j + 1])), f2(f.x, f.y), o[0]);
          o[1] = fma2(f2(__uint_as_float(v[c][j + 2]), __uint_as_float(v[c][j + 3])), f2(f.z, f.w), o[1]);
        }
      if (++acc == NA) { acc = 0; acc_phase ^= 1; }
    }
    if constexpr (kMany) {
      // The last accumulator is complete, so every MMA has read the ring and
      // every copy has landed; after an abort one may not have: no sums then.
      if (!*abort_flag) {
#pragma unroll
        for (int i = 0; i < COLS; ++i) {
          float lo, hi;
          f2split(sum[i / 2], lo, hi);
          sums[(c0 + i) * 128 + row] = (i & 1) ? hi : lo;
        }
      }
    } else {
      cluster_started(p.splits);
      // to the CTA that owns the activation row
      const int per = TN / p.splits;  // a power of two
      const int shift = 31 - __clz(per);
      const uint32_t to = smem_u32(sums) + (rank * per * 128 + row) * 4;
#pragma unroll
      for (int i = 0; i < COLS; ++i) {
        const int c = c0 + i;
        if (m0 + c < p.out.M) {
          float lo, hi;
          f2split(sum[i / 2], lo, hi);
          st_cluster(cluster_addr(to + (c & (per - 1)) * 512, c >> shift), (i & 1) ? hi : lo);
        }
      }
    }
  }
  tc_fence_before();
  if (p.splits > 1) cluster_sync_all();  // the cluster's sums have arrived
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::kTmemCols);
  // one warp per activation row: 128 weight rows are one 1 x 128 output block
  const int per = TN / p.splits;
  for (int c = warp; c < per && m0 + rank * per + c < p.out.M; c += Cfg::kThreads / 32) {
    const float *at = sums + c * 128 + lane * 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int r = 0; r < p.splits; ++r) {
      const float4 f = *reinterpret_cast<const float4 *>(at + r * per * 128);
      v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    }
    store_block_row(p.out, p.epi, m0 + rank * per + c, n0 + lane * 4, v, lane);
  }
}

// ===========================================================================
// Many rows: a pair of CTAs (cta_group::2) on neighbouring SMs takes a
// 256 x 256 tile, as the bf16 GEMM's pair kernel does (gemm_tc.cuh): CTA r
// holds tile rows [128 r, 128 r + 128) of A and of the accumulator and loads
// half of B; the leader (r = 0) issues every MMA.  Persistent, one CTA per SM.
//
// TMEM holds two 256-column accumulators, one K block each, in halves of 128
// columns that are handed over one by one: a warp of its own issues each half's
// MMAs, and four epilogue warps per CTA scale and add it into fp32 sums in
// registers (thread = one row x 128 columns: one weight block, so one scale per
// thread and K block).
// A thread's 128 columns are also one 1 x 128 output block, so the 8-bit
// epilogue finds its maximum without leaving the thread.
//
// What bounds it: an accumulator's way round.  A K block takes about 900 cycles
// where its MMAs take 512 (short runs: 16384 x 2048 x 8192 with the residual add
// 248 us, 2.22 PFLOP/s; 32768 x 5120 x 1280 with relu^2 to 8 bits 228 us, 1.88;
// long ones, under the power cap, 289 and 267 us); the loop without sums, one
// hand-over a tile, runs at 180 us and 3.06 PFLOP/s.  Two accumulators are all
// that TMEM holds at this tile; smaller tiles were not measured.  Handing over
// whole accumulators measured 274 us, sixteen epilogue warps of 64 columns 7 %
// more than eight.
//
// Few tiles leave SMs idle, so K is cut over the pairs of a larger cluster (2
// or 4): each CTA then leaves its sums in its ring's memory and adds, for its
// part of the rows, those of the cluster's pairs in order.
//
// Each epilogue warp stages its 32 rows x 128 columns alone, in two boxes of
// 32 rows x 128 bytes (128-byte swizzle) that leave by TMA; an epilogue that
// adds to D has them loaded while the K loop runs.
constexpr int PSTAGES = 5;
constexpr int PSTAGE_BYTES = 2 * 128 * BK;  // A and B rows of one CTA: 32 KB
constexpr int PEPI_WARPS = 8;
// Three warpgroups: warp 0 TMA, warps 1 and 2 MMA (warp 3 idle), warps 4..11 the
// epilogue, which holds 128 sums a thread.  The first gives registers to the
// others: 128 x 24 + 256 x 240 = 64,512, all of the 384 x 168 of the launch
// (init() checks that count), so every increase can be met.
constexpr int PTHREADS = 128 + 32 * PEPI_WARPS;
constexpr int PREGS = 168, PREGS_LOW = 24, PREGS_HIGH = 240;
static_assert(128 * PREGS_LOW + 32 * PEPI_WARPS * PREGS_HIGH <= PTHREADS * PREGS, "register split within the launch");
constexpr int PSPLITS = kMaxPairSplits;
constexpr int PBOX = 32 * 128;
constexpr int PSMEM = PSTAGES * PSTAGE_BYTES + PEPI_WARPS * 2 * PBOX + 256 + 1024;
static_assert(PSMEM <= 232448, "shared memory per CTA");
static_assert(128 * 256 * 4 <= PSTAGES * PSTAGE_BYTES, "a split's sums fit the ring");

// A TMA store writes whole 16-byte units of a row (measured: one byte per
// element, N % 16 == 8, wrote eight bytes past N), so the map of D ends at the
// last whole unit, column n_tma, and the threads take the rest of their row.
struct PairParams {
  Out out;
  PairTiles tiles;
  int kblocks, splits;  // pairs per cluster
  int units, n_tma;
  const float *sa, *sb;
  int64_t lsa, lsb;
  int *status;
};

// The columns [n_tma, N) of row m that lie in [n, n + width): from or to the
// warp's staged boxes (row at `my`, column n at byte 0), es bytes each.
template <bool kLoad, typename E>
__device__ __forceinline__ void pair_tail(const PairParams &p, uint8_t *my, int lane, int m, int n, int width) {
  if (m >= p.out.M) return;
  for (int c = max(p.n_tma, n); c < min(p.out.N, n + width); ++c) {
    const int b = (c - n) * (int)sizeof(E);
    E *e = reinterpret_cast<E *>(my + (b >> 7) * PBOX + ((((b >> 4) & 7) ^ (lane & 7)) << 4) + (b & 15));
    E *d = reinterpret_cast<E *>(p.out.D) + (int64_t)m * p.out.ldd + c;
    if (kLoad) *e = *d;
    else *d = *e;
  }
}

// the wait for two tmem_ld32_nw; their registers pass through it
__device__ __forceinline__ void tmem_wait32(uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]), "+r"(a[21]), "+r"(a[22]), "+r"(a[23]),
                 "+r"(a[24]), "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]), "+r"(a[30]), "+r"(a[31])::"memory");
  asm volatile(""
               : "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                 "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15]),
                 "+r"(b[16]), "+r"(b[17]), "+r"(b[18]), "+r"(b[19]), "+r"(b[20]), "+r"(b[21]), "+r"(b[22]), "+r"(b[23]),
                 "+r"(b[24]), "+r"(b[25]), "+r"(b[26]), "+r"(b[27]), "+r"(b[28]), "+r"(b[29]), "+r"(b[30]), "+r"(b[31]));
}
// Arrive on a barrier of the cluster (shared::cluster address) without
// release semantics: what it hands over is TMEM whose reads have completed
// (tcgen05.wait::ld returned their values).  A releasing arrive at cluster
// scope first waits for the thread's global loads (the scales fetched ahead):
// measured 596 against 341 us at 16384 x 2048 x 8192.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

__device__ __forceinline__ void mma8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int EPI>
__global__ void __launch_bounds__(PTHREADS, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap map_d, const PairParams p) {
  constexpr int S = PSTAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *staging = smem + S * PSTAGE_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(staging + PEPI_WARPS * 2 * PBOX);
  // bars: full[S], done[2 S], tempty[4], drain, aux[PEPI_WARPS]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 3 * S + 5 + PEPI_WARPS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert((3 * S + 5 + PEPI_WARPS) * 8 + 8 <= 256, "barriers, TMEM slot and abort flag fit their 256 bytes");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a cluster holds `splits` pairs; each takes its part of K of the same tile
  const uint32_t cta = cluster_rank(), lead = cta & ~1u, rank = cta & 1;
  const bool leader = rank == 0;
  const uint16_t both = (uint16_t)(0x3 << lead);
  const int cluster = blockIdx.x / (2 * p.splits), n_clusters = gridDim.x / (2 * p.splits);
  const int split = (int)(cta >> 1);
  const int kb0 = (int)((int64_t)p.kblocks * split / p.splits);
  const int kb1 = (int)((int64_t)p.kblocks * (split + 1) / p.splits);
  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  // done[s, h]: the MMAs of stage s and column half h are complete, so that
  // half of its accumulator is full, and with both the stage is free.
  // (The epilogue cannot miss a phase: the stage's next MMAs wait for an
  // accumulator that it has yet to hand back.)
  auto done_bar = [&](int s, int h) { return smem_u32(bars + S + 2 * s + h); };
  auto tempty_bar = [&](int a) { return smem_u32(bars + 3 * S + a); };
  const uint32_t drain_bar = smem_u32(bars + 3 * S + 4);
  auto aux_bar = [&](int w) { return smem_u32(bars + 3 * S + 5 + w); };

  if (threadIdx.x == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_d)) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(done_bar(s, 0), 1);
      mbar_init(done_bar(s, 1), 1);
    }
    for (int a = 0; a < 4; ++a) mbar_init(tempty_bar(a), PEPI_WARPS);  // a column half's epilogue warps of both CTAs
    mbar_init(drain_bar, 2);  // both MMA warps
    for (int w = 0; w < PEPI_WARPS; ++w) mbar_init(aux_bar(w), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  fp8::pdl_start();  // only now: a successor's CTA that waits for this grid must not hold the TMEM that this one needs
  fp8::pdl_wait();

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PREGS_LOW));
  if (warp == 0) {
    // ---------------- TMA producer ----------------
    const uint32_t elected = elect_one();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = cluster; u < p.units && ok; u += n_clusters) {
      int m_blk, n_blk;
      p.tiles.tile(u, m_blk, n_blk);
      const int m_row = m_blk * 256 + (int)rank * 128, n_row = n_blk * 256 + (int)rank * 64;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(0xffffffffu, wait8(done_bar(stage, 0), phase ^ 1, abort_flag, p.status) &&
                                         wait8(done_bar(stage, 1), phase ^ 1, abort_flag, p.status));
        if (!ok) break;
        const uint32_t sa = smem_u32(smem + stage * PSTAGE_BYTES);
        const uint32_t fb = cluster_addr(full_bar(stage), lead);
        if (elected) {
          if (leader) mbar_expect_tx(full_bar(stage), 2 * PSTAGE_BYTES);
          tma_load_2d_pair(sa, &map_a, kb * BK, m_row, fb);
          // this CTA's half of each column half: an MMA of N = 128 takes 64 rows of B from each CTA
          tma_load_2d_pair(sa + 128 * BK, &map_b, kb * BK, n_row, fb);
          tma_load_2d_pair(sa + 192 * BK, &map_b, kb * BK, n_row + 128, fb);
        }
        __syncwarp();
        issued = min(issued + 1, S);
        if (++stage == S) { stage = 0; phase ^= 1; }
      }
    }
    // both CTAs' copies count on the leader's barriers: it sees them landed
    // (bounded) before the next cluster barrier
    if (leader)
      for (int i = 0; i < issued; ++i) {
        if (--stage < 0) { stage = S - 1; phase ^= 1; }
        const uint64_t t0 = globaltimer();
        while (!mbar_try(full_bar(stage), phase) && globaltimer() - t0 < kWaitNs) {}
      }
    __syncwarp();
  } else if (warp <= 2) {
    if (leader) {
      // ---------------- MMA issuers: warp 1 the left column half, warp 2 the right ----------------
      const int half = warp - 1;
      const uint32_t idesc = idesc8(256, 128);
      const uint32_t elected = elect_one();
      const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024);
      const uint32_t d0 = tmem_base + half * 128;
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = cluster; u < p.units && ok; u += n_clusters) {
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = __all_sync(0xffffffffu, wait8(full_bar(stage), phase, abort_flag, p.status) &&
                                           wait8(tempty_bar(2 * acc + half), acc_phase ^ 1, abort_flag, p.status));
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = desc0 + (uint64_t)(stage * (PSTAGE_BYTES >> 4)), bd = ad + ((128 + 64 * half) * BK >> 4);
          if (elected) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk) mma8_pair(d0 + acc * 256, ad + 2 * kk, bd + 2 * kk, idesc, kk > 0);
            tc_commit_pair(done_bar(stage, half), both);
          }
          __syncwarp();
          if (++stage == S) { stage = 0; phase ^= 1; }
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
      }
      if (elected) {
        tc_commit_pair(drain_bar, (uint16_t)(1 << lead));
        const uint64_t t0 = globaltimer();
        while (!mbar_try(drain_bar, 0) && globaltimer() - t0 < kWaitNs) {}
      }
      __syncwarp();
    }
  }
  if (p.splits > 1) cluster_sync_all();  // the split sums (below)
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PREGS_HIGH));
    // ---------------- epilogue warps 4..11 (both CTAs) ----------------
    const int quarter = warp & 3;
    const int cg = (warp - 4) >> 2;  // columns [128 cg, 128 cg + 128) of the tile
    const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + cg * 128;
    uint8_t *const box = staging + (warp - 4) * 2 * PBOX;
    uint8_t *const my = box + lane * 128;  // 16-byte unit u of this row's 128 bytes sits at u ^ (row % 8)
    const uint32_t aux = aux_bar(warp - 4);
    uint32_t aux_phase = 0;
    bool aux_inflight = false;
    int acc = 0, stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t tempty0 = cluster_addr(tempty_bar(cg), lead);
    // This thread's two scales of AHEAD K blocks, fetched together while those
    // of the AHEAD before are used (a wait for the older of outstanding loads
    // would be one for the newer too).  Rows and columns outside the matrix
    // take the scales of the last one inside; they are not stored.
    // us at 16384 x 2048 x 8192: 2 262, 3 252, 4 248, 5 246, 6 262.  At 5 the kernel
    // spills four to seven registers, outside the loop over the K blocks' columns.
    constexpr int AHEAD = 5;
    float fa[AHEAD], fb[AHEAD];
    const float *pa = nullptr, *pb = nullptr;
    auto fetch = [&](int kb) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int k = min(kb + i, kb1 - 1);
        fa[i] = pa[k * p.lsa];
        fb[i] = pb[k];
      }
    };
    auto first_scales = [&](int u) {
      int m_blk, n_blk;
      p.tiles.tile(u, m_blk, n_blk);
      pa = p.sa + min(m_blk * 256 + (int)rank * 128 + quarter * 32 + lane, p.out.M - 1);
      pb = p.sb + (int64_t)min(n_blk * 2 + cg, (p.out.N - 1) >> 7) * p.lsb;
      fetch(kb0);
    };
    auto wait_done = [&]() {
      const bool r = __all_sync(0xffffffffu, wait8(done_bar(stage, cg), phase, abort_flag, p.status));
      tc_fence_after();
      return r;
    };
    if (cluster < p.units) first_scales(cluster);
    for (int u = cluster; u < p.units; u += n_clusters) {
      int m_blk, n_blk;
      p.tiles.tile(u, m_blk, n_blk);
      const int mw = m_blk * 256 + (int)rank * 128 + quarter * 32;  // this warp's first row
      const int n0 = n_blk * 256 + cg * 128;
      const bool mine = mw < p.out.M && n0 < p.out.N;
      const bool by_tma = n0 < p.n_tma, two = n0 + 64 < p.n_tma;
      if (EPI == EPI_ADD && p.splits == 1 && mine && by_tma && lane == 0) {
        bulk_wait_read0();  // the previous tile's stores have read the boxes
        mbar_expect_tx(aux, two ? 2 * PBOX : PBOX);
        tma_load_2d(smem_u32(box), &map_d, n0, mw, aux);
        if (two) tma_load_2d(smem_u32(box) + PBOX, &map_d, n0 + 64, mw, aux);
        aux_inflight = true;
      }
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      // Two 32-column loads are in flight at a time.
      uint32_t v0[32], v1[32];
      auto add = [&](uint32_t (&v)[32], int c, uint64_t f) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          sum[16 * c + j] = fma2(f2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), f, sum[16 * c + j]);
      };
      ok = wait_done();
      if (ok) {
        tmem_ld32_nw(t_row + acc * 256, v0);
        tmem_ld32_nw(t_row + acc * 256 + 32, v1);
      }
      for (int kp = kb0; kp < kb1 && ok; kp += AHEAD) {
        float sc[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) sc[i] = fa[i] * fb[i];
        if (kp + AHEAD < kb1) fetch(kp + AHEAD);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int kb = kp + i;
          if (kb >= kb1) break;
          const uint64_t f = f2(sc[i], sc[i]);
          tmem_wait32(v0, v1);
          add(v0, 0, f);
          tmem_ld32_nw(t_row + acc * 256 + 64, v0);
          add(v1, 1, f);
          tmem_ld32_nw(t_row + acc * 256 + 96, v1);
          tmem_wait32(v0, v1);
          tc_fence_before();
          __syncwarp();  // all lanes have read it: it goes back
          if (lane == 0) mbar_arrive_relaxed(tempty0 + acc * 16);
          acc ^= 1;
          if (++stage == S) { stage = 0; phase ^= 1; }
          // the rest of this block's work comes before the next one is looked
          // for: what lies between that and its hand-back is the way round
          add(v0, 2, f);
          add(v1, 3, f);
          if (kb + 1 < kb1) {
            ok = wait_done();
            if (!ok) break;
            tmem_ld32_nw(t_row + acc * 256, v0);
            tmem_ld32_nw(t_row + acc * 256 + 32, v1);
          }
        }
      }
      if (u + n_clusters < p.units) first_scales(u + n_clusters);
      if (!ok) break;
      if (p.splits > 1) {  // the cluster's only tile: its sums go to shared memory
        const int last = stage ? stage - 1 : S - 1;
        ok = __all_sync(0xffffffffu, wait8(done_bar(last, cg ^ 1), stage ? phase : phase ^ 1, abort_flag, p.status));
        if (!ok) break;
        // no MMA reads the ring and no copy is on its way to it any more
        const int row = quarter * 32 + lane;
        uint8_t *const to = smem + row * 1024;  // 16-byte unit u of a row sits at u ^ (row % 8)
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          float o[4];
          f2split(sum[2 * q], o[0], o[1]);
          f2split(sum[2 * q + 1], o[2], o[3]);
          *reinterpret_cast<float4 *>(to + (((cg * 32 + q) ^ (row & 7)) << 4)) = make_float4(o[0], o[1], o[2], o[3]);
        }
        break;
      }
      if (!mine) continue;
      if (EPI == EPI_ADD && by_tma) {
        ok = __all_sync(0xffffffffu, wait8(aux, aux_phase, abort_flag, p.status));
        if (!ok) break;
        aux_phase ^= 1;
        aux_inflight = false;
      } else {
        if (lane == 0) bulk_wait_read0();
        __syncwarp();
      }
      if constexpr (EPI == EPI_STORE_F32) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (b == 2) {
            if (lane == 0) bulk_wait_read0();
            __syncwarp();
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float o[4];
            f2split(sum[16 * b + 2 * q], o[0], o[1]);
            f2split(sum[16 * b + 2 * q + 1], o[2], o[3]);
            *reinterpret_cast<float4 *>(my + (b & 1) * PBOX + ((q ^ (lane & 7)) << 4)) = make_float4(o[0], o[1], o[2], o[3]);
          }
          if (b & 1) {
            const int n = n0 + (b - 1) * 32;
            pair_tail<false, float>(p, my, lane, mw + lane, n, 64);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              if (n < p.n_tma) tma_store_2d(&map_d, smem_u32(box), n, mw);
              if (n + 32 < p.n_tma) tma_store_2d(&map_d, smem_u32(box) + PBOX, n + 32, mw);
              bulk_commit();
            }
          }
        }
        continue;
      }
      if constexpr (EPI == EPI_RELU2_FP8) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float lo, hi;
          f2split(sum[i], lo, hi);
          sum[i] = f2(relu_nan(lo), relu_nan(hi));
          sum[i] = mul2(sum[i], sum[i]);
          f2split(sum[i], lo, hi);
          a = max3(a, lo, hi);
        }
        const fp8::Ratio z(a);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = z.codes4(sum[8 * q + 2 * j], sum[8 * q + 2 * j + 1]);
          *reinterpret_cast<uint4 *>(my + ((q ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        pair_tail<false, uint8_t>(p, my, lane, mw + lane, n0, 128);
        if (mw + lane < p.out.M) p.out.sd[(int64_t)(n0 >> 7) * p.out.lsd + mw + lane] = __fdiv_rn(a, fp8::kMax);
      } else {
        if (EPI == EPI_ADD) pair_tail<true, bf16>(p, my, lane, mw + lane, n0, 128);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          bf16 *d = reinterpret_cast<bf16 *>(my + (q >> 3) * PBOX + (((q & 7) ^ (lane & 7)) << 4));
          float o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) f2split(sum[4 * q + j], o[2 * j], o[2 * j + 1]);
          if (EPI == EPI_ADD) {
            float old[8];
            Vec8<bf16>::load(d, old);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += old[j];
          } else if (EPI == EPI_RELU2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[j] = relu_nan(o[j]);
              o[j] *= o[j];
            }
          } else if (EPI == EPI_SOFTCAP) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = softcap8(o[j]);
          }
          Vec8<bf16>::store(d, o);
        }
        pair_tail<false, bf16>(p, my, lane, mw + lane, n0, 128);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        if (by_tma) tma_store_2d(&map_d, smem_u32(box), n0, mw);
        if (EPI != EPI_RELU2_FP8 && two) tma_store_2d(&map_d, smem_u32(box) + PBOX, n0 + 64, mw);
        bulk_commit();
      }
    }
    if (p.splits > 1) {
      cluster_sync_all();  // every pair's sums are in shared memory
      // This CTA's part of its rows: one warp per row and 128-column block, the
      // pairs' sums added in order, four such rows' reads in flight.
      int m_blk, n_blk;
      p.tiles.tile(cluster, m_blk, n_blk);
      const int per = 128 / p.splits, first = m_blk * 256 + (int)rank * 128;
#pragma unroll 1
      for (int i0 = (warp - 4) * 4; i0 < 2 * per && ok; i0 += 4 * PEPI_WARPS) {
        float4 f[4][PSPLITS];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = split * per + ((i0 + q) >> 1), unit = ((i0 + q) & 1) * 32 + lane;
          const uint32_t at = smem_u32(smem) + row * 1024 + ((unit ^ (row & 7)) << 4);
#pragma unroll
          for (int r = 0; r < PSPLITS; ++r)
            if (r < p.splits) f[q][r] = ld_cluster(cluster_addr(at, 2 * r + rank));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = first + split * per + ((i0 + q) >> 1), n = n_blk * 256 + ((i0 + q) & 1) * 128;
          float v[4] = {f[q][0].x, f[q][0].y, f[q][0].z, f[q][0].w};
#pragma unroll
          for (int r = 1; r < PSPLITS; ++r)
            if (r < p.splits) { v[0] += f[q][r].x; v[1] += f[q][r].y; v[2] += f[q][r].z; v[3] += f[q][r].w; }
          if (m < p.out.M && n < p.out.N) store_block_row(p.out, EPI, m, n + lane * 4, v, lane);
        }
      }
    }
    if (lane == 0) {
      bulk_wait0();
      // only after an abort: a load of D that was never taken lands first (bounded)
      const uint64_t t0 = globaltimer();
      while (aux_inflight && !mbar_try(aux, aux_phase) && globaltimer() - t0 < kWaitNs) {}
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer can still signal or read it
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                 : "memory");
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

inline Out out_of(const GemmFp8Problem &g) { return Out{g.M, g.N, g.D, g.ldd, g.sd, g.lsd}; }

template <int TN, bool kMany>
inline cudaError_t launch_rows(const GemmFp8Problem &g, const Plan &plan, int *status, cudaStream_t st) {
  using Cfg = RowsCfg<TN, kMany>;
  CUtensorMap mw, mx;
  if (!make_map8(&mw, g.B, g.N, g.K, g.ldb, 128) || !make_map8(&mx, g.A, g.M, g.K, g.lda, TN)) return cudaErrorInvalidValue;
  RowsParams p;
  p.out = out_of(g);
  p.kblocks = (g.K + BK - 1) / BK;
  p.n_m = (g.M + TN - 1) / TN;
  p.sa = g.sa; p.lsa = g.lsa; p.sb = g.sb; p.lsb = g.lsb;
  p.epi = g.epi; p.status = status;
  p.splits = plan.splits;
  return fp8::launch(gemm_fp8_rows_kernel<TN, kMany>, (unsigned)(plan.tiles * p.splits), Cfg::kThreads, Cfg::kSmem, p.splits, st, mw,
                     mx, p);
}

inline cudaError_t launch_pair(const GemmFp8Problem &g, const Plan &plan, int num_sms, int *status, cudaStream_t st) {
  CUtensorMap ma, mb, md;
  bool ok = make_map8(&ma, g.A, g.M, g.K, g.lda, 128) && make_map8(&mb, g.B, g.N, g.K, g.ldb, 64);
  PairParams p{out_of(g), PairTiles((g.M + 255) / 256, (g.N + 255) / 256)};
  const int unit = g.epi == EPI_RELU2_FP8 ? 16 : g.epi == EPI_STORE_F32 ? 4 : 8;  // values in 16 bytes
  p.n_tma = g.N / unit * unit;
  const int64_t cols = max(p.n_tma, unit);  // a D narrower than a unit leaves without the map
  if (g.epi == EPI_RELU2_FP8) {
    ok = ok && make_map8(&md, g.D, g.M, cols, g.ldd, 32);
  } else if (g.epi == EPI_STORE_F32) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)g.M}, strides[1] = {(cuuint64_t)g.ldd * 4};
    const cuuint32_t box[2] = {32, 32}, estr[2] = {1, 1};
    ok = ok && encode_fn()(&md, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, g.D, dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  } else {
    ok = ok && make_map(&md, g.D, g.M, cols, g.ldd, 64, 32);
  }
  if (!ok) return cudaErrorInvalidValue;
  p.kblocks = (g.K + BK - 1) / BK;
  p.units = (int)plan.tiles;  // at most 2^30: a unit and the grid together stay an int
  p.splits = plan.splits;
  p.sa = g.sa; p.lsa = g.lsa; p.sb = g.sb; p.lsb = g.lsb;
  p.status = status;
  auto go = [&](auto *kernel) {
    return fp8::launch(kernel, (unsigned)(2 * p.splits * std::min(p.units, num_sms / 2)), PTHREADS, PSMEM, 2 * p.splits, st, ma,
                       mb, md, p);
  };
  switch (g.epi) {
    case EPI_STORE: return go(gemm_fp8_pair_kernel<EPI_STORE>);
    case EPI_STORE_F32: return go(gemm_fp8_pair_kernel<EPI_STORE_F32>);
    case EPI_ADD: return go(gemm_fp8_pair_kernel<EPI_ADD>);
    case EPI_RELU2: return go(gemm_fp8_pair_kernel<EPI_RELU2>);
    case EPI_SOFTCAP: return go(gemm_fp8_pair_kernel<EPI_SOFTCAP>);
    default: return go(gemm_fp8_pair_kernel<EPI_RELU2_FP8>);
  }
}

inline cudaError_t init() {
  cudaError_t e = tc_init();
  auto big = [&](auto *k, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  big(gemm_fp8_rows_kernel<16, true>, RowsCfg<16, true>::kSmem);
  big(gemm_fp8_rows_kernel<16, false>, RowsCfg<16, false>::kSmem);
  big(gemm_fp8_rows_kernel<32, false>, RowsCfg<32, false>::kSmem);
  big(gemm_fp8_rows_kernel<64, false>, RowsCfg<64, false>::kSmem);
  big(gemm_fp8_rows_kernel<128, false>, RowsCfg<128, false>::kSmem);
  auto pair = [&](auto *k) {
    big(k, PSMEM);
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k);
    if (e == cudaSuccess && a.numRegs != PREGS) e = cudaErrorInvalidConfiguration;  // the register split would not add up
  };
  pair(gemm_fp8_pair_kernel<EPI_STORE>);
  pair(gemm_fp8_pair_kernel<EPI_STORE_F32>);
  pair(gemm_fp8_pair_kernel<EPI_ADD>);
  pair(gemm_fp8_pair_kernel<EPI_RELU2>);
  pair(gemm_fp8_pair_kernel<EPI_SOFTCAP>);
  pair(gemm_fp8_pair_kernel<EPI_RELU2_FP8>);
  return e;
}

}  // namespace tc8

inline cudaError_t launch_gemm_fp8(const GemmFp8Problem &g, int num_sms, int *status, cudaStream_t st) {
  const tc8::Plan p = tc8::plan(g.M, g.N, g.K, num_sms);
  if (p.pair) return tc8::launch_pair(g, p, num_sms, status, st);
  if (p.many) return tc8::launch_rows<16, true>(g, p, status, st);
  switch (p.tn) {
    case 16: return tc8::launch_rows<16, false>(g, p, status, st);
    case 32: return tc8::launch_rows<32, false>(g, p, status, st);
    case 64: return tc8::launch_rows<64, false>(g, p, status, st);
    default: return tc8::launch_rows<128, false>(g, p, status, st);
  }
}

}  // namespace nc
