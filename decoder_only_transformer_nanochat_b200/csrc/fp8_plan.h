// Which kernel an 8-bit product takes, over how many CTAs its K is cut, and
// which tile a CTA pair takes when: host arithmetic (the tile order is the
// device's too), plain C++ so that tests compile it without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define NC_PLAN_FN __host__ __device__ __forceinline__
#else
#define NC_PLAN_FN inline
#endif

namespace nc {
namespace tc8 {

// Division of numbers below 2^31 by a number known on the host, as a multiply
// by its rounded-up reciprocal (Granlund and Montgomery, "Division by invariant
// integers using multiplication"): every tile's epilogue waits for its place.
struct ByHost {
  uint32_t mul;
  int shift;
  explicit ByHost(uint32_t d = 1) {
    shift = 31;
    while ((1ull << (shift - 31)) < d) ++shift;
    mul = (uint32_t)(((1ull << shift) + d - 1) / d);
  }
  NC_PLAN_FN uint32_t div(uint32_t u) const { return (uint32_t)(((uint64_t)u * mul) >> shift); }
};

// Tiles of 256 x 256, n_m x n_n of them.  Those in flight at once share operand
// panels in L2: with few N tiles those of an M block are consecutive, with many
// 16 M blocks share each B panel.
struct PairTiles {
  int n_m, n_n;
  ByHost by_n, by_group;  // n_n, 16 n_n
  PairTiles(int m, int n) : n_m(m), n_n(n), by_n((uint32_t)n), by_group(16u * (uint32_t)n) {}
  NC_PLAN_FN void tile(uint32_t u, int &m_blk, int &n_blk) const {
    if (n_n <= 16) {
      m_blk = (int)by_n.div(u);
      n_blk = (int)u - m_blk * n_n;
      return;
    }
    const uint32_t g = by_group.div(u), r = u - g * 16 * (uint32_t)n_n;
    const int first = (int)g * 16, size = n_m - first < 16 ? n_m - first : 16;
    n_blk = (int)(size == 16 ? r / 16 : r / (uint32_t)size);
    m_blk = first + (int)r - n_blk * size;
  }
};

// CTAs of clusters of `size` that run at once, per_sm of them on an SM.  A
// cluster stays within one of the groups of SMs that the GPU is made of: on 148
// SMs 33 clusters of four and 15 of eight find room at one CTA per SM, 71 and 33 at two
// (cudaOccupancyMaxActiveClusters).  One more is a second turn of the whole
// product: 36 clusters of four, 1536 x 1536 x 6144, 49.2 us against 27.1 whole; 18
// of eight, 768 x 1536 x 6144, 31.6 against 23.4 as clusters of four.  Fixed shares
// and not the device's own answer, so that equal SM counts give equal sums.
inline int cluster_room(int num_sms, int size, int per_sm) {
  if (size < 4) return num_sms * per_sm;
  if (per_sm > 1) return per_sm * (num_sms * 7 / 8);
  return size < 8 ? num_sms * 9 / 10 : num_sms * 13 / 16;
}

constexpr int kMaxPairSplits = 4;  // pairs per cluster at most: eight CTAs

struct Plan {
  bool pair;      // pairs of CTAs on 256 x 256 tiles; else weight rows x tn activation rows, a CTA each
  int tn;         // 16, 32, 64, 128
  bool many;      // (tn 16) four CTAs per SM, K not cut
  int splits;     // CTAs (pairs of them) that share a tile's K
  int64_t tiles;
};

// CTAs per SM of the form without pairs
constexpr int rows_ctas(int tn, bool many) { return many ? 4 : tn > 64 ? 1 : 2; }

inline Plan plan(int M, int N, int K, int num_sms) {
  // 128-row tiles where K can be cut over four CTAs that all run at once (300 x
  // 1280 x 5120: 13.8 us against 17.4 with 256-row tiles, 4000 x 128 x 4096: 13.3
  // against 15.8; with two K blocks, 3643 x 101 x 144, 10.4 against 8.1), up to
  // 256 rows where it can over two (96 x 1280 x 5120: 12.7 against 16.9; 256 x
  // 5120 x 1280, where it cannot: 17.1 against 12.2).  256-row tiles otherwise.
  const int kblocks = (K + 127) / 128;
  const int64_t across = ((int64_t)N + 127) / 128, tall = across * (((int64_t)M + 127) / 128);
  const bool few = 4 * tall <= cluster_room(num_sms, 4, 1) && kblocks > 7;
  Plan p = {};
  p.splits = 1;
  if (M > 64 && !few && (M > 256 || 2 * tall > num_sms)) {
    p.pair = true;
    p.tiles = (((int64_t)M + 255) / 256) * (((int64_t)N + 255) / 256);
    // A split costs about 6 us to exchange its sums (15 bytes a cycle and SM
    // between shared memories), what ten K blocks take; with twelve blocks left
    // to each it pays (512 x 1536 x 6144: 31.1 us whole, 19.6 us in four; 1024 x
    // 1280 x 1280: 12.0 us whole, 14.9 us in two).
    while (p.splits < kMaxPairSplits && kblocks >= 24 * p.splits && p.tiles * 4 * p.splits <= cluster_room(num_sms, 4 * p.splits, 1))
      p.splits *= 2;
    return p;
  }
  // the logits of a few rows (16 x 65,536 x 1280: 21.2 us with four CTAs per SM, 24.9 with two)
  p.many = M <= 16 && across > 2 * num_sms;
  p.tn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  p.tiles = across * (((int64_t)M + p.tn - 1) / p.tn);
  // cut K while every CTA still finds a place at once and keeps a K block
  while (!p.many && p.splits < 8 && 2 * p.splits <= kblocks &&
         p.tiles * 2 * p.splits <= cluster_room(num_sms, 2 * p.splits, rows_ctas(p.tn, false)))
    p.splits *= 2;
  return p;
}

}  // namespace tc8
}  // namespace nc
