// Shared by the tensor-core kernels of the grouped products: the tiles, and the PTX of
// a pair of CTAs (a cluster of two) that works on one tile.
#pragma once

#include "grouped_products.h"
#include "sm100_ptx.cuh"

namespace swl {
namespace {

struct Tile {
  int t;           // -1: no more
  int e, m0, row0, rows, n, n0;
  int kb;          // steps, 64 deep
  int k0;          // bf16: first step of this piece of the sum, and what it is joined with
  int part;        //       (kAddSum, kKeepSum)
};
enum : int { kAddSum = 1, kKeepSum = 2 };

// What the tile decoder needs.  off and prefix are read by ordinary loads: the plan writes
// prefix while the product's CTAs may be on the GPU already, which rules out the read-only
// path (its lines may be older than the plan's wait).
struct TileShape {
  const int* off;
  const int* prefix;
  int N;
  int m_tiles;     // 256-row tiles of D per group
  int n_tiles;     // dW: column tiles of D
  int cols;        // dW: columns of D
  int bn_cols;     // dW: columns of a tile
  int k_blocks;    // y, dx: ceil(depth / 64)
};

constexpr int kBK = 64;       // depth of a stage
constexpr int kBand = 8;      // row tiles of a band
constexpr int kUnit = 32;     // rows a tile's n grows by

// Tile t of a product (t < 0 in the result: past the last).
template <int W>
__device__ __forceinline__ Tile decode_tile(int t, int total, const TileShape& s) {
  Tile ts = {};
  ts.t = t < total ? t : -1;
  if (ts.t < 0) return ts;
  if constexpr (W == kGroupedDw) {
    const int per = s.m_tiles * s.n_tiles;
    ts.e = t / per;
    const int r = t - ts.e * per;
    ts.m0 = r / s.n_tiles * 256;
    ts.n0 = (r % s.n_tiles) * s.bn_cols;
    ts.row0 = s.off[ts.e];
    ts.rows = s.off[ts.e + 1] - ts.row0;
    ts.n = min(s.bn_cols, (s.cols - ts.n0 + 127) & ~127);
    ts.kb = (ts.rows + kBK - 1) / kBK;
  } else {
    const int q = t / s.m_tiles;
    int lo = 0, hi = s.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.prefix[mid] <= q) lo = mid;
      else hi = mid;
    }
    const int p0 = s.prefix[lo], nts = s.prefix[lo + 1] - p0;
    // bands of kBand row tiles go through all of W, row tiles fastest: the tiles
    // running together share few rows of x and few of W (one group of 32768 x 2048 by
    // 5120 x 2048: 573 us with all its row tiles in one band, 483 with bands of 8)
    const int local = t - p0 * s.m_tiles;
    const int band = local / (kBand * s.m_tiles);
    const int r = local - band * kBand * s.m_tiles;
    const int in_band = min(kBand, nts - band * kBand);
    const int nt = band * kBand + r % in_band;
    ts.e = lo;
    ts.m0 = r / in_band * 256;
    // the group's rows in nts parts of whole units, as even as they go: no short
    // tile that loads as much W as a full one
    const int begin = s.off[lo], rows = s.off[lo + 1] - begin;
    const int units = (rows + kUnit - 1) / kUnit;
    const int per = units / nts, more = units - per * nts;
    const int first = (nt * per + min(nt, more)) * kUnit;
    ts.row0 = begin + first;
    ts.n = (per + (nt < more ? 1 : 0)) * kUnit;
    ts.rows = min(ts.n, rows - first);
    ts.kb = s.k_blocks;
  }
  return ts;
}

// ---------------------------------------------------------------- pair PTX
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Address of the first CTA's copy of a shared variable.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(ptx::smem_u32(p)));
  return a;
}
// Arrivals on the other CTA's barrier.  A release at cluster scope waits for everything
// its thread has in flight (dW of 16384 x 1024 x 4096 over 128 groups: 334 against
// 259 us), so it is left to threads that have little: arrive_at publishes what this
// CTA's threads wrote (and told the calling thread of); arrive_relaxed_at only says
// that TMEM has been read (tcgen05.wait and the tcgen05 fences order that).
__device__ __forceinline__ void arrive_relaxed_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   ptx::smem_u32(dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on both CTAs' copies of `bar` once this thread's products have finished.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  const uint16_t both = 3;
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(ptx::smem_u32(bar)),
      "h"(both)
      : "memory");
}
// TMA loads into this CTA's shared memory that complete on the first CTA's barrier.
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, uint32_t bar,
                                             int c0, int c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, uint32_t bar,
                                             int c0, int c1, int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// MN-major bf16 tile in 128-byte-swizzled boxes of [64 k][64 mn]: 8-row groups along
// k 1024 bytes apart (stride offset), boxes along mn 8192 bytes apart (leading offset).
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
template <bool kMn>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int k) {
  // 16 deep: 32 bytes along a K-major row, or 16 rows of 128 bytes
  return kMn ? desc_mn_major(base + k * 2048) : ptx::umma_desc_sw128_kmajor(base + k * 32);
}

// Bounded wait for arrivals of the other CTA's threads (acquire at cluster scope).
__device__ __forceinline__ bool cluster_bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(ptx::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool cluster_bar_wait(uint64_t* bar, uint32_t parity,
                                                 volatile int* abort_flag, uint64_t limit_ns) {
  if (cluster_bar_try(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    if (cluster_bar_try(bar, parity)) return true;
    if ((n & 31u) == 0 && (*abort_flag || ptx::globaltimer_ns() - t0 > limit_ns)) return false;
  }
}

}  // namespace
}  // namespace swl
