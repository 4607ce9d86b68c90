// Products grouped by expert on the 5th-generation tensor cores, bf16 with fp32
// accumulation in TMEM: y = x W^T + b, dx = dy W and dW = dy^T x over ragged
// row ranges, one persistent kernel for each.
//
// A pair of CTAs (a cluster of two, cta_group::2) computes D[256, n], n <= 256:
// each CTA holds 128 of the 256 rows of A and n / 2 of the n rows of B, so a
// 64-deep step of a full tile brings 32 KB into each SM for 512 cycles of
// tensor work; a single CTA's 128 x 256 tile would need 48 KB, more than the L2
// delivers.  D lies in TMEM, lane = row of A, column = row of B:
//   y, dx:  A = 256 features of W[e], B = the tile's token rows.  The ragged side is
//           n, which follows the rows that are there in steps of 32: a group of a few
//           rows reads W once and multiplies little.
//   dW:     A = 256 columns of dy, B = 256 columns of x, summed over the group's rows.
//           The tensor maps of dy and x end at the group's last row (the plan writes a
//           pair of maps per group): the hardware fills the rows behind it with zeros,
//           whatever the next group holds there.
// An operand whose contiguous axis is the summed one is K-major (W and x for y,
// dy for dx); one whose summed axis is the slow one is MN-major (W for dx; dy and x
// for dW).  Both come by TMA in 128-byte-swizzled boxes 64 elements wide; no operand
// is transposed in memory.
//
// The tensor cores cut their running sums instead of rounding them: dW of positive terms
// over one group of 2^16, 2^20 and 2^22 rows came out short by 4e-4, 7e-3 and 2e-2 (half a
// step of bf16 is 2e-3 to 4e-3).  A sum of more than 32768 terms is therefore made in pieces
// of so many, a piece a tile of its own in TMEM; the epilogue threads add the pieces up in
// fp32, rounded, in the workspace (each thread its own numbers, 128 KB per CTA, which stay
// in L2).
//
// Roles of a CTA's 12 warps: 0 and 2 TMA producers of A and B, 1 MMA issuer (first CTA
// of the pair only), 3 tile decoder, 4-11 epilogue (two warps per lane quarter).  Two
// 256-column accumulators, so a tile's epilogue runs under the next tile's products.
// Tiles go round the pairs in order; the row tiles of a group are consecutive.
// Every wait is bounded: one that runs out sets the device error word and the CTA
// drains and leaves.
//
// Bound: tensor cores for groups of many rows (32768 x 2048 by 8 groups of 5120 x 2048:
// 490 us, 1.40 PFLOP/s, 0.86 of the burst peak), W's bytes for few (16384 rows over 128
// groups, 1024 -> 4096: y 208 us and dx 194 us where the bytes take 189 us), dW's stores
// (the same sizes: 259 us; a plain fill of 1.07 GB takes 275 us).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "grouped_products.h"
#include "grouped_sm100.cuh"

namespace swl {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kABytes = 128 * kBK * 2;      // a CTA's half of A
constexpr int kMaxStages = 12;
constexpr int kAccs = 2;
constexpr int kTmemCols = 512;
constexpr int kTileRing = 8;
constexpr int kPiece = 512;                      // most steps of a sum in TMEM
constexpr int kSummingPairs = 128;
// Staging of an epilogue warp: y, dx: 32 rows of 32 features; dW: 32 rows of 64 columns,
// twice (the next rows are converted while a store reads the last ones).
template <int W>
constexpr int epi_bytes() {
  return kEpiWarps * 32 * (W == kGroupedDw ? 2 * 64 : 32) * 2;
}
constexpr size_t kSmemLimit = 227 * 1024;

struct Args {
  TileShape shape;
  WsHeader* hdr;
  const CUtensorMap* maps;      // dW: [2 N] maps of dy and x per group
  const __nv_bfloat16* bias;
  __nv_bfloat16* out;
  float* sums;                  // this launch's CTAs' [256][128] each
  unsigned long long wait_ns;
  int m;           // rows of D per group: O (y, dW) or K (dx); the epilogue's features
  int bn;          // most rows of B per tile
  int stages;
  int keep_w;      // W is read by several row tiles: no evict-first
};

// The row operand of y and dx with boxes of 16, 32, .. 128 rows: a CTA's half of a
// tile's rows comes in one copy whatever their number (four boxes of 32 rows keep the
// copy engine too busy: 545 against 490 us for 32768 x 2048 by 8 x 5120 x 2048).
constexpr int kBoxes = 8;
struct RowMaps {
  CUtensorMap box[kBoxes];
};


// ---------------------------------------------------------------- the kernel
template <int W>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
grouped_sm100_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ RowMaps tmB,
                     const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ Args args) {
  constexpr bool kAmn = W != kGroupedFwd, kBmn = W == kGroupedDw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int stages = args.stages;
  const uint32_t b_bytes = static_cast<uint32_t>(args.bn / 2) * kBK * 2;
  uint8_t* smem_a = smem;
  uint8_t* smem_b = smem_a + stages * kABytes;
  uint8_t* epi = smem_b + stages * b_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + epi_bytes<W>());
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + kAccs;
  uint64_t* drain = tempty + kAccs;
  uint64_t* ring_full = drain + 1;
  uint64_t* ring_empty = ring_full + kTileRing;
  Tile* ring = reinterpret_cast<Tile*>(ring_empty + kTileRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + kTileRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], 2 * kEpiWarps);     // both CTAs' epilogue warps
    }
    ptx::mbar_init(drain, 1);
    for (int i = 0; i < kTileRing; ++i) {
      ptx::mbar_init(&ring_full[i], 1);
      ptx::mbar_init(&ring_empty[i], kEpiWarps + 2 + (leader ? 1 : 0));
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
    if (W != kGroupedDw) {
      ptx::prefetch_tmap(&tmA);
      for (int i = 0; i < kBoxes; ++i) ptx::prefetch_tmap(&tmB.box[i]);
    }
  }
  __syncthreads();
  if (warp == 2) pair_tmem_alloc(tmem_slot, kTmemCols);
  ptx::tc_fence_before();
  cluster_sync();              // barriers and TMEM of both CTAs exist
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  const int total = W == kGroupedDw ? (args.hdr->err ? 0 : args.shape.N * args.shape.m_tiles * args.shape.n_tiles)
                                    : args.shape.prefix[args.shape.N] * args.shape.m_tiles;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto fail = [&]() {
    *abort_flag = 1;
    atomicExch(&args.hdr->err, static_cast<int>(kDevPipelineTimeout));
  };

  if (warp == 3) {
    // ------------------------------------------------------------ tile decoder
    if (lane == 0) {
      bool more = true;
      for (int i = 0, t = pair; more; t += pairs) {
        Tile ts = decode_tile<W>(t, total, args.shape);
        const int steps = ts.kb;
        more = ts.t >= 0;
        do {
          const int slot = i % kTileRing;
          if (!ptx::mbar_wait(&ring_empty[slot], ((i / kTileRing) & 1) ^ 1u, abort_flag, args.wait_ns)) {
            fail();
            more = false;
            break;
          }
          ts.kb = min(steps - ts.k0, kPiece);
          ts.part = (ts.k0 > 0 ? kAddSum : 0) | (ts.k0 + ts.kb < steps ? kKeepSum : 0);
          ring[slot] = ts;
          ptx::mbar_arrive(&ring_full[slot]);
          ++i;
          ts.k0 += ts.kb;
        } while (ts.k0 < steps);
      }
    }
    __syncwarp();
  } else if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers
    // Warp 0 loads A (and, in the first CTA, announces the stage's bytes), warp 2
    // loads B: one thread for both is not fast enough for full tiles.
    if (lane == 0) {
      const bool is_a = warp == 0;
      const uint64_t norm = l2_policy_normal();
      const uint64_t pol = W == kGroupedDw || (is_a && args.keep_w)
                               ? norm
                               : is_a ? ptx::l2_policy_evict_first() : ptx::l2_policy_evict_last();
      const uint32_t bar0 = leader_addr(&full[0]);
      int stage = 0, last_e = -1;
      uint32_t ph = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int slot = i % kTileRing;
        if (!ptx::mbar_wait(&ring_full[slot], (i / kTileRing) & 1, abort_flag, args.wait_ns)) {
          fail();
          ok = false;
          break;
        }
        const Tile ts = ring[slot];
        ptx::mbar_arrive(&ring_empty[slot]);
        if (ts.t < 0) break;
        const CUtensorMap* map = &tmA;
        if constexpr (W == kGroupedDw) {
          // written by another kernel's ordinary stores
          map = args.maps + 2 * ts.e + (is_a ? 0 : 1);
          if (ts.e != last_e && ts.kb > 0)
            asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
          if (ts.kb > 0) last_e = ts.e;
        }
        const int half = ts.n >> 1;              // this CTA's rows of B
        const int m0 = ts.m0 + static_cast<int>(rank) * 128;
        const int b0 = (W == kGroupedDw ? ts.n0 : ts.row0) + static_cast<int>(rank) * half;
        const uint32_t bytes = 2 * (kABytes + static_cast<uint32_t>(half) * kBK * 2);
        for (int kb = ts.k0; kb < ts.k0 + ts.kb; ++kb) {
          if (!ptx::mbar_wait(&empty[stage], ph ^ 1u, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t bar = bar0 + stage * 8;
          if (is_a) {
            if (leader) ptx::mbar_arrive_expect_tx(&full[stage], bytes);
            uint8_t* a = smem_a + stage * kABytes;
            if constexpr (W == kGroupedFwd) {
              pair_load_3d(a, map, bar, kb * kBK, m0, ts.e, pol);
            } else if constexpr (W == kGroupedDx) {
              pair_load_3d(a, map, bar, m0, kb * kBK, ts.e, pol);
              pair_load_3d(a + 8192, map, bar, m0 + 64, kb * kBK, ts.e, pol);
            } else {
              pair_load_2d(a, map, bar, m0, ts.row0 + kb * kBK, pol);
              pair_load_2d(a + 8192, map, bar, m0 + 64, ts.row0 + kb * kBK, pol);
            }
          } else {
            uint8_t* b = smem_b + stage * b_bytes;
            if constexpr (W == kGroupedDw) {
              for (int j = 0; j < half; j += 64)
                pair_load_2d(b + j * 128, map, bar, b0 + j, ts.row0 + kb * kBK, pol);
            } else {
              pair_load_2d(b, &tmB.box[half / 16 - 1], bar, kb * kBK, b0, pol);
            }
          }
          if (++stage == stages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
      // after a failure: copies in flight (microseconds) land before the CTAs leave
      if (!ok)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader && lane == 0) {
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int slot = i % kTileRing;
        if (!ptx::mbar_wait(&ring_full[slot], (i / kTileRing) & 1, abort_flag, args.wait_ns)) {
          fail();
          break;
        }
        const Tile ts = ring[slot];
        ptx::mbar_arrive(&ring_empty[slot]);
        if (ts.t < 0) break;
        if (ts.kb == 0) continue;
        if (!cluster_bar_wait(&tempty[acc], aph ^ 1u, abort_flag, args.wait_ns)) {
          fail();
          break;
        }
        ptx::tc_fence_after();
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (kAmn ? 1u << 15 : 0u) |
                               (kBmn ? 1u << 16 : 0u) | ((static_cast<uint32_t>(ts.n) >> 3) << 17) |
                               ((256u >> 4) << 24);
        const uint32_t d = tmem + static_cast<uint32_t>(acc * (kTmemCols / kAccs));
        for (int kb = 0; kb < ts.kb; ++kb) {
          if (!ptx::mbar_wait(&full[stage], ph, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a = ptx::smem_u32(smem_a + stage * kABytes);
          const uint32_t b = ptx::smem_u32(smem_b + stage * b_bytes);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            pair_mma(d, operand_desc<kAmn>(a, k), operand_desc<kBmn>(b, k), idesc,
                     kb != 0 || k != 0 ? 1u : 0u);
          pair_commit(&empty[stage]);
          if (++stage == stages) {
            stage = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        pair_commit(&tfull[acc]);
        if (++acc == kAccs) {
          acc = 0;
          aph ^= 1u;
        }
      }
      // every product has finished before the pair's memory is given back
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
              ptx::smem_u32(drain))
          : "memory");
      volatile int never = 0;
      if (!ptx::mbar_wait(drain, 0u, &never, args.wait_ns)) fail();
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, side = (warp - 4) >> 2;
    uint8_t* const stage_out = epi + (warp - 4) * (epi_bytes<W>() / kEpiWarps);
    __nv_bfloat16* const st = reinterpret_cast<__nv_bfloat16*>(stage_out);
    const uint32_t tempty0 = leader_addr(&tempty[0]), tempty1 = leader_addr(&tempty[1]);
    int acc = 0;
    uint32_t aph = 0;
    bool flip = false;
    // this thread's numbers of a sum in pieces: column c at [c][q * 32 + lane]
    float* const sums = args.sums + static_cast<size_t>(blockIdx.x) * kSumsPerCta + q * 32 + lane;
    auto join = [&](uint32_t (&r)[32], int c0, int part) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float* const s = sums + (c0 + j) * 128;
        float v = __uint_as_float(r[j]);
        if (part & kAddSum) v += *s;
        if (part & kKeepSum) *s = v;
        r[j] = __float_as_uint(v);
      }
    };
    for (int i = 0;; ++i) {
      const int slot = i % kTileRing;
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(&ring_full[slot], (i / kTileRing) & 1, abort_flag,
                                                  args.wait_ns))) {
        fail();
        break;
      }
      const Tile ts = ring[slot];
      if (ts.t < 0) break;
      const int f0 = ts.m0 + static_cast<int>(rank) * 128 + q * 32;   // this warp's rows of D
      const int f = f0 + lane;
      float bias = 0.f;
      if (W == kGroupedFwd && args.bias != nullptr && f < args.m)
        bias = __bfloat162float(args.bias[static_cast<size_t>(ts.e) * args.m + f]);
      const uint32_t t0 = tmem + static_cast<uint32_t>(acc * (kTmemCols / kAccs)) +
                          (static_cast<uint32_t>(q * 32) << 16);
      if (ts.kb > 0) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&tfull[acc], aph, abort_flag, args.wait_ns))) {
          fail();
          break;
        }
        ptx::tc_fence_after();
      }
      if constexpr (W == kGroupedDw) {
        // 64 columns at a time: a lane converts its row, the rows go out by a TMA store
        // from 128-byte-swizzled staging (whole 128-byte lines; rows and columns past the
        // end of the group's matrix are not written)
        const int width = min(ts.n, args.shape.cols - ts.n0);
        for (int c0 = side * 64; c0 < width; c0 += 128) {
          uint32_t r[2][32];
          if (ts.kb > 0) {
            ptx::tmem_ld_32x32b_x32(t0 + static_cast<uint32_t>(c0), r[0]);
            ptx::tmem_ld_32x32b_x32(t0 + static_cast<uint32_t>(c0 + 32), r[1]);
            ptx::tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) r[j >> 5][j & 31] = 0u;
          }
          if (ts.part) {
            join(r[0], c0, ts.part);
            join(r[1], c0 + 32, ts.part);
            if (ts.part & kKeepSum) continue;
          }
          // this half of the staging is free once the store before the last has read it
          uint8_t* const half_out = stage_out + (flip ? 4096 : 0);
          flip = !flip;
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            __nv_bfloat162 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int c = j * 8 + 2 * k;
              v[k] = __floats2bfloat162_rn(__uint_as_float(r[c >> 5][c & 31]),
                                           __uint_as_float(r[(c + 1) >> 5][(c + 1) & 31]));
            }
            *reinterpret_cast<uint4*>(half_out + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                *reinterpret_cast<const uint4*>(v);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (f0 < args.m) asm volatile(
                "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                    reinterpret_cast<uint64_t>(&tmOut)),
                "r"(ptx::smem_u32(half_out)), "r"(ts.n0 + c0), "r"(f0), "r"(ts.e)
                : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      } else {
        for (int c0 = side * 32; c0 < ts.rows; c0 += 64) {
          uint32_t r[32];
          ptx::tmem_ld_32x32b_x32(t0 + static_cast<uint32_t>(c0), r);
          ptx::tmem_ld_wait();
          if (ts.part) {
            join(r, c0, ts.part);
            if (ts.part & kKeepSum) continue;
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) {     // two rows per conversion
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[j]) + bias,
                                                           __uint_as_float(r[j + 1]) + bias);
            st[j * 32 + lane] = h.x;
            st[(j + 1) * 32 + lane] = h.y;
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int idx = lane + 32 * k;
            const int j = idx >> 2, part = idx & 3;
            if (c0 + j < ts.rows && f0 + part * 8 < args.m)
              *reinterpret_cast<uint4*>(args.out + static_cast<size_t>(ts.row0 + c0 + j) * args.m +
                                        f0 + part * 8) =
                  *reinterpret_cast<const uint4*>(st + j * 32 + part * 8);
          }
          __syncwarp();
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (ts.kb > 0) arrive_relaxed_at(acc == 0 ? tempty0 : tempty1);
        ptx::mbar_arrive(&ring_empty[slot]);
      }
      if (ts.kb > 0 && ++acc == kAccs) {
        acc = 0;
        aph ^= 1u;
      }
    }
    if (W == kGroupedDw && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  ptx::tc_fence_before();
  cluster_sync();              // neither CTA leaves while the other may reach into it
  if (warp == 2) {
    ptx::tc_fence_after();
    pair_tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

bool grouped_sm100_templates(const GroupedShape& s, const void* dy, const void* x, CUtensorMap* out) {
  const uint64_t dd[2] = {static_cast<uint64_t>(s.O), static_cast<uint64_t>(s.R)};
  const uint64_t dx[2] = {static_cast<uint64_t>(s.K), static_cast<uint64_t>(s.R)};
  const uint32_t box[2] = {64, 64};
  return encode_tmap_bf16(&out[0], dy, 2, dd, box) && encode_tmap_bf16(&out[1], x, 2, dx, box);
}

// Rows of B per tile, at most: 256 from 40 rows per group on average on (one pass over W
// for most groups), 64 below (more stages of W fit).  128 groups of 2048 x 1024, rows
// spread unevenly: 24 per group 95 us with 256 and 90 with 64, 40: 99 and 99, 64: 104
// and 117, 96: 110 and 166.
int grouped_sm100_tile_rows(const GroupedShape& s) { return s.R >= 40 * s.N ? 256 : 64; }
int grouped_sm100_summing_ctas(const GroupedShape& s) {
  constexpr int64_t most = int64_t{kPiece} * kBK;
  if (s.K > most || s.O > most) return 2 * kSummingPairs;
  const int64_t tiles = s.N * ((s.O + 255) / 256) * ((s.K + 255) / 256);      // dW's
  return s.R <= most ? 0 : static_cast<int>(2 * (tiles < kSummingPairs ? tiles : kSummingPairs));
}
int64_t grouped_sm100_most_tiles(const GroupedShape& s) {
  const int64_t few = (s.R < 40 * s.N ? s.R : 40 * s.N - 1) / 64, all = s.R / grouped_sm100_tile_rows(s);
  return (few > all ? few : all) + s.N;
}

cudaError_t launch_grouped_sm100(const GroupedShape& s, const GroupedPlan& p, GroupedWhich which,
                                 const int* offsets, const void* a, const void* b,
                                 const void* bias, void* out, int num_sms, cudaStream_t stream) {
  const uint64_t K = s.K, O = s.O, N = s.N, R = s.R;
  CUtensorMap mapA = {}, mapOut = {};
  RowMaps rows = {};
  Args g = {};
  g.shape.off = offsets;
  g.shape.prefix = p.tile_prefix;
  g.hdr = p.hdr;
  g.maps = static_cast<const CUtensorMap*>(p.maps);
  g.bias = static_cast<const __nv_bfloat16*>(bias);
  g.out = static_cast<__nv_bfloat16*>(out);
  g.sums = p.sums;
  g.wait_ns = grouped_wait_ns(which == kGroupedFwd ? s.K : which == kGroupedDx ? s.O : s.R);
  g.shape.N = static_cast<int>(N);
  int64_t tiles;      // at most
  if (which == kGroupedDw) {
    const uint64_t dout[3] = {K, O, N};
    const uint32_t bout[3] = {64, 32, 1};
    if (!encode_tmap_bf16(&mapOut, out, 3, dout, bout)) return cudaErrorInvalidValue;
    g.m = static_cast<int>(O);
    g.shape.cols = static_cast<int>(K);
    g.shape.n_tiles = static_cast<int>((K + 255) / 256);
    g.shape.bn_cols = 256;
    g.bn = K <= 128 ? 128 : 256;
    g.shape.m_tiles = (g.m + 255) / 256;
    tiles = static_cast<int64_t>(N) * g.shape.m_tiles * g.shape.n_tiles;
  } else {
    const uint64_t dw[3] = {K, O, N}, dr[2] = {which == kGroupedFwd ? K : O, R};
    const uint32_t bw[3] = {64, which == kGroupedFwd ? 128u : 64u, 1};
    g.bn = grouped_sm100_tile_rows(s);
    // a is the row operand (x, dy), b is W
    if (!encode_tmap_bf16(&mapA, b, 3, dw, bw)) return cudaErrorInvalidValue;
    for (int i = 0; i < kBoxes; ++i) {
      const uint32_t br[2] = {64, 16u * (i + 1)};
      if (!encode_tmap_bf16(&rows.box[i], a, 2, dr, br)) return cudaErrorInvalidValue;
    }
    g.m = static_cast<int>(which == kGroupedFwd ? O : K);
    g.shape.k_blocks = static_cast<int>((dr[0] + kBK - 1) / kBK);
    g.shape.m_tiles = (g.m + 255) / 256;
    g.keep_w = s.R > 2 * g.bn * s.N;
    tiles = (s.R / g.bn + s.N) * g.shape.m_tiles;
  }
  const size_t stage = kABytes + static_cast<size_t>(g.bn / 2) * kBK * 2;
  const size_t fixed = 1024 + (which == kGroupedDw ? epi_bytes<kGroupedDw>() : epi_bytes<kGroupedFwd>()) + (2 * kMaxStages + 2 * kAccs + 1 + 2 * kTileRing) * 8 +
                       kTileRing * sizeof(Tile) + 64;
  int stages = static_cast<int>((kSmemLimit - fixed) / stage);
  g.stages = stages < kMaxStages ? stages : kMaxStages;
  const size_t smem = fixed + g.stages * stage;
  auto* kernel = which == kGroupedFwd  ? grouped_sm100_kernel<kGroupedFwd>
                 : which == kGroupedDx ? grouped_sm100_kernel<kGroupedDx>
                                       : grouped_sm100_kernel<kGroupedDw>;
  // the limit holds for the process: always the same value, so that a call of another
  // shape in another thread cannot lower it between here and the launch
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmemLimit));
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::min(num_sms / 2, kSummingPairs);
  count_launch();
  return launch_dependent(kernel, dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs))),
                          dim3(kThreads), smem, stream, mapA, rows, mapOut, g);
}

}  // namespace swl
