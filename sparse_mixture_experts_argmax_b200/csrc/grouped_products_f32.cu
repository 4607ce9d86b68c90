// Products grouped by expert on the tensor cores for fp32 tensors: y = x W^T + b,
// dx = dy W and dW = dy^T x over ragged row ranges.
//
// An fp32 number is the sum of three bf16 numbers: its leading 8 significant bits, the
// next 8 and the last 8 (x = hi + mid + lo, cut, not rounded: two instructions a piece,
// and nothing overflows; of a number that is not finite a rest is NaN).  Exactly so from
// 2^-110 on; bf16 ends at 2^-133, and what a smaller number has below that is cut off.  A
// product is then eight bf16 products, each exact in fp32,
//   lo mid' + mid lo' + lo hi' + hi lo' + mid mid' + mid hi' + hi mid' + hi hi',
// the ninth, lo lo', being under 2^-28 of it.  Eight tensor-core products cost 0.37 of
// one fp32 FMA per term at these units' rates (1.64 PFLOP/s against 75 TFLOP/s).  Six
// products of pieces rounded to nearest leave out 2^-23, and the rounding cost more than
// the two products.
//
// The tensor cores cut their running sums instead of rounding them, so a long sum
// would drift by half a unit per step.  Sums in TMEM therefore run over 64 terms only,
// the small products first (their sum is 2^-7 of the whole, so cutting it costs
// nothing); the epilogue warps add the partial sums up in registers, rounded.
//
// A pair of CTAs (cta_group::2) computes D[256, n], n <= 128; lane = row of A:
//   y, dx:  A = 256 features of W[e], B = the tile's token rows (n follows them)
//   dW:     A = 256 columns of x, B = 128 columns of dy, summed over the group's rows
// so that the 32 lanes of a store are consecutive in memory and no staging is needed.
// Bound: the converting warps read fp32 operands from memory (any alignment, any width;
// columns and rows past the end become zeros), split them and store three
// 128-byte-swizzled tiles each, 11 instructions per 2 elements; at n = 128 the eight
// products of a 64-deep step take 2048 cycles and its 12288 elements about 600 issue
// cycles of splitting, for fewer rows the loads bound it.
//
// Measured: 4095 rows over 60 groups, 765 -> 1021 (no row aligned): 130 us, bytes 33 us;
// 16384 rows over 8 groups, 1024 -> 2048: 516 us, 133 TFLOP/s of fp32 products (fp32 FMA
// tiles took 367 us for the first).  A step takes about 2.2 us, the converters' loads,
// splits and stores following one another in 8 warps; what is left of it is there.
//
// Roles of a CTA's 20 warps: 0 MMA issuer (first CTA only), 1 TMEM, 2 tile decoder, 3
// relay between the converters and the first CTA, 4-11 sums and stores (two warps per
// lane quarter), 12-19 converters.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "grouped_sm100.cuh"

namespace swl {
namespace {

constexpr int kSumWarps = 8, kConvWarps = 8;
constexpr int kThreads = 128 + 32 * (kSumWarps + kConvWarps);
constexpr int kBN = 128;                               // most rows of B per tile
constexpr uint32_t kAPlane = 128 * kBK * 2;            // a CTA's half of A, one piece
constexpr uint32_t kBPlane = kBN / 2 * kBK * 2;
constexpr uint32_t kStageBytes = 3 * (kAPlane + kBPlane);
constexpr int kStages = 3;
constexpr int kAccs = 4;
constexpr int kAccCols = kBN;
constexpr int kTileRing = 8;

struct Args {
  TileShape shape;
  WsHeader* hdr;
  const float* a;      // W (y, dx) or x (dW)
  const float* b;      // x, dy, dy
  const float* bias;
  float* out;
  unsigned long long wait_ns;
  int O, K;
  bool even_a, even_b;   // every row of the operand starts on an 8-byte boundary
};

// The three pieces of two numbers, packed.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  const float r0 = x0 - __uint_as_float(__float_as_uint(x0) & 0xffff0000u);
  const float r1 = x1 - __uint_as_float(__float_as_uint(x1) & 0xffff0000u);
  const float s0 = r0 - __uint_as_float(__float_as_uint(r0) & 0xffff0000u);
  const float s1 = r1 - __uint_as_float(__float_as_uint(r1) & 0xffff0000u);
  hi = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
  mid = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
  lo = __byte_perm(__float_as_uint(s0), __float_as_uint(s1), 0x7632);
}

// What a converting thread holds of a stage: kCount runs of kRun consecutive floats of
// the operands' lines.  kWide (every row of both operands on a 16-byte boundary): runs
// of 8, two 16-byte loads each, a line taken by 8 threads.  Else runs of 2, a line taken
// by a whole warp, so that its loads stay within the line's sectors (8 floats per thread
// by single loads touch every sector 8 times): one 8-byte load when the operand's rows
// all start on one, else two loads.
template <bool kWide>
struct Runs {
  static constexpr int kRun = kWide ? 8 : 2;
  static constexpr int kPerLine = kBK / kRun;
  static constexpr int kLines = 32 * kConvWarps / kPerLine;      // lines a round takes
  static constexpr int kA = 128 / kLines, kB = kBN / 2 / kLines;   // rounds of A and of B
  static constexpr int kSet = (kA + kB) / 2;
  static_assert(kA >= kSet && kA + kB == 2 * kSet, "two sets, the first of A alone");
  float v[2][kSet][kRun];
};
template <bool kWide>
__device__ __forceinline__ void load_run(const float* p, int n, bool even,
                                         float (&v)[Runs<kWide>::kRun]) {
  if constexpr (kWide) {       // n is a multiple of 4
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (n > 0) a = *reinterpret_cast<const float4*>(p);
    if (n > 4) b = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else if (even) {           // n is even
    float2 a = make_float2(0.f, 0.f);
    if (n > 0) a = *reinterpret_cast<const float2*>(p);
    v[0] = a.x, v[1] = a.y;
  } else {
    v[0] = n > 0 ? *p : 0.f;
    v[1] = n > 1 ? p[1] : 0.f;
  }
}

// One operand of a tile as a converting thread walks it.  A line is 64 consecutive
// floats, 128 bytes of each of the bf16 tiles.  K-major: a line is a row of the operand
// and runs along the depth, its next depth block is 64 floats on; MN-major: a line is
// a depth and runs along 64 of the operand's rows (lines 64 on: the next 64 rows), the
// next depth block is 64 lines on.
template <bool kMn>
struct Side {
  const float* p;    // this thread's element of line line0, this depth block
  int64_t ld;
  int lines;         // lines that are there, of this depth block on (K-major: of the tile)
  int n;             // elements that are there from p on
  __device__ __forceinline__ void start(const float* base, int64_t stride, int there, int width,
                                        int line0, int c) {
    p = base + line0 * stride + c;
    ld = stride;
    lines = there;
    n = width - c;
  }
  __device__ __forceinline__ void next() {
    p += kMn ? kBK * ld : kBK;
    if (kMn) lines -= kBK;
    else n -= kBK;
  }
  // Round j's run: line line0 + kLines j.
  template <bool kWide>
  __device__ __forceinline__ void load(int j, int line0, bool even,
                                       float (&v)[Runs<kWide>::kRun]) const {
    const int first = Runs<kWide>::kLines * j;
    const int line = kMn ? first & 63 : first, box = kMn ? first >> 6 : 0;
    const int there = line0 + line < lines ? n - box * 64 : 0;
    load_run<kWide>(p + line * ld + box * 64, there, even, v);
  }
};

template <int W, bool kWide>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
grouped_f32_kernel(const __grid_constant__ Args args) {
  constexpr bool kAmn = W != kGroupedFwd, kBmn = W == kGroupedDw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* mine = full + kStages;        // this CTA's half of a stage is there
  uint64_t* empty = mine + kStages;
  uint64_t* tfull = empty + kStages;
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
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 2);                 // both CTAs' halves
      ptx::mbar_init(&mine[s], kConvWarps);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], 2 * kSumWarps);
    }
    ptx::mbar_init(drain, 1);
    for (int i = 0; i < kTileRing; ++i) {
      ptx::mbar_init(&ring_full[i], 1);
      ptx::mbar_init(&ring_empty[i], kSumWarps + kConvWarps + 1 + (leader ? 1 : 0));
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (warp == 1) pair_tmem_alloc(tmem_slot, kAccs * kAccCols);
  ptx::tc_fence_before();
  cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  const int total = W == kGroupedDw
                        ? (args.hdr->err ? 0 : args.shape.N * args.shape.m_tiles * args.shape.n_tiles)
                        : args.shape.prefix[args.shape.N] * args.shape.m_tiles;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto fail = [&]() {
    *abort_flag = 1;
    atomicExch(&args.hdr->err, static_cast<int>(kDevPipelineTimeout));
  };
  // every lane of a warp leaves together
  auto next_tile = [&](int i, Tile& ts) -> bool {
    const int slot = i % kTileRing;
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(&ring_full[slot], (i / kTileRing) & 1, abort_flag,
                                                args.wait_ns))) {
      fail();
      return false;
    }
    ts = ring[slot];
    return ts.t >= 0;
  };

  if (warp == 2) {
    // ------------------------------------------------------------ tile decoder
    if (lane == 0) {
      int t = pair;
      for (int i = 0;; ++i, t += pairs) {
        const int slot = i % kTileRing;
        if (!ptx::mbar_wait(&ring_empty[slot], ((i / kTileRing) & 1) ^ 1u, abort_flag, args.wait_ns)) {
          fail();
          break;
        }
        const Tile ts = decode_tile<W>(t, total, args.shape);
        ring[slot] = ts;
        ptx::mbar_arrive(&ring_full[slot]);
        if (ts.t < 0) break;
      }
    }
    __syncwarp();
  } else if (warp == 0) {
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
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (kAmn ? 1u << 15 : 0u) |
                               (kBmn ? 1u << 16 : 0u) | ((static_cast<uint32_t>(ts.n) >> 3) << 17) |
                               ((256u >> 4) << 24);
        for (int kb = 0; kb < ts.kb; ++kb) {
          if (!cluster_bar_wait(&tempty[acc], aph ^ 1u, abort_flag, args.wait_ns) ||
              !cluster_bar_wait(&full[stage], ph, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a = ptx::smem_u32(smem + stage * kStageBytes), b = a + 3 * kAPlane;
          const uint32_t d = tmem + static_cast<uint32_t>(acc * kAccCols);
          // pieces 0 hi, 1 mid, 2 lo; the small products first
          constexpr int kPa[8] = {2, 1, 2, 0, 1, 1, 0, 0}, kPb[8] = {1, 2, 0, 2, 1, 0, 1, 0};
#pragma unroll
          for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              pair_mma(d, operand_desc<kAmn>(a + kPa[p] * kAPlane, k),
                       operand_desc<kBmn>(b + kPb[p] * kBPlane, k), idesc, p != 0 || k != 0 ? 1u : 0u);
          pair_commit(&empty[stage]);
          pair_commit(&tfull[acc]);
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1u;
          }
          if (++acc == kAccs) {
            acc = 0;
            aph ^= 1u;
          }
        }
      }
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
              ptx::smem_u32(drain))
          : "memory");
      volatile int never = 0;
      if (!ptx::mbar_wait(drain, 0u, &never, args.wait_ns)) fail();
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ relay
    // Tells the first CTA of this CTA's halves, one release at cluster scope for all
    // converter warps.
    if (lane == 0) {
      const uint32_t full0 = leader_addr(&full[0]);
      int stage = 0;
      uint32_t ph = 0;
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
        for (int kb = 0; kb < ts.kb; ++kb) {
          if (!ptx::mbar_wait(&mine[stage], ph, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          arrive_at(full0 + stage * 8);
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp >= 4 + kSumWarps) {
    // ------------------------------------------------------------ converters
    const int tid = threadIdx.x - 32 * (4 + kSumWarps);
    int stage = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      Tile ts;
      if (!next_tile(i, ts)) break;
      if (lane == 0) ptx::mbar_arrive(&ring_empty[i % kTileRing]);
      const int half = ts.n >> 1;
      const int m0 = ts.m0 + static_cast<int>(rank) * 128;
      const int b0 = static_cast<int>(rank) * half;
      using R = Runs<kWide>;
      const int line0 = tid / R::kPerLine, c = (tid % R::kPerLine) * R::kRun;
      Side<kAmn> A;
      Side<kBmn> B;
      if constexpr (W == kGroupedFwd) {
        A.start(args.a + (static_cast<int64_t>(ts.e) * args.O + m0) * args.K, args.K, args.O - m0,
                args.K, line0, c);
        B.start(args.b + (static_cast<int64_t>(ts.row0) + b0) * args.K, args.K,
                min(half, ts.rows - b0), args.K, line0, c);
      } else if constexpr (W == kGroupedDx) {
        A.start(args.a + static_cast<int64_t>(ts.e) * args.O * args.K + m0, args.K, args.O,
                args.K - m0, line0, c);
        B.start(args.b + (static_cast<int64_t>(ts.row0) + b0) * args.O, args.O,
                min(half, ts.rows - b0), args.O, line0, c);
      } else {
        A.start(args.a + static_cast<int64_t>(ts.row0) * args.K + m0, args.K, ts.rows, args.K - m0,
                line0, c);
        B.start(args.b + static_cast<int64_t>(ts.row0) * args.O + ts.n0 + b0, args.O, ts.rows,
                args.O - ts.n0 - b0, line0, c);
      }
      R runs;
      // two sets: one is in flight while the other is split
      auto fetch_set = [&](int s) {
#pragma unroll
        for (int j = 0; j < R::kSet; ++j) {
          const int q = s * R::kSet + j;
          if (q < R::kA) A.template load<kWide>(q, line0, args.even_a, runs.v[s][j]);
          else B.template load<kWide>(q - R::kA, line0, args.even_b, runs.v[s][j]);
        }
      };
      const uint32_t at0 = line0 * 128 + (((c >> 3) ^ (line0 & 7)) << 4) + (c & 7) * 2;
      auto put_set = [&](int s, uint8_t* a) {
#pragma unroll
        for (int j = 0; j < R::kSet; ++j) {
          const int q = s * R::kSet + j;
          const uint32_t plane = q < R::kA ? kAPlane : kBPlane;
          // (rounds are whole multiples of 8 lines: the swizzle stays)
          uint8_t* at = a + at0 + (q < R::kA ? q * R::kLines * 128
                                             : 3 * kAPlane + (q - R::kA) * R::kLines * 128);
          uint32_t w[3][R::kRun / 2];
          const float* v = runs.v[s][j];
#pragma unroll
          for (int i = 0; i < R::kRun / 2; ++i)
            split2(v[2 * i], v[2 * i + 1], w[0][i], w[1][i], w[2][i]);
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            if constexpr (kWide)
              *reinterpret_cast<uint4*>(at + i * plane) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            else
              *reinterpret_cast<uint32_t*>(at + i * plane) = w[i][0];
          }
        }
      };
      if (ts.kb > 0) {
        fetch_set(0);
        fetch_set(1);
      }
      for (int kb = 0; kb < ts.kb; ++kb) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&empty[stage], ph ^ 1u, abort_flag, args.wait_ns))) {
          fail();
          ok = false;
          break;
        }
        uint8_t* a = smem + stage * kStageBytes;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s == 0) {
            A.next();
            B.next();
          }
          put_set(s, a);
          if (kb + 1 < ts.kb) fetch_set(s);
        }
        ptx::fence_proxy_async_smem();       // the stores, before the tensor cores' reads
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&mine[stage]);
        if (++stage == kStages) {
          stage = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums and stores
    const int q = warp & 3, side = (warp - 4) >> 2;
    const uint32_t tempty0 = leader_addr(&tempty[0]);
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      Tile ts;
      if (!next_tile(i, ts)) break;
      const int f = ts.m0 + static_cast<int>(rank) * 128 + q * 32 + lane;     // this lane's row of D
      const int c0 = side * (kBN / 2);                                          // its 64 columns
      float sum[kBN / 2];
#pragma unroll
      for (int j = 0; j < kBN / 2; ++j) sum[j] = 0.f;
      for (int kb = 0; kb < ts.kb; ++kb) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&tfull[acc], aph, abort_flag, args.wait_ns))) {
          fail();
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t t0 = tmem + static_cast<uint32_t>(acc * kAccCols + c0) +
                            (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (c0 + h * 32 >= ts.n) break;
          uint32_t r[32];
          ptx::tmem_ld_32x32b_x32(t0 + h * 32, r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[h * 32 + j] += __uint_as_float(r[j]);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed_at(tempty0 + acc * 8);
        if (++acc == kAccs) {
          acc = 0;
          aph ^= 1u;
        }
      }
      if (!ok) break;
      if constexpr (W == kGroupedDw) {
        // lane = column k of dW[e], its 64 sums = rows o
        const int n = args.O - ts.n0 - c0;
        if (f < args.K) {
          float* o = args.out + (static_cast<int64_t>(ts.e) * args.O + ts.n0 + c0) * args.K + f;
#pragma unroll
          for (int j = 0; j < kBN / 2; ++j)
            if (j < n) o[static_cast<int64_t>(j) * args.K] = sum[j];
        }
      } else {
        const int m = W == kGroupedFwd ? args.O : args.K;
        const int n = ts.rows - c0;
        if (f < m) {
          float bias = 0.f;
          if (W == kGroupedFwd && args.bias) bias = args.bias[static_cast<int64_t>(ts.e) * m + f];
          float* o = args.out + (static_cast<int64_t>(ts.row0) + c0) * m + f;
#pragma unroll
          for (int j = 0; j < kBN / 2; ++j)
            if (j < n) o[static_cast<int64_t>(j) * m] = sum[j] + bias;
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ring_empty[i % kTileRing]);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    pair_tmem_dealloc(tmem, kAccs * kAccCols);
  }
}

}  // namespace

int grouped_f32_tile_rows() { return kBN; }

cudaError_t launch_grouped_f32(const GroupedShape& s, const GroupedPlan& p, GroupedWhich which,
                               const int* offsets, const void* a, const void* b, const void* bias,
                               void* out, int num_sms, cudaStream_t stream) {
  Args g = {};
  const bool dw = which == kGroupedDw;
  // callers give (x, W), (dy, W) and (dy, x)
  g.a = static_cast<const float*>(b);
  g.b = static_cast<const float*>(a);
  g.bias = static_cast<const float*>(bias);
  g.out = static_cast<float*>(out);
  g.hdr = p.hdr;
  g.wait_ns = grouped_wait_ns(which == kGroupedFwd ? s.K : which == kGroupedDx ? s.O : s.R);
  g.O = static_cast<int>(s.O);
  g.K = static_cast<int>(s.K);
  g.shape.off = offsets;
  g.shape.prefix = p.tile_prefix;
  g.shape.N = static_cast<int>(s.N);
  const int64_t m = which == kGroupedFwd ? s.O : s.K, depth = which == kGroupedFwd ? s.K : s.O;
  g.shape.m_tiles = static_cast<int>((m + 255) / 256);
  g.shape.n_tiles = static_cast<int>((s.O + kBN - 1) / kBN);
  g.shape.cols = g.O;
  g.shape.bn_cols = kBN;
  g.shape.k_blocks = static_cast<int>((depth + kBK - 1) / kBK);
  const int64_t tiles = dw ? s.N * g.shape.m_tiles * g.shape.n_tiles
                           : (s.R / kBN + s.N) * g.shape.m_tiles;      // at most
  // 16-byte loads when every row of both operands starts on a 16-byte boundary
  auto aligned = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool wide = aligned(a) && aligned(b) && s.K % 4 == 0 && s.O % 4 == 0;
  auto even = [](const void* q, int64_t row) {
    return (reinterpret_cast<uintptr_t>(q) & 7) == 0 && row % 2 == 0;
  };
  g.even_a = even(g.a, s.K);
  g.even_b = even(g.b, which == kGroupedFwd ? s.K : s.O);
  auto* kernel = which == kGroupedFwd  ? (wide ? grouped_f32_kernel<kGroupedFwd, true>
                                               : grouped_f32_kernel<kGroupedFwd, false>)
                 : which == kGroupedDx ? (wide ? grouped_f32_kernel<kGroupedDx, true>
                                               : grouped_f32_kernel<kGroupedDx, false>)
                                       : (wide ? grouped_f32_kernel<kGroupedDw, true>
                                               : grouped_f32_kernel<kGroupedDw, false>);
  const size_t smem = 1024 + kStages * kStageBytes + (3 * kStages + 2 * kAccs + 1 + 2 * kTileRing) * 8 +
                      kTileRing * sizeof(Tile) + 64;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t pairs = num_sms / 2;
  count_launch();
  return launch_dependent(kernel, dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs))),
                          dim3(kThreads), smem, stream, g);
}

}  // namespace swl
