// Products grouped by expert over ragged row ranges: the plan kernel, the bias
// gradient and the C entry points.
//
// Group e owns the rows offsets[e] <= r < offsets[e + 1] of x [R, K], y [R, O]:
//   y[r]  = W[e] x[r] + b[e]                  W [N, O, K], b [N, O]
//   dx[r] = W[e]^T dy[r]
//   dW[e] = sum_r dy[r] x[r]^T,  db[e] = sum_r dy[r]
// Rows outside every group have no part in any result and are not written.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "grouped_products.h"
#include "switch_layer.h"

namespace swl {
namespace {

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;

// Inclusive sum over the CTA; every thread gets its own prefix, *total the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int before = warp > 0 ? warp_sums[warp - 1] : 0;
  *total = warp_sums[31];
  __syncthreads();
  return v + before;
}

struct PlanArgs {
  const int* off;
  int* prefix;
  WsHeader* hdr;
  CUtensorMap* maps;
  int N, R, tile_rows;
};
struct MapPair {
  CUtensorMap m[2];
};

// CTA 0 counts (a group has at most R / tile_rows + 1 tiles, so the counts fit an int);
// the others make dW's maps, a warp per group: the templates with the rows ended at
// the group's last one.  A map's end is clipped to R whatever the offsets say.
// It lets the product start at once (a trigger behind the wait: 653 instead of 638 us for
// 32768 rows of 64 skewed groups, 2048 -> 5120, call after call), so the kernels behind it
// may be on the GPU while the call's inputs are still being written: they read all of
// them, and the plan's results, by ordinary loads or the copy engine, never through the
// read-only path, which does not promise to see what was written after their start.
__global__ void __launch_bounds__(kPlanThreads)
grouped_plan_kernel(const __grid_constant__ PlanArgs a, const __grid_constant__ MapPair templates) {
  __shared__ int warp_sums[32];
  pdl_trigger();
  pdl_wait();
  const int* off = a.off;
  int* prefix = a.prefix;
  WsHeader* hdr = a.hdr;
  const int N = a.N, R = a.R, tile_rows = a.tile_rows;
  if (blockIdx.x > 0) {
    const int e = (blockIdx.x - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (e >= N) return;
    const int end = min(off[e + 1], R);
    if (end <= off[e] || end <= 0) return;       // no rows: its maps are never read
    CUtensorMap* m = a.maps + 2 * static_cast<size_t>(e);
    if (lane < 16)
      reinterpret_cast<uint4*>(m)[lane] = reinterpret_cast<const uint4*>(&templates)[lane];
    __syncwarp();
    if (lane < 2) {
      asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(m + lane),
                   "r"(end)
                   : "memory");
      asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
    }
    return;
  }
  int base = 0;
  bool bad = false;
  for (int e0 = 0; e0 < N; e0 += kPlanThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    int tiles = 0;
    if (e < N) {
      const int a = off[e], b = off[e + 1];
      if (a < 0 || b < a || b > R) bad = true;
      else tiles = (b - a + tile_rows - 1) / tile_rows;
    }
    int total;
    const int incl = block_scan(tiles, warp_sums, &total);
    if (e < N) prefix[e + 1] = base + incl;
    base += total;
  }
  if (__syncthreads_or(bad)) {      // the prefix says: nothing to do
    for (int e = threadIdx.x; e <= N; e += kPlanThreads) prefix[e] = 0;
    if (threadIdx.x == 0) hdr->err = kDevIndexOutOfRange;
  } else if (threadIdx.x == 0) {
    prefix[0] = 0;
    hdr->err = kDevOk;
  }
  if (threadIdx.x == 0) hdr->next_tile = 0;
}

// Last e with P[e] <= q (P[N] > q).
__device__ __forceinline__ int find_group(const int* P, int N, int q) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (P[mid] <= q) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- bias gradient
// A CTA sums one row tile of a group (the plan's tiles) over 32 V columns: 8
// interleaved runs of rows (a warp each, 16-byte loads for bf16), then the runs in order.
// A group of one tile is then done; the tiles of a larger one leave fp32 partial sums
// that the second kernel adds in order, so a group of many rows is spread over as many
// CTAs as it has tiles.  Bound: one read of dy.
template <typename T>
struct BiasVec;
template <>
struct BiasVec<__nv_bfloat16> {
  static constexpr int V = 8;
  __device__ static __forceinline__ void add(const __nv_bfloat16* p, float (&s)[V]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const unsigned u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] += __uint_as_float(u[i] << 16);
      s[2 * i + 1] += __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct BiasVec<float> {
  static constexpr int V = 1;       // any width, any alignment of a float
  __device__ static __forceinline__ void add(const float* p, float (&s)[V]) { s[0] += *p; }
};

template <typename T>
__global__ void __launch_bounds__(256)
grouped_bias_tile_kernel(const T* dy, const int* off, const int* prefix, T* db, float* part,
                         const WsHeader* hdr, int O, int N, int tile_rows) {
  constexpr int V = BiasVec<T>::V;
  __shared__ float buf[8][32 * V];
  pdl_trigger();
  pdl_wait();
  const int q = blockIdx.x;
  if (hdr->err || q >= prefix[N]) return;
  const int e = find_group(prefix, N, q);
  const int nt = q - prefix[e];
  const int r0 = off[e] + nt * tile_rows, r1 = min(off[e + 1], r0 + tile_rows);
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = (blockIdx.y * 32 + lane) * V;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.f;
  if (c < O)
#pragma unroll 8
    for (int r = r0 + k; r < r1; r += 8) BiasVec<T>::add(dy + static_cast<int64_t>(r) * O + c, s);
#pragma unroll
  for (int i = 0; i < V; ++i) buf[k][lane + 32 * i] = s[i];
  __syncthreads();
  const bool one = prefix[e + 1] - prefix[e] == 1;
  for (int x = threadIdx.x; x < 32 * V; x += 256) {
    const int col = (blockIdx.y * 32 + (x & 31)) * V + (x >> 5);
    if (col >= O) continue;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += buf[i][x];
    if (one) db[static_cast<int64_t>(e) * O + col] = static_cast<T>(v);
    else part[static_cast<int64_t>(q) * O + col] = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
grouped_bias_sum_kernel(const int* prefix, T* db, const float* part, const WsHeader* hdr, int O,
                        int N) {
  pdl_trigger();
  pdl_wait();
  if (hdr->err) return;
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= O) return;
  const int e = blockIdx.x, a = prefix[e], b = prefix[e + 1];
  if (b - a == 1) return;                 // written by its tile
  float v = 0.f;
#pragma unroll 4
  for (int q = a; q < b; ++q) v += part[static_cast<int64_t>(q) * O + c];
  db[static_cast<int64_t>(e) * O + c] = static_cast<T>(v);
}

}  // namespace

cudaError_t launch_grouped_plan(const GroupedShape& s, const GroupedPlan& p, const int* offsets,
                                int tile_rows, const CUtensorMap* maps, cudaStream_t stream) {
  const PlanArgs a = {offsets, p.tile_prefix, p.hdr, static_cast<CUtensorMap*>(p.maps),
                      static_cast<int>(s.N), static_cast<int>(s.R), tile_rows};
  MapPair templates = {};
  if (maps) templates = {{maps[0], maps[1]}};
  constexpr int per = kPlanThreads / 32;
  const unsigned grid = 1 + (maps ? static_cast<unsigned>((s.N + per - 1) / per) : 0);
  count_launch();
  return launch_dependent(grouped_plan_kernel, dim3(grid), dim3(kPlanThreads), 0, stream, a,
                          templates);
}

template <typename T>
static cudaError_t launch_bias(const GroupedShape& s, const GroupedPlan& p, const int* offsets,
                               const void* dy, void* db, int tile_rows, cudaStream_t stream) {
  const int O = static_cast<int>(s.O), N = static_cast<int>(s.N);
  if (s.R > 0) {
    const dim3 grid(static_cast<unsigned>(s.R / tile_rows + s.N),      // row tiles, at most
                    static_cast<unsigned>((s.O + 32 * BiasVec<T>::V - 1) / (32 * BiasVec<T>::V)));
    count_launch();
    const cudaError_t e = launch_dependent(grouped_bias_tile_kernel<T>, grid, dim3(256), 0, stream,
                                           static_cast<const T*>(dy), offsets, p.tile_prefix,
                                           static_cast<T*>(db), p.bias_part, p.hdr, O, N, tile_rows);
    if (e != cudaSuccess) return e;
  }
  count_launch();
  return launch_dependent(grouped_bias_sum_kernel<T>,
                          dim3(static_cast<unsigned>(s.N), static_cast<unsigned>((s.O + 255) / 256)),
                          dim3(256), 0, stream, p.tile_prefix, static_cast<T*>(db), p.bias_part,
                          p.hdr, O, N);
}

cudaError_t launch_grouped_bias_grad(const GroupedShape& s, const GroupedPlan& p,
                                     const int* offsets, const void* dy, void* db, int tile_rows,
                                     cudaStream_t stream) {
  return (s.dtype == SWL_BF16 ? launch_bias<__nv_bfloat16> : launch_bias<float>)(
      s, p, offsets, dy, db, tile_rows, stream);
}

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

swl_status grouped_shape(int64_t R, int64_t K, int64_t O, int64_t N, int dtype, GroupedShape* s) {
  if (R < 0 || K <= 0 || O <= 0 || N <= 0) return SWL_ERR_INVALID_ARG;
  if (dtype != SWL_F32 && dtype != SWL_BF16) return SWL_ERR_INVALID_ARG;
  if (dtype == SWL_BF16 && (K % 8 != 0 || O % 8 != 0)) return SWL_ERR_UNSUPPORTED;
  const int64_t lim = INT32_MAX;
  if (N > kMaxExperts || R > lim / 2 || K > lim / 2 || O > lim / 2) return SWL_ERR_UNSUPPORTED;
  if (N * (K > O ? K : O) > lim) return SWL_ERR_UNSUPPORTED;     // as the layer's weights
  // work items of a launch fit an int
  const int64_t wide = ((K > O ? K : O) + 31) / 32;
  if ((R / 32 + N) * wide > lim || N * ((O + 31) / 32) * ((K + 31) / 32) > lim)
    return SWL_ERR_UNSUPPORTED;
  if ((O + 31) / 32 > 65535) return SWL_ERR_UNSUPPORTED;
  *s = {R, K, O, N, dtype};
  return SWL_OK;
}

int tile_rows(const GroupedShape& s) {
  return s.dtype == SWL_BF16 ? grouped_sm100_tile_rows(s) : grouped_f32_tile_rows();
}

size_t grouped_layout(const GroupedShape& s, uintptr_t base, GroupedPlan* p) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return base + o;
  };
  GroupedPlan q;
  q.hdr = reinterpret_cast<WsHeader*>(take(sizeof(WsHeader)));
  q.tile_prefix = reinterpret_cast<int*>(take((static_cast<size_t>(s.N) + 1) * 4));
  q.maps = reinterpret_cast<void*>(
      take(s.dtype == SWL_BF16 ? static_cast<size_t>(s.N) * 2 * sizeof(CUtensorMap) : 0));
  // for any call of up to R rows: a program sizes its workspace by the largest batch
  const int64_t tiles = s.dtype == SWL_BF16 ? grouped_sm100_most_tiles(s)
                                            : s.R / grouped_f32_tile_rows() + s.N;
  q.bias_part = reinterpret_cast<float*>(take(static_cast<size_t>(tiles) * s.O * 4));
  q.sums = reinterpret_cast<float*>(
      take(s.dtype == SWL_BF16 ? grouped_sm100_summing_ctas(s) * kSumsPerCta * 4 : 0));
  if (p) *p = q;
  return at;
}

int grouped_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

cudaError_t launch_product(const GroupedShape& s, const GroupedPlan& p, GroupedWhich which,
                           const int* offsets, const void* a, const void* b, const void* bias,
                           void* out, int sms, cudaStream_t stream) {
  return (s.dtype == SWL_BF16 ? launch_grouped_sm100 : launch_grouped_f32)(
      s, p, which, offsets, a, b, bias, out, sms, stream);
}

struct GroupedSpan {
  const void* p;
  int64_t n;      // bytes
};
bool grouped_meet(const GroupedSpan& a, const GroupedSpan& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// Written ranges share a byte with one another or with a read one?
bool grouped_clash(std::initializer_list<GroupedSpan> written,
                   std::initializer_list<GroupedSpan> read) {
  for (const GroupedSpan* a = written.begin(); a != written.end(); ++a) {
    for (const GroupedSpan* b = written.begin(); b != a; ++b)
      if (grouped_meet(*a, *b)) return true;
    for (const GroupedSpan& r : read)
      if (grouped_meet(*a, r)) return true;
  }
  return false;
}

}  // namespace
}  // namespace swl

using namespace swl;

extern "C" swl_status switch_layer_grouped_workspace_size(int64_t R, int64_t K, int64_t O,
                                                          int64_t N, int dtype, size_t* bytes) {
  if (!bytes) return SWL_ERR_INVALID_ARG;
  GroupedShape s;
  const swl_status st = grouped_shape(R, K, O, N, dtype, &s);
  if (st == SWL_OK) *bytes = grouped_layout(s, 0, nullptr);
  return st;
}

extern "C" swl_status switch_layer_grouped_matmul(int64_t R, int64_t K, int64_t O, int64_t N,
                                                  int dtype, const void* x,
                                                  const int32_t* offsets, const void* W,
                                                  const void* bias, void* y, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
  GroupedShape s;
  swl_status st = grouped_shape(R, K, O, N, dtype, &s);
  if (st != SWL_OK) return st;
  if (!offsets || !W || !workspace || (R > 0 && (!x || !y))) return SWL_ERR_INVALID_ARG;
  const int64_t e = dtype == SWL_BF16 ? 2 : 4;
  const uintptr_t al = dtype == SWL_BF16 ? 16 : 4;
  if (!aligned_to(x, al) || !aligned_to(W, al) || !aligned_to(y, al) || !aligned_to(bias, dtype == SWL_BF16 ? 2 : 4) ||
      !aligned_to(offsets, 4) || !aligned_to(workspace, 256))
    return SWL_ERR_UNSUPPORTED;
  GroupedPlan p;
  const size_t need = grouped_layout(s, reinterpret_cast<uintptr_t>(workspace), &p);
  if (workspace_bytes < need) return SWL_ERR_WORKSPACE;
  if (grouped_clash({{y, R * O * e}, {workspace, static_cast<int64_t>(need)}},
                    {{x, R * K * e}, {W, N * O * K * e}, {bias, N * O * e}, {offsets, (N + 1) * 4}}))
    return SWL_ERR_INVALID_ARG;
  const int sms = grouped_sms();
  if (sms <= 0) return SWL_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (grouped_few(s))
    return launch_grouped_few(s, p, offsets, x, W, bias, y, cs) == cudaSuccess ? SWL_OK
                                                                              : SWL_ERR_CUDA;
  if (launch_grouped_plan(s, p, offsets, tile_rows(s), nullptr, cs) != cudaSuccess)
    return SWL_ERR_CUDA;
  if (R == 0) return SWL_OK;
  if (launch_product(s, p, kGroupedFwd, offsets, x, W, bias, y, sms, cs) != cudaSuccess)
    return SWL_ERR_CUDA;
  return SWL_OK;
}

extern "C" swl_status switch_layer_grouped_matmul_backward(
    int64_t R, int64_t K, int64_t O, int64_t N, int dtype, const void* dy, const void* x,
    const int32_t* offsets, const void* W, void* dx, void* dW, void* db, void* workspace,
    size_t workspace_bytes, void* stream) {
  GroupedShape s;
  swl_status st = grouped_shape(R, K, O, N, dtype, &s);
  if (st != SWL_OK) return st;
  if (!offsets || !workspace || (R > 0 && (!dy || (dW && !x) || (dx && !W))) ||
      (!dx && !dW && !db && R > 0))
    return SWL_ERR_INVALID_ARG;
  const int64_t e = dtype == SWL_BF16 ? 2 : 4;
  const uintptr_t al = dtype == SWL_BF16 ? 16 : 4;
  if (!aligned_to(dy, al) || !aligned_to(x, al) || !aligned_to(W, al) || !aligned_to(dx, al) ||
      !aligned_to(dW, al) || !aligned_to(db, dtype == SWL_BF16 ? 2 : 4) || !aligned_to(offsets, 4) ||
      !aligned_to(workspace, 256))
    return SWL_ERR_UNSUPPORTED;
  GroupedPlan p;
  const size_t need = grouped_layout(s, reinterpret_cast<uintptr_t>(workspace), &p);
  if (workspace_bytes < need) return SWL_ERR_WORKSPACE;
  if (grouped_clash({{dx, R * K * e},
                     {dW, N * O * K * e},
                     {db, N * O * e},
                     {workspace, static_cast<int64_t>(need)}},
                    {{dy, R * O * e},
                     {x, dW ? R * K * e : 0},
                     {W, dx ? N * O * K * e : 0},
                     {offsets, (N + 1) * 4}}))
    return SWL_ERR_INVALID_ARG;
  const int sms = grouped_sms();
  if (sms <= 0) return SWL_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  CUtensorMap maps[2];
  const bool map = dtype == SWL_BF16 && dW && R > 0;
  if (map && !grouped_sm100_templates(s, dy, x, maps)) return SWL_ERR_CUDA;
  if (launch_grouped_plan(s, p, offsets, tile_rows(s), map ? maps : nullptr, cs) != cudaSuccess)
    return SWL_ERR_CUDA;
  if (dx && R > 0 &&
      launch_product(s, p, kGroupedDx, offsets, dy, W, nullptr, dx, sms, cs) != cudaSuccess)
    return SWL_ERR_CUDA;
  if (dW &&
      launch_product(s, p, kGroupedDw, offsets, dy, x, nullptr, dW, sms, cs) != cudaSuccess)
    return SWL_ERR_CUDA;
  if (db && launch_grouped_bias_grad(s, p, offsets, dy, db, tile_rows(s), cs) != cudaSuccess) return SWL_ERR_CUDA;
  return SWL_OK;
}
