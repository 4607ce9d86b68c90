// y = x W^T + b grouped by expert for a handful of rows (decoded tokens): W of the
// groups that have rows is streamed once, straight from memory.
//
// Bound: HBM, W's bytes; a row's products are 2 FLOPs per element of W.  The plan
// and the tile pipeline of the tensor-core kernel cost more than the products
// here, so this kernel is the only launch: a CTA per (row, 32 features) looks the row's
// group up in the offsets and goes on if the row is the group's first; it then
// multiplies all rows of the group.  A warp takes kF features at a time, its lanes 16
// bytes of each feature's weights per step, several steps in flight; x's rows come from
// L1.  (Ordinary loads: the kernel may be on the GPU while the one before still writes
// x.)  fp32 FMAs, a lane's partial sums joined by shuffles.
// Measured with 8 bf16 tokens over 128 experts of 4096 x 1024: 12.1 us on the device, 5.4
// TB/s of the touched experts' weights (floor 10.0 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "grouped_products.h"

namespace swl {
namespace {

constexpr int kThreads = 128;
constexpr int kF = 4;                        // features per warp at a time
constexpr int kPerCta = 32;                  // features of a CTA

template <typename T, int V>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 q;
  __device__ __forceinline__ void get(float (&o)[8]) const {
    const unsigned u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(u[i] << 16);
      o[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Piece<float, 4> {
  float4 q;
  __device__ __forceinline__ void get(float (&o)[4]) const { o[0] = q.x, o[1] = q.y, o[2] = q.z, o[3] = q.w; }
};
template <>
struct Piece<float, 1> {
  float q;
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = q; }
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_once(const T* p) {      // weights: read by one CTA
  Piece<T, V> r;
  r.q = __ldcs(reinterpret_cast<const decltype(r.q)*>(p));
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_row(const T* p) {
  Piece<T, V> r;
  r.q = *reinterpret_cast<const decltype(r.q)*>(p);
  return r;
}

template <typename T>
struct FewArgs {
  const T* x;
  const T* W;
  const T* bias;
  T* y;
  const int* off;
  WsHeader* hdr;
  int R, K, O, N;
};

// Rows row0 .. row0 + n of group e, n <= kRows, features [o0, o0 + kPerCta).
template <typename T, int V, int kRows>
__device__ __forceinline__ void few_rows(const FewArgs<T>& a, int e, int row0, int n, int o0) {
  constexpr int kSteps = kRows <= 4 ? 4 : kRows <= 8 ? 2 : 1;      // steps in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = a.x + static_cast<int64_t>(row0) * a.K;
  for (int f0 = o0 + warp * kF; f0 < min(o0 + kPerCta, a.O); f0 += kThreads / 32 * kF) {
    const T* w[kF];
#pragma unroll
    for (int f = 0; f < kF; ++f)       // past the last feature: the last again, not stored
      w[f] = a.W + (static_cast<int64_t>(e) * a.O + min(f0 + f, a.O - 1)) * a.K;
    float acc[kF][kRows];
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
      for (int r = 0; r < kRows; ++r) acc[f][r] = 0.f;
    for (int k0 = lane * V; k0 < a.K; k0 += 32 * V * kSteps) {
      Piece<T, V> q[kSteps][kF];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int f = 0; f < kF; ++f) {
          const int k = k0 + s * 32 * V;
          q[s][f].q = decltype(q[s][f].q){};
          if (k < a.K) q[s][f] = load_once<T, V>(w[f] + k);
        }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int k = k0 + s * 32 * V;
        if (k >= a.K) break;
        float wf[kF][V];
#pragma unroll
        for (int f = 0; f < kF; ++f) q[s][f].get(wf[f]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (r >= n) break;
          float xf[V];
          load_row<T, V>(x + static_cast<int64_t>(r) * a.K + k).get(xf);
#pragma unroll
          for (int f = 0; f < kF; ++f)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[f][r] = fmaf(wf[f][i], xf[i], acc[f][r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r >= n) break;
#pragma unroll
      for (int f = 0; f < kF; ++f) {
        float v = acc[f][r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == f && f0 + f < a.O) {
          if (a.bias) v += static_cast<float>(a.bias[static_cast<int64_t>(e) * a.O + f0 + f]);
          a.y[static_cast<int64_t>(row0 + r) * a.O + f0 + f] = static_cast<T>(v);
        }
      }
    }
  }
}

// kMax: most rows of a call (a group of many rows takes registers that the others of the
// kernel would have to do without).
template <typename T, int V, int kMax>
__global__ void __launch_bounds__(kThreads)
grouped_few_kernel(const __grid_constant__ FewArgs<T> a) {
  __shared__ int s_e, s_bad;
  pdl_trigger();
  if (threadIdx.x == 0) s_e = s_bad = 0;
  __syncthreads();
  pdl_wait();
  // the row's group: the number of groups that end at or before it
  const int row = blockIdx.y;
  int before = 0;
  bool bad = false;
  for (int i = threadIdx.x; i < a.N; i += kThreads) {
    const int b = a.off[i], e = a.off[i + 1];
    bad = bad || b < 0 || e < b || e > a.R;
    before += e <= row;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if ((threadIdx.x & 31) == 0) atomicAdd(&s_e, before);
  if (bad) s_bad = 1;
  __syncthreads();
  const int e = s_e;
  if (blockIdx.x == 0 && row == 0 && threadIdx.x == 0) a.hdr->err = s_bad ? kDevIndexOutOfRange : kDevOk;
  if (s_bad || e >= a.N || a.off[e] != row) return;     // of no group, or not its first
  const int n = a.off[e + 1] - row, o0 = blockIdx.x * kPerCta;
  if (n == 1) few_rows<T, V, 1>(a, e, row, n, o0);
  else if (n == 2) few_rows<T, V, 2>(a, e, row, n, o0);
  else if (n <= 4) few_rows<T, V, 4>(a, e, row, n, o0);
  else if (kMax == 8 || n <= 8) few_rows<T, V, 8>(a, e, row, n, o0);
  else if (kMax == 16 || n <= 16) few_rows<T, V, kMax < 16 ? 8 : 16>(a, e, row, n, o0);
  else few_rows<T, V, kMax>(a, e, row, n, o0);
}

template <typename T, int V>
cudaError_t launch(const GroupedShape& s, const GroupedPlan& p, const int* offsets, const void* x,
                   const void* W, const void* bias, void* y, cudaStream_t stream) {
  const FewArgs<T> a = {static_cast<const T*>(x), static_cast<const T*>(W),
                        static_cast<const T*>(bias), static_cast<T*>(y), offsets, p.hdr,
                        static_cast<int>(s.R), static_cast<int>(s.K), static_cast<int>(s.O),
                        static_cast<int>(s.N)};
  const dim3 grid(static_cast<unsigned>((s.O + kPerCta - 1) / kPerCta), static_cast<unsigned>(s.R));
  count_launch();
  auto* kernel = s.R <= 8 ? grouped_few_kernel<T, V, 8> : grouped_few_kernel<T, V, 16>;
  if constexpr (sizeof(T) == 4)
    if (s.R > 16) kernel = grouped_few_kernel<T, V, 32>;
  return launch_dependent(kernel, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_grouped_few(const GroupedShape& s, const GroupedPlan& p, const int* offsets,
                               const void* x, const void* W, const void* bias, void* y,
                               cudaStream_t stream) {
  if (s.dtype == 1)    // bf16: rows are whole 16-byte pieces
    return launch<__nv_bfloat16, 8>(s, p, offsets, x, W, bias, y, stream);
  const bool wide = s.K % 4 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(W)) & 15) == 0;
  return wide ? launch<float, 4>(s, p, offsets, x, W, bias, y, stream)
              : launch<float, 1>(s, p, offsets, x, W, bias, y, stream);
}

}  // namespace swl
