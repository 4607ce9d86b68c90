// The norms before and after a block, fused with the block's gate, the residual
// scale and the residual addition, and their backward pass.
//
//   n(v; w, b) = (v - mu) rho w + b,  rho = 1 / sqrt(mean((v - mu)^2) + eps),
//                mu = mean(v) (layer norm) or 0 (RMS norm, without b)
//   u_t = n(y_t; w_post, b_post), or y_t without w_post
//   r_t = x_t + gate_t * scale . u_t       (r = x without y)
//   h_t = n(r_t; w_pre, b_pre)             (the next block's input; optional)
//
// Backward, from the gradients dr of r (its other uses) and dh of h, with
// v^ = (v - mu) rho and N(g; v, w) = rho (a - [layer] mean(a) - v^ mean(a v^)),
// a = w . g:
//   D = dr + N(dh; r, w_pre),   dx = D,
//   dgate_t = sum_j D_j scale_j u_j,   dscale = sum_t gate_t D u,
//   du = gate_t scale . D,   dy = N(du; y, w_post) (du without w_post),
//   dw_pre = sum_t dh r^, db_pre = sum_t dh, dw_post = sum_t du y^, db_post = sum_t du.
// The statistics are recomputed from r and y, which the pass reads anyway: the
// forward pass saves nothing.  h is taken from the unrounded r.
//
// Bound: HBM, one read of every input row and one write of every output row
// (forward 4, backward 6 row-sized arrays).  A row is held in registers by a group
// of `span` threads (E elements each, 16 bytes per load where widths and pointers
// allow); sums over the row go through warp shuffles and, for rows wider than a
// warp, one exchange in shared memory behind a barrier of the group alone, so
// several rows are in flight per SM without waiting for one another.  The rows
// ahead are copied to shared memory by cp.async, each thread its own columns, so no
// thread waits for another's copy and no registers hold what is in flight.  All sums are fp32, a
// layer norm's variance is taken about the mean in a second sum.  The parameters'
// gradients are column sums over all rows: a thread keeps its columns' sums in
// registers over all the rows it sees (grid-stride), the groups of a CTA add theirs
// in order, and a second kernel adds the CTAs' sums in order: no atomics, the same
// result every time.
//
// Measured at 32768 x 2048 bf16, RMS norms on both sides, gate and scale: forward 110 us
// (floor 82 us), backward 243 us (floor 123 us); one row of 1024: 2.7 us in a graph.  The
// backward pass issues 60 instructions per element on 16 warps per SM (the column sums
// take their registers) and moves 24 KB of fp32 parameters per row through L1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "kernels.h"
#include "switch_layer.h"

namespace swl {
namespace {

constexpr int kMaxWarps = 16;         // warps per row, at most
constexpr int kMaxWidth = 16384;      // 512 threads x 32 elements
constexpr int kSums = 5;              // column sums: w_pre, b_pre, w_post, b_post, scale

template <typename T, int V>
struct Vec;
template <>
struct Vec<float, 4> {
  float4 q;
  __device__ __forceinline__ void get(float* o) const { o[0] = q.x, o[1] = q.y, o[2] = q.z, o[3] = q.w; }
  __device__ __forceinline__ void set(const float* o) { q = make_float4(o[0], o[1], o[2], o[3]); }
};
template <>
struct Vec<float, 2> {
  float2 q;
  __device__ __forceinline__ void get(float* o) const { o[0] = q.x, o[1] = q.y; }
};
template <>
struct Vec<float, 1> {
  float q;
  __device__ __forceinline__ void get(float* o) const { o[0] = q; }
  __device__ __forceinline__ void set(const float* o) { q = o[0]; }
};
__device__ __forceinline__ unsigned pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&v);
}
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 q;
  __device__ __forceinline__ void get(float* o) const {
    const unsigned u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(u[i] << 16);
      o[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float* o) {
    q = make_uint4(pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]), pack2(o[6], o[7]));
  }
};
template <>
struct Vec<__nv_bfloat16, 2> {
  unsigned q;
  __device__ __forceinline__ void get(float* o) const {
    o[0] = __uint_as_float(q << 16), o[1] = __uint_as_float(q & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float* o) { q = pack2(o[0], o[1]); }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  unsigned short q;
  __device__ __forceinline__ void get(float* o) const { o[0] = __uint_as_float(static_cast<unsigned>(q) << 16); }
  __device__ __forceinline__ void set(const float* o) {
    const __nv_bfloat16 v = __float2bfloat16_rn(o[0]);
    q = *reinterpret_cast<const unsigned short*>(&v);
  }
};

// Two fp32 operations in one instruction, each rounded as by itself: the element-wise
// work is what these kernels issue most.  d may be an operand.
__device__ __forceinline__ void fma2(float* d, const float* a, const float* b, const float* c) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void mul2(float* d, const float* a, const float* b) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void add2(float* d, const float* a, const float* b) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
// A scalar for both halves.
struct Both {
  float v[2];
  __device__ __forceinline__ explicit Both(float x) : v{x, x} {}
  __device__ __forceinline__ operator const float*() const { return v; }
};

struct Params {
  const float* w_pre;
  const float* b_pre;
  const float* w_post;
  const float* b_post;
  const float* scale;
  const float* gate;
  float eps, inv_d;
  int d;
  int64_t T;
  int span;           // threads per row (a power of two)
};
struct FwdArgs {
  Params p;
  const void* x;
  const void* y;
  void* r;
  void* h;
};
struct BwdArgsN {
  Params p;
  const void* dr;
  const void* dh;
  const void* r;
  const void* y;
  void* dx;
  void* dy;
  float* dgate;
  float* part;        // [grid][kSums][d] column sums of each CTA
  unsigned wanted;    // bit s: column sum s is asked for
};

// A thread's place: its group's rows and its own columns (vector k starts at
// column (k * span + tid) * V).
template <int V, int E>
struct Lane {
  int tid, group, groups, span;     // span: threads of a group
  __device__ __forceinline__ explicit Lane(int threads_per_row) {
    span = threads_per_row;
    group = threadIdx.x / span;
    tid = threadIdx.x - group * span;
    groups = blockDim.x / span;
  }
  __device__ __forceinline__ int col(int k) const { return (k * span + tid) * V; }
};

template <typename T, int V, int E>
struct Row {
  Vec<T, V> v[E / V];
  __device__ __forceinline__ void load(const void* base, int64_t row, bool valid, int d,
                                       const Lane<V, E>& l) {
    const T* p = static_cast<const T*>(base) + row * d;
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
      const int c = l.col(k);
      if (valid && c < d) v[k].q = *reinterpret_cast<const decltype(v[k].q)*>(p + c);
      else v[k].q = decltype(v[k].q){};
    }
  }
  __device__ __forceinline__ void get(float (&o)[E]) const {
#pragma unroll
    for (int k = 0; k < E / V; ++k) v[k].get(o + k * V);
  }
};

// The rows ahead of the one being worked on (kStages - 1 of them), for A arrays:
// vector k of array a of a stage lies at [(stage A + a) E / V + k][thread].  Every
// thread copies and reads its own columns only.  Vectors under 4 bytes (cp.async
// has none) and rows too wide for shared memory are loaded where they are used.  One row
// ahead: a second one takes the L1 that the parameter vectors are read from (32768 x 2048
// backward: 261 against 243 us).
constexpr int kStages = 2;
template <typename T, int V, int E>
constexpr bool use_ring() {
  return sizeof(T) * V >= 4 && sizeof(T) * E <= 32;
}
template <typename T, int V, int E, int A>
struct Ring {
  static constexpr int kBytes = sizeof(T) * V;
  static constexpr bool kOn = use_ring<T, V, E>();
  unsigned char* smem;
  uint32_t base;
  int fill = 0, take = 0;
  __device__ __forceinline__ explicit Ring(unsigned char* s)
      : smem(s), base(static_cast<uint32_t>(__cvta_generic_to_shared(s))) {}
  __device__ __forceinline__ int slot(int stage, int a, int k) const {
    return (((stage * A + a) * (E / V) + k) * static_cast<int>(blockDim.x) +
            static_cast<int>(threadIdx.x)) * kBytes;
  }
  __device__ __forceinline__ void put(int a, const void* src, int64_t row, bool valid, int d,
                                      const Lane<V, E>& l) const {
    const T* p = static_cast<const T*>(src) + row * d;
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
      const int c = l.col(k);
      const bool in = valid && c < d;
      // zero bytes are read (and the slot zero-filled) past the row and past T
      const T* from = in ? p + c : static_cast<const T*>(src);
      const int n = in ? kBytes : 0;
      if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + slot(fill, a, k)),
                     "l"(from), "r"(n)
                     : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(base + slot(fill, a, k)),
                     "l"(from), "n"(kBytes < 4 ? 4 : kBytes), "r"(n)
                     : "memory");
    }
  }
  __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + 1 == kStages ? 0 : fill + 1;
  }
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
  }
  __device__ __forceinline__ void get(int a, float (&o)[E]) const {
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
      Vec<T, V> v;
      v.q = *reinterpret_cast<const decltype(v.q)*>(smem + slot(take, a, k));
      v.get(o + k * V);
    }
  }
  __device__ __forceinline__ void next() { take = take + 1 == kStages ? 0 : take + 1; }
};

template <typename T, int V, int E>
__device__ __forceinline__ void store_row(void* base, int64_t row, bool valid, int d,
                                          const Lane<V, E>& l, const float (&o)[E]) {
  T* p = static_cast<T*>(base) + row * d;
#pragma unroll
  for (int k = 0; k < E / V; ++k) {
    const int c = l.col(k);
    Vec<T, V> v;
    v.set(o + k * V);
    if (valid && c < d) *reinterpret_cast<decltype(v.q)*>(p + c) = v.q;
  }
}
// A parameter vector's values at this thread's columns (fp32; the loads hit L1).
template <int V, int E>
__device__ __forceinline__ void load_param(const float* p, int d, const Lane<V, E>& l,
                                           float (&o)[E]) {
  constexpr int F = V > 4 ? 4 : V;      // floats per load
#pragma unroll
  for (int k = 0; k < E / V; ++k) {
    const int c = l.col(k);
#pragma unroll
    for (int i = 0; i < V; i += F) {
      Vec<float, F> v;
      v.q = decltype(v.q){};
      if (c < d) v.q = __ldg(reinterpret_cast<const decltype(v.q)*>(p + c + i));
      v.get(o + k * V + i);
    }
  }
}

// Sums over the row of N values per thread, the same in every thread of the
// group.  The two buffers alternate, so one barrier per sum is enough: a thread
// that writes a buffer again has passed the next sum's barrier, which follows
// every read.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int span, float (*buf)[4][kMaxWarps],
                                        int& turn) {
  if (span < 32) {
    for (int o = span >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (span == 32) return;
  const int warps = span >> 5, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / span, first = group * warps;
  float(*b)[kMaxWarps] = buf[turn];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) b[i][warp] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(span) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (warps == 2) {
      const float2 q = *reinterpret_cast<const float2*>(&b[i][first]);
      v[i] = q.x + q.y;
    } else {
      v[i] = 0.f;
      for (int w = 0; w < warps; w += 4) {
        const float4 q = *reinterpret_cast<const float4*>(&b[i][first + w]);
        v[i] += (q.x + q.y) + (q.z + q.w);
      }
    }
  }
}

// v becomes v - mu in the row's columns, zero behind them.
template <int V, int E>
__device__ __forceinline__ void subtract(float (&v)[E], float mu, int d, const Lane<V, E>& l) {
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = l.col(i / V) < d ? v[i] - mu : 0.f;
}

// v becomes v - mu (layer norm; v itself for RMS norm); returns rho.
template <bool kLayer, int V, int E>
__device__ __forceinline__ float center(float (&v)[E], const Params& p, const Lane<V, E>& l,
                                        float (*buf)[4][kMaxWarps], int& turn) {
  if constexpr (kLayer) {
    float t[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; i += 2) add2(t, t, v + i);       // columns past d hold zeros
    float s[1] = {t[0] + t[1]};
    row_sum(s, p.span, buf, turn);
    subtract(v, s[0] * p.inv_d, p.d, l);
  }
  float t[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < E; i += 2) fma2(t, v + i, v + i, t);
  float s[1] = {t[0] + t[1]};
  row_sum(s, p.span, buf, turn);
  return rsqrtf(fmaf(s[0], p.inv_d, p.eps));
}

template <typename T, int V, int E, int kThreads, bool kLayer>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 1)
norm_residual_kernel(const __grid_constant__ FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float buf[2][4][kMaxWarps];
  const Params& p = a.p;
  const Lane<V, E> l(p.span);
  using R = Ring<T, V, E, 2>;
  R ring(smem);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * l.groups;
  // every group of a CTA takes the same number of steps (a warp may hold several groups)
  const int64_t first = static_cast<int64_t>(blockIdx.x) * l.groups;
  int turn = 0;
  auto fetch = [&](int64_t t) {
    if (t < p.T + l.groups) {      // (past the last row nothing is read)
      ring.put(0, a.x, t, t < p.T, p.d, l);
      if (a.y) ring.put(1, a.y, t, t < p.T, p.d, l);
    }
    ring.commit();
  };
  if constexpr (R::kOn) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + l.group + s * stride);
  }
  for (int64_t base = first; base < p.T; base += stride) {
    const int64_t row = base + l.group;
    const bool valid = row < p.T;
    const float g = p.gate && valid ? p.gate[row] : 1.f;
    float r[E], u[E], w[E];
    if constexpr (R::kOn) {
      ring.wait();
      ring.get(0, r);
      if (a.y) ring.get(1, u);
      ring.next();
      fetch(row + (kStages - 1) * stride);     // into the stage read in the last step
    } else {
      Row<T, V, E> q;
      q.load(a.x, row, valid, p.d, l);
      q.get(r);
      if (a.y) {
        q.load(a.y, row, valid, p.d, l);
        q.get(u);
      }
    }
    if (a.y) {
      float f = g;
      if (p.w_post) {
        const float rho = center<kLayer>(u, p, l, buf, turn);
        load_param(p.w_post, p.d, l, w);
        if (kLayer && p.b_post) {
          float b[E];
          load_param(p.b_post, p.d, l, b);
          const Both rr(rho);
#pragma unroll
          for (int i = 0; i < E; i += 2) {
            mul2(u + i, u + i, rr);
            fma2(u + i, u + i, w + i, b + i);
          }
        } else {
          f *= rho;
#pragma unroll
          for (int i = 0; i < E; i += 2) mul2(u + i, u + i, w + i);
        }
      }
      if (p.scale) {
        load_param(p.scale, p.d, l, w);
#pragma unroll
        for (int i = 0; i < E; i += 2) mul2(u + i, u + i, w + i);
      }
      const Both ff(f);
#pragma unroll
      for (int i = 0; i < E; i += 2) fma2(r + i, ff, u + i, r + i);
      store_row<T>(a.r, row, valid, p.d, l, r);
    }
    if (a.h) {
      const Both rr(center<kLayer>(r, p, l, buf, turn));
      load_param(p.w_pre, p.d, l, w);
      if (kLayer && p.b_pre) {
        load_param(p.b_pre, p.d, l, u);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          mul2(r + i, r + i, rr);
          fma2(r + i, r + i, w + i, u + i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          mul2(r + i, r + i, rr);
          mul2(r + i, r + i, w + i);
        }
      }
      store_row<T>(a.h, row, valid, p.d, l, r);
    }
  }
  if constexpr (R::kOn) asm volatile("cp.async.wait_all;" ::: "memory");
}

// Row statistics of the backward pass: v becomes v - mu; returns rho, and
// (through m0, m1) mean(a) and mean(a (v - mu)).
template <bool kLayer, int V, int E>
__device__ __forceinline__ float center_with(float (&v)[E], const float (&a)[E], const Params& p,
                                             const Lane<V, E>& l, float (*buf)[4][kMaxWarps],
                                             int& turn, float& m0, float& m1) {
  m0 = 0.f;
  if constexpr (kLayer) {
    float t[2] = {0.f, 0.f}, u[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      add2(t, t, v + i);
      add2(u, u, a + i);
    }
    float s[2] = {t[0] + t[1], u[0] + u[1]};
    row_sum(s, p.span, buf, turn);
    m0 = s[1] * p.inv_d;
    subtract(v, s[0] * p.inv_d, p.d, l);
  }
  float t[2] = {0.f, 0.f}, u[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    fma2(t, v + i, v + i, t);
    fma2(u, a + i, v + i, u);
  }
  float s[2] = {t[0] + t[1], u[0] + u[1]};
  row_sum(s, p.span, buf, turn);
  m1 = s[1] * p.inv_d;
  return rsqrtf(fmaf(s[0], p.inv_d, p.eps));
}

template <typename T, int V, int E, int kThreads, bool kLayer>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1)
norm_residual_bwd_kernel(const __grid_constant__ BwdArgsN a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float buf[2][4][kMaxWarps];
  const Params& p = a.p;
  const Lane<V, E> l(p.span);
  using R = Ring<T, V, E, 4>;
  R ring(smem);
  if (a.wanted) pdl_trigger();      // the column sums' kernel follows
  const int64_t stride = static_cast<int64_t>(gridDim.x) * l.groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * l.groups;
  int turn = 0;
  float acc[kSums][E];      // (RMS norm: the two bias sums are never touched)
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int i = 0; i < E; ++i) acc[s][i] = 0.f;
  auto fetch = [&](int64_t t) {
    if (t < p.T + l.groups) {
      const bool in = t < p.T;
      if (a.dr) ring.put(0, a.dr, t, in, p.d, l);
      if (a.dh) {
        ring.put(1, a.dh, t, in, p.d, l);
        ring.put(2, a.r, t, in, p.d, l);
      }
      if (a.y) ring.put(3, a.y, t, in, p.d, l);
    }
    ring.commit();
  };
  if constexpr (R::kOn) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + l.group + s * stride);
  }
  for (int64_t base = first; base < p.T; base += stride) {
    const int64_t row = base + l.group;
    const bool valid = row < p.T;
    float D[E], w[E], g[E], v[E], y[E];
    // dx may be dr: a row's dr is read here, before its dx is written
    auto take = [&](int k, const void* src, float (&o)[E]) {
      if constexpr (R::kOn) {
        ring.get(k, o);
      } else {
        Row<T, V, E> q;
        q.load(src, row, valid, p.d, l);
        q.get(o);
      }
    };
    if constexpr (R::kOn) ring.wait();
    if (a.dr) {
      take(0, a.dr, D);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) D[i] = 0.f;
    }
    if (a.dh) {
      take(1, a.dh, g);
      take(2, a.r, v);
    }
    if (a.dh) {
      load_param(p.w_pre, p.d, l, w);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        if constexpr (kLayer) add2(acc[1] + i, acc[1] + i, g + i);
        mul2(w + i, g + i, w + i);          // a = w dh
      }
      float m0, m1;
      const float rho = center_with<kLayer>(v, w, p, l, buf, turn, m0, m1);
      const Both rr(rho), mm0(-m0), mm2(-m1 * rho * rho);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        float t[2];
        if constexpr (kLayer) add2(w + i, w + i, mm0);
        fma2(t, mm2, v + i, w + i);
        fma2(D + i, t, rr, D + i);
        mul2(v + i, v + i, rr);
        fma2(acc[0] + i, g + i, v + i, acc[0] + i);
      }
    }
    store_row<T>(a.dx, row, valid, p.d, l, D);
    if (a.y) take(3, a.y, y);
    if constexpr (R::kOn) {
      ring.next();
      fetch(row + (kStages - 1) * stride);     // into the stage read in the last step
    }
    if (!a.y) continue;
    const float gate = p.gate && valid ? p.gate[row] : 1.f;
    // without the gate, which its own gradient needs; sc: the residual scale
    float sc[E];
    if (p.scale) {
      load_param(p.scale, p.d, l, sc);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) sc[i] = 1.f;
    }
    if (p.w_post) {
      const float rho = center<kLayer>(y, p, l, buf, turn);
      load_param(p.w_post, p.d, l, w);
      float s[3] = {0.f, 0.f, 0.f};       // sums of scale D w, scale D w y^, scale D b
      const Both gg(gate), rr(rho);
      float t0[2] = {0.f, 0.f}, t1[2] = {0.f, 0.f};
      if (kLayer && p.b_post) {
        float bias[E], t2[2] = {0.f, 0.f};
        load_param(p.b_post, p.d, l, bias);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          float z[2];
          mul2(z, gg, D + i);
          fma2(acc[4] + i, z, bias + i, acc[4] + i);
          mul2(z, D + i, sc + i);
          fma2(t2, z, bias + i, t2);
        }
        s[2] = t2[0] + t2[1];
      }
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        float gy[2], z[2];
        mul2(y + i, y + i, rr);             // y^
        mul2(gy, gg, y + i);
        mul2(z, D + i, sc + i);
        fma2(acc[2] + i, z, gy, acc[2] + i);
        if constexpr (kLayer) fma2(acc[3] + i, gg, z, acc[3] + i);
        mul2(D + i, D + i, w + i);
        fma2(acc[4] + i, D + i, gy, acc[4] + i);
        mul2(D + i, z, w + i);              // scale D w
        if constexpr (kLayer) add2(t0, t0, D + i);
        fma2(t1, D + i, y + i, t1);
      }
      s[0] = t0[0] + t0[1];
      s[1] = t1[0] + t1[1];
      if constexpr (kLayer) {
        row_sum(s, p.span, buf, turn);
      } else {
        float one[1] = {s[1]};
        row_sum(one, p.span, buf, turn);
        s[1] = one[0];
      }
      if (a.dgate && valid && l.tid == 0) a.dgate[row] = s[1] + s[2];
      const Both m0(-s[0] * p.inv_d), m1(-s[1] * p.inv_d), f(gate * rho);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        if constexpr (kLayer) add2(D + i, D + i, m0);
        fma2(D + i, m1, y + i, D + i);
        mul2(D + i, D + i, f);
      }
    } else {
      const Both gg(gate);
      float t1[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        float gy[2];
        mul2(gy, gg, y + i);
        fma2(acc[4] + i, D + i, gy, acc[4] + i);
        mul2(D + i, D + i, sc + i);
        fma2(t1, D + i, y + i, t1);
        mul2(D + i, D + i, gg);
      }
      if (a.dgate) {
        float s[1] = {t1[0] + t1[1]};
        row_sum(s, p.span, buf, turn);
        if (valid && l.tid == 0) a.dgate[row] = s[0];
      }
    }
    store_row<T>(a.dy, row, valid, p.d, l, D);
  }
  if constexpr (R::kOn) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float* const columns = reinterpret_cast<float*>(smem);   // [d], the ring is done with
  // this CTA's column sums: its groups add theirs in order
  float* part = a.part + static_cast<size_t>(blockIdx.x) * kSums * p.d;
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    if (!(a.wanted >> s & 1u)) continue;
    for (int g = 0; g < l.groups; ++g) {
      if (l.groups > 1) __syncthreads();
      if (l.group != g) continue;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = l.col(i / V) + i % V;
        if (c >= p.d) continue;
        const float v = g == 0 ? acc[s][i] : acc[s][i] + columns[c];
        if (g == l.groups - 1) part[static_cast<size_t>(s) * p.d + c] = v;
        else columns[c] = v;
      }
    }
  }
}

struct SumArgs {
  const float* part;
  float* out[kSums];
  int parts, d;
};
// out[s][c] = sum over the CTAs' partial sums, in a fixed order: 16 interleaved
// runs of CTAs per column, then the runs.
__global__ void __launch_bounds__(512)
norm_residual_sum_kernel(const __grid_constant__ SumArgs a) {
  __shared__ float buf[16][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5, s = blockIdx.y;
  pdl_wait();
  if (!a.out[s]) return;
  float v = 0.f;
  if (c < a.d) {
    const float* p = a.part + static_cast<size_t>(s) * a.d + c;
#pragma unroll 4
    for (int i = k; i < a.parts; i += 16) v += p[static_cast<size_t>(i) * kSums * a.d];
  }
  buf[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k == 0 && c < a.d) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += buf[i][threadIdx.x & 31];
    a.out[s][c] = v;
  }
}

// ---------------------------------------------------------------- host
struct Plan {
  int V, E, span, threads, groups;
};
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Elements per thread E and threads per row.  More elements per thread spread a
// row's fixed work (sums, addresses) over more of them (32768 x 2048 bf16 backward: 267 us
// with 16, 297 with 8); fewer give a small batch more threads, and keep in registers a layer
// norm's backward pass with its five column sums per element (8192 x 4096: 256 us with 8
// on 512 threads, 310 with 16) and the narrow loads of odd widths.  `elems`: pointers into
// rows; `params`: fp32 vectors.
Plan make_plan(int64_t T, int64_t d, int dtype, bool small_e, int sms,
               std::initializer_list<const void*> elems,
               std::initializer_list<const float*> params) {
  Plan q;
  const int full = dtype == SWL_BF16 ? 8 : 4;
  auto fits = [&](int v) {
    if (d % v) return false;
    for (const void* e : elems)
      if (!aligned(e, dtype == SWL_BF16 ? 2 * v : 4 * v)) return false;
    for (const float* f : params)
      if (!aligned(f, v > 4 ? 16 : 4 * v)) return false;
    return true;
  };
  q.V = fits(full) ? full : dtype == SWL_BF16 && fits(2) ? 2 : 1;
  q.threads = 256;
  // E = 16 (bf16) once its threads fill the GPU's SMs with two warps per scheduler
  if (dtype == SWL_BF16 && d <= 4096) {
    const bool few = small_e || q.V < 8;
    q.E = few || (d <= 2048 && (d <= 256 || T * (d / 16) < sms * 256ll)) ? 8 : 16;
    if (q.E == 8 && d > 2048) q.threads = 512;
  } else if (dtype == SWL_F32 && d <= 2048) {
    q.E = 8;
  } else {
    q.threads = 512;
    q.E = dtype == SWL_F32 && d <= 4096 ? 8 : d <= 8192 ? 16 : 32;
  }
  q.span = 8;
  while (q.span * q.E < d) q.span *= 2;
  q.groups = q.threads / q.span;
  return q;
}

template <typename F>
bool dispatch(const Plan& q, int dtype, bool layer, F f) {
#define SWL_L(T, V, E, H) \
  return layer ? f.template run<T, V, E, H, true>() : f.template run<T, V, E, H, false>();
#define SWL_V(T, V)                                      \
  if (q.threads == 256) {                                \
    if (q.E == 8) { SWL_L(T, V, 8, 256) }                \
    if constexpr (sizeof(T) * V == 16 && sizeof(T) == 2) { SWL_L(T, V, 16, 256) } \
  }                                                      \
  if (q.E == 8) { SWL_L(T, V, 8, 512) }                  \
  if (q.E == 16) { SWL_L(T, V, 16, 512) }                \
  SWL_L(T, V, 32, 512)
  if (dtype == SWL_BF16) {
    if (q.V == 8) { SWL_V(__nv_bfloat16, 8) }
    if (q.V == 2) { SWL_V(__nv_bfloat16, 2) }
    SWL_V(__nv_bfloat16, 1)
  }
  if (q.V == 4) { SWL_V(float, 4) }
  SWL_V(float, 1)
#undef SWL_V
#undef SWL_L
}

// Shared memory beyond 48 KB (with the static arrays) has to be asked for.
template <typename K>
bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 40 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bytes)) == cudaSuccess;
}

struct RunFwd {
  const FwdArgs& a;
  const Plan& q;
  int grid;
  cudaStream_t st;
  template <typename T, int V, int E, int H, bool L>
  bool run() {
    const size_t smem = use_ring<T, V, E>() ? size_t{kStages} * 2 * H * E * sizeof(T) : 0;
    if (!allow_smem(norm_residual_kernel<T, V, E, H, L>, smem)) return false;
    norm_residual_kernel<T, V, E, H, L><<<grid, H, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess;
  }
};
struct RunBwd {
  const BwdArgsN& a;
  const Plan& q;
  int grid;
  cudaStream_t st;
  template <typename T, int V, int E, int H, bool L>
  bool run() {
    size_t smem = use_ring<T, V, E>() ? size_t{kStages} * 4 * H * E * sizeof(T) : 0;
    if (q.groups > 1 && smem < static_cast<size_t>(a.p.d) * 4) smem = static_cast<size_t>(a.p.d) * 4;
    if (!allow_smem(norm_residual_bwd_kernel<T, V, E, H, L>, smem)) return false;
    norm_residual_bwd_kernel<T, V, E, H, L><<<grid, H, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess;
  }
};

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

constexpr int kBwdCtasPerSm = 2;
constexpr int kMaxSms = 256;     // the workspace is sized without asking the device

swl_status check(int64_t T, int64_t d, int dtype, const swl_norm* n, bool y, bool pre) {
  if (T < 0 || d <= 0 || (dtype != SWL_F32 && dtype != SWL_BF16) || !n) return SWL_ERR_INVALID_ARG;
  if (n->kind != SWL_NORM_RMS && n->kind != SWL_NORM_LAYER) return SWL_ERR_INVALID_ARG;
  if (!std::isfinite(n->eps) || !(n->eps > 0)) return SWL_ERR_INVALID_ARG;
  if (n->kind == SWL_NORM_RMS && (n->b_pre || n->b_post)) return SWL_ERR_INVALID_ARG;
  if ((n->b_pre && !n->w_pre) || (n->b_post && !n->w_post)) return SWL_ERR_INVALID_ARG;
  if (!y && (n->w_post || n->scale)) return SWL_ERR_INVALID_ARG;
  if (!y && !pre) return SWL_ERR_INVALID_ARG;
  if (pre != (n->w_pre != nullptr)) return SWL_ERR_INVALID_ARG;
  if (d > kMaxWidth || T > (int64_t{1} << 40)) return SWL_ERR_UNSUPPORTED;
  for (const float* f : {n->w_pre, n->b_pre, n->w_post, n->b_post, n->scale})
    if (!aligned(f, 4)) return SWL_ERR_UNSUPPORTED;
  return SWL_OK;
}

Params params_of(int64_t T, int64_t d, const swl_norm* n, const float* gate, int span) {
  return {n->w_pre, n->b_pre, n->w_post, n->b_post, n->scale, gate, n->eps,
          static_cast<float>(1.0 / static_cast<double>(d)), static_cast<int>(d), T, span};
}

// Do [a, a + na) and [b, b + nb) share a byte?  (NULL: no)
bool meet(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace swl

using namespace swl;

extern "C" swl_status switch_layer_norm_residual(int64_t T, int64_t d, int dtype, const void* x,
                                                 const void* y, const float* gate,
                                                 const swl_norm* norm, void* r, void* h,
                                                 void* stream) {
  swl_status st = check(T, d, dtype, norm, y != nullptr || T == 0, h != nullptr || (T == 0 && norm && norm->w_pre));
  if (st != SWL_OK) return st;
  if (T == 0) return SWL_OK;
  if (!x || (y != nullptr) != (r != nullptr) || (gate && !y)) return SWL_ERR_INVALID_ARG;
  const uintptr_t e = dtype == SWL_BF16 ? 2 : 4;
  for (const void* p : {x, y, static_cast<const void*>(r), static_cast<const void*>(h)})
    if (!aligned(p, e)) return SWL_ERR_UNSUPPORTED;
  if (!aligned(gate, 4)) return SWL_ERR_UNSUPPORTED;
  // r and h may be x or y themselves (a thread has read its columns before it
  // writes them), but not lie across them, nor on a parameter
  const size_t n = static_cast<size_t>(T) * d * e, nd = static_cast<size_t>(d) * 4;
  if (meet(r, n, h, n)) return SWL_ERR_INVALID_ARG;
  for (const void* o : {static_cast<const void*>(r), static_cast<const void*>(h)}) {
    for (const void* i : {x, y})
      if (o != i && meet(o, n, i, n)) return SWL_ERR_INVALID_ARG;
    if (meet(o, n, gate, static_cast<size_t>(T) * 4)) return SWL_ERR_INVALID_ARG;
    for (const float* f : {norm->w_pre, norm->b_pre, norm->w_post, norm->b_post, norm->scale})
      if (meet(o, n, f, nd)) return SWL_ERR_INVALID_ARG;
  }
  const int sms = sm_count();
  if (sms <= 0) return SWL_ERR_CUDA;
  const Plan q = make_plan(T, d, dtype, false, sms, {x, y, r, h},
                           {norm->w_pre, norm->b_pre, norm->w_post, norm->b_post, norm->scale});
  const FwdArgs a = {params_of(T, d, norm, gate, q.span), x, y, r, h};
  const int64_t want = (T + q.groups - 1) / q.groups;
  const int64_t most = static_cast<int64_t>(sms) * (q.threads == 256 ? 3 : 1);
  RunFwd run = {a, q, static_cast<int>(want < most ? want : most), static_cast<cudaStream_t>(stream)};
  if (!dispatch(q, dtype, norm->kind == SWL_NORM_LAYER, run)) return SWL_ERR_CUDA;
  count_launch();
  return SWL_OK;
}

extern "C" swl_status switch_layer_norm_residual_backward_workspace_size(int64_t T, int64_t d,
                                                                         int dtype,
                                                                         size_t* bytes) {
  if (T < 0 || d <= 0 || (dtype != SWL_F32 && dtype != SWL_BF16) || !bytes)
    return SWL_ERR_INVALID_ARG;
  if (d > kMaxWidth || T > (int64_t{1} << 40)) return SWL_ERR_UNSUPPORTED;
  const int64_t most = static_cast<int64_t>(kMaxSms) * kBwdCtasPerSm;
  *bytes = static_cast<size_t>(T < most ? (T > 0 ? T : 1) : most) * kSums * d * 4;
  return SWL_OK;
}

extern "C" swl_status switch_layer_norm_residual_backward(
    int64_t T, int64_t d, int dtype, const void* dr, const void* dh, const void* r, const void* y,
    const float* gate, const swl_norm* norm, const swl_norm_grads* grads, void* workspace,
    size_t workspace_bytes, void* stream) {
  const bool pre = norm && norm->w_pre;
  swl_status st = check(T, d, dtype, norm, y != nullptr || T == 0, pre);
  if (st != SWL_OK) return st;
  if (!grads || !workspace) return SWL_ERR_INVALID_ARG;
  const swl_norm_grads& o = *grads;
  if (T > 0) {
    if ((dh != nullptr) != pre || (pre && !r) || (!dr && !dh) || !o.dx ||
        (y != nullptr) != (o.dy != nullptr) || (gate && !y) || (o.dgate && !gate))
      return SWL_ERR_INVALID_ARG;
  }
  if ((o.dw_pre && !norm->w_pre) || (o.db_pre && !norm->b_pre) || (o.dw_post && !norm->w_post) ||
      (o.db_post && !norm->b_post) || (o.dscale && !norm->scale))
    return SWL_ERR_INVALID_ARG;
  const uintptr_t e = dtype == SWL_BF16 ? 2 : 4;
  const void* in[4] = {dr, dh, r, y};
  for (const void* p : in)
    if (!aligned(p, e)) return SWL_ERR_UNSUPPORTED;
  float* const sums[kSums] = {o.dw_pre, o.db_pre, o.dw_post, o.db_post, o.dscale};
  for (const float* p : sums)
    if (!aligned(p, 4)) return SWL_ERR_UNSUPPORTED;
  if (!aligned(o.dx, e) || !aligned(o.dy, e) || !aligned(o.dgate, 4) || !aligned(gate, 4) ||
      !aligned(workspace, 256))
    return SWL_ERR_UNSUPPORTED;
  size_t need = 0;
  st = switch_layer_norm_residual_backward_workspace_size(T, d, dtype, &need);
  if (st != SWL_OK) return st;
  if (workspace_bytes < need) return SWL_ERR_WORKSPACE;
  // what is written must not lie on what is read or on one another; dx may be dr
  struct Span {
    const void* p;
    size_t n;
  };
  const size_t n = static_cast<size_t>(T) * d * e, nd = static_cast<size_t>(d) * 4, nt = static_cast<size_t>(T) * 4;
  const Span out[9] = {{o.dx, n}, {o.dy, n}, {o.dgate, nt}, {sums[0], nd}, {sums[1], nd},
                       {sums[2], nd}, {sums[3], nd}, {sums[4], nd}, {workspace, need}};
  const Span read[10] = {{dr, n}, {dh, n}, {r, pre ? n : 0}, {y, n}, {gate, nt}, {norm->w_pre, nd},
                         {norm->b_pre, nd}, {norm->w_post, nd}, {norm->b_post, nd}, {norm->scale, nd}};
  for (int i = 0; i < 9; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(out[i].p, out[i].n, out[j].p, out[j].n)) return SWL_ERR_INVALID_ARG;
    for (int j = 0; j < 10; ++j)
      if (meet(out[i].p, out[i].n, read[j].p, read[j].n) && !(i == 0 && j == 0 && o.dx == dr))
        return SWL_ERR_INVALID_ARG;
  }
  const int sms = sm_count();
  if (sms <= 0) return SWL_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  SumArgs s = {static_cast<const float*>(workspace), {}, 0, static_cast<int>(d)};
  unsigned wanted = 0;
  for (int i = 0; i < kSums; ++i) {
    s.out[i] = sums[i];
    wanted |= sums[i] ? 1u << i : 0u;
  }
  if (T > 0) {
    const Plan q = make_plan(T, d, dtype, norm->kind == SWL_NORM_LAYER, sms, {dr, dh, pre ? r : nullptr, y, o.dx, o.dy},
                             {norm->w_pre, norm->b_pre, norm->w_post, norm->b_post, norm->scale});
    const BwdArgsN a = {params_of(T, d, norm, gate, q.span), dr, dh, r, y, o.dx, o.dy, o.dgate,
                        static_cast<float*>(workspace), wanted};
    const int64_t want = (T + q.groups - 1) / q.groups;
    const int64_t most = static_cast<int64_t>(sms < kMaxSms ? sms : kMaxSms) * (q.threads == 256 ? kBwdCtasPerSm : 1);
    s.parts = static_cast<int>(want < most ? want : most);
    RunBwd run = {a, q, s.parts, cs};
    if (!dispatch(q, dtype, norm->kind == SWL_NORM_LAYER, run)) return SWL_ERR_CUDA;
    count_launch();
  }
  if (wanted) {
    if (launch_dependent(norm_residual_sum_kernel, dim3(static_cast<unsigned>((d + 31) / 32), kSums),
                         dim3(512), 0, cs, s) != cudaSuccess)
      return SWL_ERR_CUDA;
    count_launch();
  }
  return SWL_OK;
}
