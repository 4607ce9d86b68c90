// One AdamW step over many tensors, one launch per kind of tensor, the states in 32
// or 8 bits.
//
// Per element, with g scaled by *grad_scale, t = steps made + 1 and lr scaled by
// *lr_scale:
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32, the bias corrections in fp64.  Every operation on the states is rounded
// on its own (no contraction), so that the 8-bit codes are a fixed function of the
// inputs whatever the compiler does; the weight's update, which nothing is rounded
// from to a code, takes the division to two units of the last place.  bf16
// parameters are rounded from w once; with an fp32 master copy w is read from
// and kept there, and the bf16 parameter is only written.
//
// 8-bit states: blocks of 256 consecutive elements share an fp32 scale, the largest
// magnitude over 448 (the largest e4m3 number).  m is held as e4m3 times the scale, rounded
// to nearest (its moving average renews a tenth of it per step with beta1 = 0.9, more than
// half a spacing; with a larger beta1 less).  v is held by its root: r = sqrt(v) has half
// the exponent range, so e4m3's 2^-9..448 spans 35 binary orders of v.  The root is rounded
// stochastically to three mantissa bits with 16 random bits per element: with b2 near 1 a
// step changes r by far less than half a spacing, and rounding to nearest would never let
// v move.  From 2^-6 down (1/28672 of the block's largest root, 30 of the 35 orders above
// it) e4m3 has one spacing, 2^-9, and the conversion rounds to that, to nearest: there a
// root may stand still, which the interface says.  The bits come from a counter (element
// pair, step, seed) through two multiply-xorshift rounds, so a step can be repeated
// exactly.  A non-zero r keeps at least the smallest code, so no element's denominator
// falls to eps alone; a block whose largest magnitude is under 2^-100 is held as zeros.
// The step itself uses the unrounded m and v.
//
// Bound: HBM.  Per element 12 bytes of fp32 weight and gradient (bf16: 6, with a
// master 12) and 16 bytes of fp32 states or 4.06 of 8-bit ones.  One warp takes one
// 256-element block at a time, four elements per lane twice, so that every type is
// read in whole vectors (fp32 16 bytes, bf16 8, codes 4) and a block's two maxima
// are five shuffles each.  The tensor table travels in the kernel's parameters
// (nothing to copy or allocate, so a captured call replays as it is) and the grid is
// persistent, so the corrections are computed once per CTA (256 threads, three CTAs per
// SM: 635 us at the size below; two 637, 128 threads with five or six CTAs 657 and 653).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <memory>
#include <new>
#include <type_traits>

#include "kernels.h"
#include "switch_layer.h"

namespace swl {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamBlock = SWL_ADAMW_BLOCK;         // elements that share a scale
constexpr int kChunkBlocks = kAdamWarps;            // blocks a CTA takes at a time
constexpr int kTableMax = 160;                      // tensors per launch (parameter space)
constexpr float kLeast = 7.888609052210118e-31f;    // 2^-100

struct AdamwEntry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  long long n;
  double wd;
  unsigned first;    // chunks of earlier tensors of this launch
};
template <int kMax>
struct AdamwTable {
  AdamwEntry t[kMax];
  int count;
  int chunks;
  int* step;               // [2]: steps made, arrivals of this launch's CTAs
  const float* grad_scale;
  const float* lr_scale;
  double lr, beta1, beta2;
  float eps, b1, c1, b2, c2;
  unsigned seed;
  int last;                // 1: this launch ends the call and counts the step
};

// What every element's step needs, in registers.
struct Rates {
  float rate, root2, gs, eps, b1, c1, b2, c2;
  double lr;
  unsigned key;
  bool scaled;       // there is a grad_scale
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ double power(double b, int t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

// Square root to one unit of the last place (the weight's update needs no more; the
// root that is kept in 8 bits is rounded correctly, so that its codes are fixed).
__device__ __forceinline__ float root_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two e4m3 codes (low byte first) to floats and back; the values are exact, the
// rounding is to nearest even, beyond the range to the largest number, NaN to NaN.
__device__ __forceinline__ void from_e4m3x2(unsigned short c, float& lo, float& hi) {
  unsigned h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
__device__ __forceinline__ unsigned short to_e4m3x2(float lo, float hi) {
  unsigned short c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

// 32 random bits of an element pair.  The multipliers are the first 32 bits of
// the fractional parts of the roots of 2 and 3 (both odd).
__device__ __forceinline__ unsigned mix(unsigned x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Four consecutive elements as they lie in memory: float4 (fp32), uint2 (bf16) or
// unsigned (codes).  kFull: all four are inside the tensor; else those at n and
// beyond read as zero and are not written.
template <typename P>
struct Quad;
template <>
struct Quad<float> {
  float4 q;
  __device__ __forceinline__ void unpack(float (&x)[4]) const {
    x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
  }
  __device__ __forceinline__ void pack(const float (&x)[4]) {
    q = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Quad<__nv_bfloat16> {
  uint2 q;
  __device__ __forceinline__ void unpack(float (&x)[4]) const {
    x[0] = __uint_as_float(q.x << 16), x[1] = __uint_as_float(q.x & 0xffff0000u);
    x[2] = __uint_as_float(q.y << 16), x[3] = __uint_as_float(q.y & 0xffff0000u);
  }
  __device__ __forceinline__ void pack(const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    q = make_uint2(*reinterpret_cast<const unsigned*>(&a), *reinterpret_cast<const unsigned*>(&b));
  }
};
template <>
struct Quad<unsigned char> {
  unsigned q;
};

// Element j of a quad and back, as raw bits.
__device__ __forceinline__ float element(const float4& q, int j) {
  return j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
}
__device__ __forceinline__ void set_element(float4& q, int j, float v) {
  (j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w) = v;
}
__device__ __forceinline__ unsigned short element(const uint2& q, int j) {
  return static_cast<unsigned short>((j < 2 ? q.x : q.y) >> (16 * (j & 1)));
}
__device__ __forceinline__ void set_element(uint2& q, int j, unsigned short v) {
  (j < 2 ? q.x : q.y) |= static_cast<unsigned>(v) << (16 * (j & 1));
}
__device__ __forceinline__ unsigned char element(const unsigned& q, int j) {
  return static_cast<unsigned char>(q >> (8 * j));
}
__device__ __forceinline__ void set_element(unsigned& q, int j, unsigned char v) {
  q |= static_cast<unsigned>(v) << (8 * j);
}

template <bool kFull, typename P>
__device__ __forceinline__ Quad<P> load_quad(const P* p, long long i0, long long n) {
  Quad<P> x;
  if constexpr (kFull) {
    x.q = *reinterpret_cast<const decltype(x.q)*>(p + i0);
  } else {
    x.q = decltype(x.q){};
    using E = decltype(element(x.q, 0));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j < n) set_element(x.q, j, reinterpret_cast<const E*>(p)[i0 + j]);
  }
  return x;
}
template <bool kFull, typename P>
__device__ __forceinline__ void store_quad(P* p, long long i0, long long n, const Quad<P>& x) {
  if constexpr (kFull) {
    *reinterpret_cast<decltype(Quad<P>::q)*>(p + i0) = x.q;
  } else {
    using E = decltype(element(x.q, 0));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j < n) reinterpret_cast<E*>(p)[i0 + j] = element(x.q, j);
  }
}
__device__ __forceinline__ void decode4(unsigned c, float s, float (&x)[4]) {
  from_e4m3x2(static_cast<unsigned short>(c), x[0], x[1]);
  from_e4m3x2(static_cast<unsigned short>(c >> 16), x[2], x[3]);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(x[j], s);
}

// One 256-element block of a tensor, as one lane of a warp holds it: elements
// 4 lane .. 4 lane + 3 of each half.
template <typename P, bool kMaster, bool kEight>
struct Block {
  using W = std::conditional_t<kMaster, float, P>;
  using S = std::conditional_t<kEight, unsigned char, float>;
  Quad<W> w[2];
  Quad<P> g[2];
  Quad<S> m[2], v[2];
  float sm, sv;

  template <bool kFull>
  __device__ __forceinline__ void load(const AdamwEntry& e, long long b) {
    const W* wp = kMaster ? reinterpret_cast<const W*>(e.master) : static_cast<const W*>(e.p);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long i0 = b * kAdamBlock + h * (kAdamBlock / 2) + (threadIdx.x & 31) * 4;
      w[h] = load_quad<kFull>(wp, i0, e.n);
      g[h] = load_quad<kFull>(static_cast<const P*>(e.g), i0, e.n);
      m[h] = load_quad<kFull>(static_cast<const S*>(e.m), i0, e.n);
      v[h] = load_quad<kFull>(static_cast<const S*>(e.v), i0, e.n);
    }
    if constexpr (kEight) {
      sm = e.m_scale[b];
      sv = e.v_scale[b];
    }
  }

  template <bool kFull>
  __device__ __forceinline__ void step(const AdamwEntry& e, long long b, float decay,
                                       const Rates& R) const {
    const int lane = threadIdx.x & 31;
    const long long base = b * kAdamBlock + lane * 4;
    float fm[2][4], fv[2][4];
    float top_m = 0.f, top_r = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long i0 = base + h * (kAdamBlock / 2);
      float fw[4], fg[4];
      w[h].unpack(fw);
      g[h].unpack(fg);
      if constexpr (kEight) {
        decode4(m[h].q, sm, fm[h]);
        decode4(v[h].q, sv, fv[h]);
      } else {
        m[h].unpack(fm[h]);
        v[h].unpack(fv[h]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float& mj = fm[h][j];
        float& vj = fv[h][j];
        if constexpr (kEight) vj = __fmul_rn(vj, vj);
        const float gj = R.scaled ? __fmul_rn(fg[j], R.gs) : fg[j];
        mj = __fadd_rn(__fmul_rn(mj, R.b1), __fmul_rn(gj, R.c1));
        vj = __fadd_rn(__fmul_rn(vj, R.b2), __fmul_rn(__fmul_rn(gj, gj), R.c2));
        const float r = kEight ? __fsqrt_rn(vj) : root_approx(vj);
        fw[j] = fmaf(-R.rate, __fdividef(mj, fmaf(r, R.root2, R.eps)), fw[j] * decay);
        if constexpr (kEight) {
          vj = r;      // the root is what is kept
          top_m = max_nan(top_m, fabsf(mj));
          top_r = max_nan(top_r, r);
        }
      }
      Quad<P> qp;
      qp.pack(fw);
      store_quad<kFull>(static_cast<P*>(e.p), i0, e.n, qp);
      if constexpr (kMaster) {
        Quad<float> qw;
        qw.pack(fw);
        store_quad<kFull>(e.master, i0, e.n, qw);
      }
      if constexpr (!kEight) {
        Quad<float> qm, qv;
        qm.pack(fm[h]);
        qv.pack(fv[h]);
        store_quad<kFull>(static_cast<float*>(e.m), i0, e.n, qm);
        store_quad<kFull>(static_cast<float*>(e.v), i0, e.n, qv);
      }
    }
    if constexpr (kEight) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        top_m = max_nan(top_m, __shfl_xor_sync(0xffffffffu, top_m, o));
        top_r = max_nan(top_r, __shfl_xor_sync(0xffffffffu, top_r, o));
      }
      // a factor of zero turns a block that is too small into zeros
      const bool no_m = top_m < kLeast, no_r = top_r < kLeast;
      const float im = no_m ? 0.f : __fmul_rn(__frcp_rn(top_m), 448.f);
      const float ir = no_r ? 0.f : __fmul_rn(__frcp_rn(top_r), 448.f);
      if (lane == 0) {
        e.m_scale[b] = no_m ? 0.f : __fmul_rn(top_m, 1.f / 448.f);
        e.v_scale[b] = no_r ? 0.f : __fmul_rn(top_r, 1.f / 448.f);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const long long i0 = base + h * (kAdamBlock / 2);
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const unsigned u = mix(static_cast<unsigned>((i0 + j) >> 1) + R.key);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float q = __fmul_rn(fv[h][j + k], ir);
            const unsigned t = (__float_as_uint(q) + ((k ? u >> 16 : u & 0xffffu) << 4) + 8u) &
                               0xfff00000u;
            x[j + k] = q <= 0.f ? 0.f : max_nan(__uint_as_float(t), 0.001953125f);
            fm[h][j + k] = __fmul_rn(fm[h][j + k], im);
          }
        }
        Quad<unsigned char> qm, qv;
        qm.q = to_e4m3x2(fm[h][0], fm[h][1]) |
               static_cast<unsigned>(to_e4m3x2(fm[h][2], fm[h][3])) << 16;
        qv.q = to_e4m3x2(x[0], x[1]) | static_cast<unsigned>(to_e4m3x2(x[2], x[3])) << 16;
        store_quad<kFull>(static_cast<unsigned char*>(e.m), i0, e.n, qm);
        store_quad<kFull>(static_cast<unsigned char*>(e.v), i0, e.n, qv);
      }
    }
  }
};

// The blocks b, b + stride, ... of a tensor by one warp: the next block is read
// before the current one is worked on, so that the loads overlap the arithmetic
// (a warp issues about 75 instructions per element of an 8-bit state; measured on
// 202 M bf16 parameters with masters and 8-bit states: 722 -> 635 us in a run of calls,
// 566 us alone, 5.7 TB/s).
template <typename P, bool kMaster, bool kEight>
__device__ __forceinline__ void step_tensor(const AdamwEntry& e, long long b, long long stride,
                                            const Rates& R) {
  const float decay = static_cast<float>(__dsub_rn(1.0, __dmul_rn(R.lr, e.wd)));
  const long long whole = e.n / kAdamBlock;
  Block<P, kMaster, kEight> cur;
  if (b < whole) cur.template load<true>(e, b);
  while (b < whole) {
    Block<P, kMaster, kEight> next;
    if (b + stride < whole) next.template load<true>(e, b + stride);
    cur.template step<true>(e, b, decay, R);
    cur = next;
    b += stride;
  }
  if (b == whole && b * kAdamBlock < e.n) {   // the short last block
    cur.template load<false>(e, b);
    cur.template step<false>(e, b, decay, R);
  }
}

// All tensors of one kind (type, master, states): one kernel for all kinds needs the
// registers of the largest for every one and spills.
template <typename P, bool kMaster, bool kEight, int kMax>
__global__ void __launch_bounds__(kAdamThreads, 3)
adamw_kernel(const __grid_constant__ AdamwTable<kMax> a) {
  __shared__ float s_rate, s_root2;
  __shared__ double s_lr;
  __shared__ unsigned s_key;
  const int t = min(max(a.step[0], 0), INT_MAX - 1) + 1;
  if (threadIdx.x == 0) {
    const double lr = a.lr * (a.lr_scale ? static_cast<double>(*a.lr_scale) : 1.0);
    s_lr = lr;
    s_rate = static_cast<float>(lr / (1.0 - power(a.beta1, t)));
    s_key = static_cast<unsigned>(t) * 0x3C6EF373u + a.seed * 0xA54FF53Bu;
  } else if (threadIdx.x == 32) {
    s_root2 = static_cast<float>(1.0 / sqrt(1.0 - power(a.beta2, t)));
  }
  Rates R;
  R.gs = a.grad_scale ? *a.grad_scale : 1.f;
  __syncthreads();
  R.rate = s_rate;
  R.root2 = s_root2;
  R.lr = s_lr;
  R.key = s_key;
  R.eps = a.eps;
  R.b1 = a.b1;
  R.c1 = a.c1;
  R.b2 = a.b2;
  R.c2 = a.c2;
  R.scaled = a.grad_scale != nullptr;
  // the launch's chunks (runs of kAdamWarps blocks) go round the CTAs
  const long long stride = static_cast<long long>(gridDim.x) * kAdamWarps;
  for (int k = 0; k < a.count; ++k) {
    const AdamwEntry& e = a.t[k];
    const unsigned ahead = e.first % gridDim.x;
    const unsigned at = blockIdx.x >= ahead ? blockIdx.x - ahead : blockIdx.x + gridDim.x - ahead;
    const long long b = static_cast<long long>(at) * kAdamWarps + (threadIdx.x >> 5);
    if (b * kAdamBlock >= e.n) continue;
    step_tensor<P, kMaster, kEight>(e, b, stride, R);
  }
  // every CTA has read the step before it arrives; the last one counts it
  if (a.last) {
    __syncthreads();
    if (threadIdx.x == 0 &&
        atomicAdd(reinterpret_cast<unsigned*>(a.step + 1), 1u) == gridDim.x - 1) {
      a.step[1] = 0;
      a.step[0] = t;
    }
  }
}

struct Range {
  uintptr_t lo, hi;
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// (bf16 ? 1 : 0) | (master ? 2 : 0) | (8-bit ? 4 : 0)
int kind_of(const swl_adamw_tensor& q) {
  return (q.dtype == SWL_BF16 ? 1 : 0) | (q.master ? 2 : 0) | (q.state_bits == 8 ? 4 : 0);
}

template <int kMax>
cudaError_t launch(int kind, const AdamwTable<kMax>& a, int sms, cudaStream_t stream) {
  const int most = sms * 3;
  const int grid = a.chunks < most ? (a.chunks > 0 ? a.chunks : 1) : most;
  using bf16 = __nv_bfloat16;
  switch (kind) {
    case 0: adamw_kernel<float, false, false, kMax><<<grid, kAdamThreads, 0, stream>>>(a); break;
    case 1: adamw_kernel<bf16, false, false, kMax><<<grid, kAdamThreads, 0, stream>>>(a); break;
    case 3: adamw_kernel<bf16, true, false, kMax><<<grid, kAdamThreads, 0, stream>>>(a); break;
    case 4: adamw_kernel<float, false, true, kMax><<<grid, kAdamThreads, 0, stream>>>(a); break;
    case 5: adamw_kernel<bf16, false, true, kMax><<<grid, kAdamThreads, 0, stream>>>(a); break;
    default: adamw_kernel<bf16, true, true, kMax><<<grid, kAdamThreads, 0, stream>>>(a); break;
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace
}  // namespace swl

using namespace swl;

extern "C" swl_status switch_layer_adamw_step(const swl_adamw_tensor* tensors, int count,
                                              const swl_adamw* cfg, int32_t* step,
                                              const float* grad_scale, const float* lr_scale,
                                              void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !cfg || !step) return SWL_ERR_INVALID_ARG;
  if (!std::isfinite(cfg->lr) || cfg->lr < 0 || !(cfg->beta1 >= 0 && cfg->beta1 < 1) ||
      !(cfg->beta2 >= 0 && cfg->beta2 < 1) || !std::isfinite(cfg->eps) || !(cfg->eps > 0) ||
      static_cast<float>(cfg->eps) <= 0.f)
    return SWL_ERR_INVALID_ARG;
  if (count > (1 << 20)) return SWL_ERR_UNSUPPORTED;
  // what the step writes must not overlap, within a tensor or between two
  const std::unique_ptr<Range[]> ranges(new (std::nothrow) Range[6 * static_cast<size_t>(count) + 1]);
  if (!ranges) return SWL_ERR_UNSUPPORTED;
  Range* const written = ranges.get();
  int nw = 0;
  auto writes = [&](const void* p, unsigned long long bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    written[nw++] = {lo, lo + static_cast<uintptr_t>(bytes)};
  };
  if (reinterpret_cast<uintptr_t>(step) & 7) return SWL_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(grad_scale) & 3 || reinterpret_cast<uintptr_t>(lr_scale) & 3)
    return SWL_ERR_UNSUPPORTED;
  writes(step, 8);
  for (int i = 0; i < count; ++i) {
    const swl_adamw_tensor& q = tensors[i];
    if (q.n < 0 || (q.dtype != SWL_F32 && q.dtype != SWL_BF16) ||
        (q.state_bits != 8 && q.state_bits != 32) || !std::isfinite(q.weight_decay) ||
        q.weight_decay < 0 || (q.master && q.dtype != SWL_BF16))
      return SWL_ERR_INVALID_ARG;
    if (q.n == 0) continue;
    if (q.n > (1ll << 40)) return SWL_ERR_UNSUPPORTED;
    if (!q.param || !q.grad || !q.m || !q.v) return SWL_ERR_INVALID_ARG;
    if ((q.state_bits == 8) != (q.m_scale != nullptr) || (q.state_bits == 8) != (q.v_scale != nullptr))
      return SWL_ERR_INVALID_ARG;
    if (!aligned16(q.param) || !aligned16(q.grad) || !aligned16(q.m) || !aligned16(q.v) ||
        !aligned16(q.master) || (reinterpret_cast<uintptr_t>(q.m_scale) & 3) ||
        (reinterpret_cast<uintptr_t>(q.v_scale) & 3))
      return SWL_ERR_UNSUPPORTED;
    const unsigned long long n = static_cast<unsigned long long>(q.n), sb = q.state_bits / 8;
    const unsigned long long nb = (n + kAdamBlock - 1) / kAdamBlock;
    writes(q.param, n * (q.dtype == SWL_BF16 ? 2 : 4));
    writes(q.m, n * sb);
    writes(q.v, n * sb);
    if (q.m_scale) writes(q.m_scale, nb * 4);
    if (q.v_scale) writes(q.v_scale, nb * 4);
    if (q.master) writes(q.master, n * 4);
  }
  std::sort(written, written + nw, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  for (int i = 1; i < nw; ++i)
    if (written[i].lo < written[i - 1].hi) return SWL_ERR_INVALID_ARG;
  // nor may it write what it reads only
  auto hits = [&](const void* p, unsigned long long bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + bytes;
    const Range* r = std::lower_bound(written, written + nw, lo,
                                      [](const Range& a, uintptr_t v) { return a.hi <= v; });
    return r != written + nw && r->lo < hi;
  };
  for (int i = 0; i < count; ++i)
    if (tensors[i].n > 0 &&
        hits(tensors[i].grad, tensors[i].n * (tensors[i].dtype == SWL_BF16 ? 2ull : 4ull)))
      return SWL_ERR_INVALID_ARG;
  if ((grad_scale && hits(grad_scale, 4)) || (lr_scale && hits(lr_scale, 4)))
    return SWL_ERR_INVALID_ARG;

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SWL_ERR_CUDA;
  // the chunks of all launches fit an int, checked before the first is made
  long long total = 0;
  int last = -1;                       // the last tensor, kind by kind: it ends the call
  for (int i = 0; i < count; ++i) {
    if (tensors[i].n == 0) continue;
    total += tensors[i].n / (kAdamBlock * kChunkBlocks) + 1;
    if (last < 0 || kind_of(tensors[i]) >= kind_of(tensors[last])) last = i;
  }
  if (total > INT_MAX / 4) return SWL_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&](auto& a) -> bool {
    a.step = step;
    a.grad_scale = grad_scale;
    a.lr_scale = lr_scale;
    a.lr = cfg->lr;
    a.beta1 = cfg->beta1;
    a.beta2 = cfg->beta2;
    a.eps = static_cast<float>(cfg->eps);
    a.b1 = static_cast<float>(cfg->beta1);
    a.c1 = static_cast<float>(1.0 - cfg->beta1);
    a.b2 = static_cast<float>(cfg->beta2);
    a.c2 = static_cast<float>(1.0 - cfg->beta2);
    a.seed = cfg->seed;
    constexpr int room = sizeof(a.t) / sizeof(a.t[0]);
    for (int kind = 0; kind < 8; ++kind) {
      a.count = a.chunks = 0;
      for (int i = 0; i < count; ++i) {
        const swl_adamw_tensor& q = tensors[i];
        if (q.n == 0 || kind_of(q) != kind) continue;
        a.t[a.count++] = {q.param, q.grad, q.m, q.v, q.m_scale, q.v_scale, q.master, q.n,
                          q.weight_decay, static_cast<unsigned>(a.chunks)};
        a.chunks += static_cast<int>((q.n + kAdamBlock * kChunkBlocks - 1) /
                                     (kAdamBlock * kChunkBlocks));
        a.last = i == last;
        if (a.count == room || a.last) {
          if (launch(kind, a, sms, st) != cudaSuccess) return false;
          a.count = a.chunks = 0;
        }
      }
      if (a.count > 0 && launch(kind, a, sms, st) != cudaSuccess) return false;
    }
    a.last = 1;
    return last >= 0 || launch(0, a, sms, st) == cudaSuccess;   // nothing but the step
  };
  if (count <= 16) {          // a small table costs less to pass
    AdamwTable<16> a;
    return run(a) ? SWL_OK : SWL_ERR_CUDA;
  }
  AdamwTable<kTableMax> a;
  return run(a) ? SWL_OK : SWL_ERR_CUDA;
}
