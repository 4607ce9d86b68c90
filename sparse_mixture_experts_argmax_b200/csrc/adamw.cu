// One AdamW step over many tensors in one launch, the states in 32 or 8 bits.
//
// Per element, with g scaled by *grad_scale, t = steps made + 1 and lr scaled by
// *lr_scale:
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32, every operation rounded on its own (no contraction), so the result is
// a fixed function of the inputs; the bias corrections are taken in fp64.  bf16
// parameters are rounded from w once; with an fp32 master copy w is read from
// and kept there, and the bf16 parameter is only written.
//
// 8-bit states: blocks of 256 consecutive elements share an fp32 scale, the
// largest magnitude over 448 (the largest e4m3 number).  m is held as e4m3
// times the scale, rounded to nearest (its moving average renews a tenth of it
// per step, more than the format's step).  v is held by its root: r = sqrt(v) has
// half the exponent range, so e4m3's 2^-9..448 spans 35 binary orders of v.  The
// root is rounded stochastically to its three mantissa bits with 16 random bits
// per element: with b2 near 1 a step changes r by far less than half a spacing,
// and rounding to nearest would never let v move.  The bits come from a
// counter (element pair, step, seed) through two multiply-xorshift rounds, so a
// step can be repeated exactly.  A non-zero r keeps at least the smallest code, so
// no element's denominator falls to eps alone; a block whose largest magnitude is
// under 2^-100 is held as zeros.  The step itself uses the unrounded m and v.
//
// Bound: HBM.  Per element 12 bytes of fp32 weight and gradient (bf16: 6, with a
// master 12) and 16 bytes of fp32 states or 4.06 of 8-bit ones.  One warp takes one
// 256-element block at a time, four elements per lane twice, so that every type is
// read in whole vectors (fp32 16 bytes, bf16 8, codes 4) and a block's two maxima
// are five shuffles each.  The tensor table travels in the kernel's parameters
// (nothing to copy or allocate, so a captured call replays as it is) and the grid is
// persistent, so the corrections are computed once per CTA.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <memory>
#include <new>

#include "kernels.h"
#include "switch_layer.h"

namespace swl {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamBlock = SWL_ADAMW_BLOCK;         // elements that share a scale
constexpr int kChunkBlocks = 2 * kAdamWarps;        // blocks per work item of a CTA
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
  int kind;          // (bf16 ? 1 : 0) | (master ? 2 : 0) | (8-bit ? 4 : 0)
  int first;         // chunks of earlier tensors of this launch
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

struct Rates {
  float rate, root2, gs;
  double lr;
  unsigned key;
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

// Four consecutive elements from i0 on, those at n and beyond read as zero and
// not written (kFull: there are none).
template <bool kFull>
__device__ __forceinline__ void load4(const float* p, long long i0, long long n, float (&x)[4]) {
  if (kFull) {
    const float4 q = *reinterpret_cast<const float4*>(p + i0);
    x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
  } else {
    for (int j = 0; j < 4; ++j) x[j] = i0 + j < n ? p[i0 + j] : 0.f;
  }
}
template <bool kFull>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, long long i0, long long n,
                                      float (&x)[4]) {
  if (kFull) {
    const uint2 q = *reinterpret_cast<const uint2*>(p + i0);
    x[0] = __uint_as_float(q.x << 16), x[1] = __uint_as_float(q.x & 0xffff0000u);
    x[2] = __uint_as_float(q.y << 16), x[3] = __uint_as_float(q.y & 0xffff0000u);
  } else {
    for (int j = 0; j < 4; ++j) x[j] = i0 + j < n ? __bfloat162float(p[i0 + j]) : 0.f;
  }
}
template <bool kFull>
__device__ __forceinline__ void store4(float* p, long long i0, long long n, const float (&x)[4]) {
  if (kFull) {
    *reinterpret_cast<float4*>(p + i0) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    for (int j = 0; j < 4; ++j)
      if (i0 + j < n) p[i0 + j] = x[j];
  }
}
template <bool kFull>
__device__ __forceinline__ void store4(__nv_bfloat16* p, long long i0, long long n,
                                       const float (&x)[4]) {
  if (kFull) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p + i0) = make_uint2(*reinterpret_cast<const unsigned*>(&a),
                                                   *reinterpret_cast<const unsigned*>(&b));
  } else {
    for (int j = 0; j < 4; ++j)
      if (i0 + j < n) p[i0 + j] = __float2bfloat16_rn(x[j]);
  }
}
template <bool kFull>
__device__ __forceinline__ unsigned load_codes(const unsigned char* p, long long i0, long long n) {
  if (kFull) return *reinterpret_cast<const unsigned*>(p + i0);
  unsigned c = 0;
  for (int j = 0; j < 4; ++j)
    if (i0 + j < n) c |= static_cast<unsigned>(p[i0 + j]) << (8 * j);
  return c;
}
template <bool kFull>
__device__ __forceinline__ void store_codes(unsigned char* p, long long i0, long long n,
                                            unsigned c) {
  if (kFull) {
    *reinterpret_cast<unsigned*>(p + i0) = c;
  } else {
    for (int j = 0; j < 4; ++j)
      if (i0 + j < n) p[i0 + j] = static_cast<unsigned char>(c >> (8 * j));
  }
}
__device__ __forceinline__ void decode4(unsigned c, float s, float (&x)[4]) {
  from_e4m3x2(static_cast<unsigned short>(c), x[0], x[1]);
  from_e4m3x2(static_cast<unsigned short>(c >> 16), x[2], x[3]);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(x[j], s);
}

// Elements [256 b, 256 b + 256) of a tensor, by one warp.
template <typename P, bool kMaster, bool kEight, bool kFull, typename A>
__device__ __forceinline__ void step_block(const AdamwEntry& e, long long b, float decay,
                                           const Rates& R, const A& a) {
  const int lane = threadIdx.x & 31;
  const long long base = b * kAdamBlock + lane * 4;
  float w[2][4], g[2][4], m[2][4], v[2][4];
  unsigned cm[2], cv[2];
  float sm = 0.f, sv = 0.f;
  const float* wsrc = kMaster ? e.master : static_cast<const float*>(e.p);
#pragma unroll
  for (int h = 0; h < 2; ++h) {      // every read in flight before the first use
    const long long i0 = base + h * (kAdamBlock / 2);
    if constexpr (kMaster || sizeof(P) == 4) load4<kFull>(wsrc, i0, e.n, w[h]);
    else load4<kFull>(static_cast<const P*>(e.p), i0, e.n, w[h]);
    load4<kFull>(static_cast<const P*>(e.g), i0, e.n, g[h]);
    if constexpr (kEight) {
      cm[h] = load_codes<kFull>(static_cast<const unsigned char*>(e.m), i0, e.n);
      cv[h] = load_codes<kFull>(static_cast<const unsigned char*>(e.v), i0, e.n);
    } else {
      load4<kFull>(static_cast<const float*>(e.m), i0, e.n, m[h]);
      load4<kFull>(static_cast<const float*>(e.v), i0, e.n, v[h]);
    }
  }
  if constexpr (kEight) {
    sm = e.m_scale[b];
    sv = e.v_scale[b];
  }
  float top_m = 0.f, top_r = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (kEight) {
      decode4(cm[h], sm, m[h]);
      decode4(cv[h], sv, v[h]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kEight) v[h][j] = __fmul_rn(v[h][j], v[h][j]);
      const float gj = a.grad_scale ? __fmul_rn(g[h][j], R.gs) : g[h][j];
      m[h][j] = __fadd_rn(__fmul_rn(m[h][j], a.b1), __fmul_rn(gj, a.c1));
      v[h][j] = __fadd_rn(__fmul_rn(v[h][j], a.b2), __fmul_rn(__fmul_rn(gj, gj), a.c2));
      const float r = __fsqrt_rn(v[h][j]);
      const float den = __fadd_rn(__fmul_rn(r, R.root2), a.eps);
      w[h][j] = __fsub_rn(__fmul_rn(w[h][j], decay), __fmul_rn(__fdiv_rn(m[h][j], den), R.rate));
      if constexpr (kEight) {
        v[h][j] = r;      // the root is what is kept
        top_m = max_nan(top_m, fabsf(m[h][j]));
        top_r = max_nan(top_r, r);
      }
    }
    const long long i0 = base + h * (kAdamBlock / 2);
    store4<kFull>(static_cast<P*>(e.p), i0, e.n, w[h]);
    if constexpr (kMaster) store4<kFull>(e.master, i0, e.n, w[h]);
    if constexpr (!kEight) {
      store4<kFull>(static_cast<float*>(e.m), i0, e.n, m[h]);
      store4<kFull>(static_cast<float*>(e.v), i0, e.n, v[h]);
    }
  }
  if constexpr (kEight) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top_m = max_nan(top_m, __shfl_xor_sync(0xffffffffu, top_m, o));
      top_r = max_nan(top_r, __shfl_xor_sync(0xffffffffu, top_r, o));
    }
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
          const float r = v[h][j + k];
          unsigned q = __float_as_uint(__fmul_rn(r, ir));
          q = (q + ((k ? u >> 16 : u & 0xffffu) << 4) + 8u) & 0xfff00000u;
          x[j + k] = (no_r || r <= 0.f) ? 0.f : max_nan(__uint_as_float(q), 0.001953125f);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) m[h][j + k] = no_m ? 0.f : __fmul_rn(m[h][j + k], im);
      }
      store_codes<kFull>(static_cast<unsigned char*>(e.m), i0, e.n,
                         to_e4m3x2(m[h][0], m[h][1]) |
                             static_cast<unsigned>(to_e4m3x2(m[h][2], m[h][3])) << 16);
      store_codes<kFull>(static_cast<unsigned char*>(e.v), i0, e.n,
                         to_e4m3x2(x[0], x[1]) |
                             static_cast<unsigned>(to_e4m3x2(x[2], x[3])) << 16);
    }
  }
}

template <typename P, bool kMaster, bool kEight, typename A>
__device__ __forceinline__ void step_chunk(const AdamwEntry& e, int chunk, const Rates& R,
                                           const A& a) {
  const float decay = static_cast<float>(__dsub_rn(1.0, __dmul_rn(R.lr, e.wd)));
  const long long nb = (e.n + kAdamBlock - 1) / kAdamBlock;
  for (int k = 0; k < kChunkBlocks / kAdamWarps; ++k) {
    const long long b = static_cast<long long>(chunk) * kChunkBlocks + k * kAdamWarps +
                        (threadIdx.x >> 5);
    if (b >= nb) break;
    if ((b + 1) * kAdamBlock <= e.n) step_block<P, kMaster, kEight, true>(e, b, decay, R, a);
    else step_block<P, kMaster, kEight, false>(e, b, decay, R, a);
  }
}

template <int kMax>
__global__ void __launch_bounds__(kAdamThreads, 3)
adamw_kernel(const __grid_constant__ AdamwTable<kMax> a) {
  __shared__ float s_rate, s_root2;
  __shared__ double s_lr;
  __shared__ unsigned s_key;
  const int t = max(a.step[0], 0) + 1;
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
  int k = 0;
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    while (k + 1 < a.count && a.t[k + 1].first <= c) ++k;
    const AdamwEntry& e = a.t[k];
    const int at = c - e.first;
    switch (e.kind) {
      case 0: step_chunk<float, false, false>(e, at, R, a); break;
      case 1: step_chunk<__nv_bfloat16, false, false>(e, at, R, a); break;
      case 3: step_chunk<__nv_bfloat16, true, false>(e, at, R, a); break;
      case 4: step_chunk<float, false, true>(e, at, R, a); break;
      case 5: step_chunk<__nv_bfloat16, false, true>(e, at, R, a); break;
      case 7: step_chunk<__nv_bfloat16, true, true>(e, at, R, a); break;
    }
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

template <int kMax>
cudaError_t launch(const AdamwTable<kMax>& a, int sms, cudaStream_t stream) {
  const int most = sms * 3;
  const int grid = a.chunks < most ? (a.chunks > 0 ? a.chunks : 1) : most;
  adamw_kernel<kMax><<<grid, kAdamThreads, 0, stream>>>(a);
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
  auto fill = [&](auto& a, int from, int to) {
    long long chunks = 0;
    a.count = 0;
    for (int i = from; i < to; ++i) {
      const swl_adamw_tensor& q = tensors[i];
      if (q.n == 0) continue;
      AdamwEntry& e = a.t[a.count++];
      e = {q.param, q.grad, q.m, q.v, q.m_scale, q.v_scale, q.master, q.n, q.weight_decay,
           (q.dtype == SWL_BF16 ? 1 : 0) | (q.master ? 2 : 0) | (q.state_bits == 8 ? 4 : 0),
           static_cast<int>(chunks)};
      chunks += (q.n + kAdamBlock * kChunkBlocks - 1) / (kAdamBlock * kChunkBlocks);
    }
    a.chunks = static_cast<int>(chunks);
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
    a.last = to == count;
  };
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the chunks of all launches fit an int, checked before the first is made
  long long total = 0;
  for (int i = 0; i < count; ++i) total += tensors[i].n / (kAdamBlock * kChunkBlocks) + 1;
  if (total > INT_MAX / 4) return SWL_ERR_UNSUPPORTED;
  if (count <= 16) {          // a small table costs less to pass
    AdamwTable<16> a;
    fill(a, 0, count);
    return launch(a, sms, st) == cudaSuccess ? SWL_OK : SWL_ERR_CUDA;
  }
  AdamwTable<kTableMax> a;
  for (int from = 0; from < count; from += kTableMax) {
    fill(a, from, std::min(count, from + kTableMax));
    if (launch(a, sms, st) != cudaSuccess) return SWL_ERR_CUDA;
  }
  return SWL_OK;
}
