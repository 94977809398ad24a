// st_ops_device.h -- conversions, activations and vector accesses shared by
// the operator kernels (st_rowops.cu, st_linear.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "st_ops.h"

namespace stmat {

// max(a, b), NaN if either is one (fmaxf drops a NaN): a row with a NaN gets
// a NaN scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}
// Two E4M3 codes, nearest even, clamped to +-448, NaN kept.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// V consecutive elements as stored, read with one or two aligned accesses.
template <class T, int V>
struct alignas(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Raw {
  T e[V];
};

template <class T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V> &r, float (&v)[V]) {
  if constexpr (V > 1 && std::is_same<T, __nv_bfloat16>::value) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_float(r.e[i]);
  }
}

// f(T{}) for the type of a 16- or 32-bit floating dtype (the branch is the
// same for every thread).
template <class F>
__device__ __forceinline__ void with_type(st_dtype dtype, F &&f) {
  if (dtype == ST_BF16) f(__nv_bfloat16{});
  else if (dtype == ST_F16) f(__half{});
  else f(float{});
}
// V consecutive elements of an array whose dtype is known at run time (the
// branch is the same for every thread).
template <int V>
__device__ __forceinline__ void load_any(const void *base, st_dtype dtype, int64_t at, float (&v)[V]) {
  with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    unpack(*reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(base) + at), v);
  });
}

// V consecutive values rounded to the dtype (F8_E4M3: already divided by the scale).
template <int V>
__device__ __forceinline__ void store_any(void *base, st_dtype dtype, int64_t at, const float (&v)[V]) {
  if constexpr (V == 1) {
    if (dtype == ST_F8_E4M3) static_cast<uint8_t *>(base)[at] = static_cast<uint8_t>(pack_e4m3(v[0], 0.0f));
    else if (dtype == ST_BF16) static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(v[0]);
    else if (dtype == ST_F16) static_cast<__half *>(base)[at] = __float2half_rn(v[0]);
    else static_cast<float *>(base)[at] = v[0];
  } else if (dtype == ST_F8_E4M3) {
    Raw<uint32_t, V / 4> u;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) u.e[i] = pack_e4m3(v[4 * i], v[4 * i + 1]) | pack_e4m3(v[4 * i + 2], v[4 * i + 3]) << 16;
    *reinterpret_cast<Raw<uint32_t, V / 4> *>(static_cast<uint8_t *>(base) + at) = u;
  } else if (dtype == ST_F32) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(static_cast<float *>(base) + at + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    Raw<uint32_t, V / 2> u;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) u.e[i] = dtype == ST_BF16 ? pack_bf16(v[2 * i], v[2 * i + 1]) : pack_f16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<Raw<uint32_t, V / 2> *>(static_cast<uint16_t *>(base) + at) = u;
  }
}

// 2^v and 1 / v from the special-function unit (16 a clock and SM), within 2
// and 1 units of the last place; results below 2^-126 are 0.
__device__ __forceinline__ float fast_exp2(float v) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float fast_rcp(float v) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}

// Activations.  For outputs of 16 and 8 bits they are formed in 5 (silu), 7
// (gelu_tanh) and 17 (gelu) operations a value: with the library's exp, tanh
// and erf and an exact division the gated activation ran at half the memory's
// rate, and a product of 3814 x 6612 x 1723 E4M3 with gelu_tanh 330 us where it
// takes 80 with bias and residual.  With e the exponential's argument they are within
// (2 |e| + 6) 2^-23 of the value, mostly the binary32 rounding of e, and for
// negative v 0 where exp(|e|) is beyond 2^126.
//   silu:      v / (1 + exp(-v)), e = v
//   gelu_tanh: (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), u = sqrt(2 / pi) (v + 0.044715 v^3), e = 2u
//   gelu:      v Phi(v), e = v^2 / 2.  Phi(-|v|) exp(v^2 / 2) is smooth in t =
//              1 / (1 + 0.304 |v|); t times a polynomial of degree 7 in t, fitted
//              to it for the least largest relative error over |v| <= 13.5 (by
//              Lawson's reweighted least squares), is off by at most 8.4e-8 of it.
// For F32 outputs (kF32) the library's exp, a reciprocal refined by a step of
// Newton's iteration, and v^2's rounding error taken into gelu's exponential:
// silu within 4 2^-23 of the value, gelu 7, gelu_tanh 2 |e| + 4.  A negative v
// takes v exp(e) / (1 + exp(e)), whose exponential does not overflow.  (Gated
// 8192 x 14336 F32 249 us with silu, 288 with gelu, 209 without; by an exact
// division and the library's normal distribution 316 and 416.)
constexpr float kLog2e = 1.44269504f;
constexpr float kTanh1 = 1.59576912f, kTanh3 = 0.0713548128f;  // 2 sqrt(2 / pi), that times 0.044715
// 1 / v for v from 1 to 2^24, within a unit of the last place.
__device__ __forceinline__ float near_rcp(float v) {
  const float r = fast_rcp(v);
  return fmaf(r, fmaf(-v, r, 1.0f), r);
}
template <bool kF32>
__device__ __forceinline__ float gelu(float v) {
  // Beyond 16 the exponential is 0, and infinities would meet in the steps.
  const float a = kF32 ? fminf(fabsf(v), 16.0f) : fabsf(v), d = fmaf(a, 0.304f, 1.0f);
  const float t = kF32 ? near_rcp(d) : fast_rcp(d);
  float q = fmaf(t, 0.0368598551f, -0.155304030f);
  q = fmaf(t, q, 0.192196801f);
  q = fmaf(t, q, -0.0431365334f);
  q = fmaf(t, q, 0.123556770f);
  q = fmaf(t, q, 0.102421626f);
  q = fmaf(t, q, 0.122170880f);
  q = fmaf(t, q, 0.121234670f);
  if constexpr (kF32) {
    const float h = a * a, x = expf(-0.5f * h);
    q = q * t * fmaf(x, -0.5f * fmaf(a, a, -h), x);
  } else {
    q = q * t * fast_exp2(v * v * (-0.5f * kLog2e));
  }
  return v * (v < 0.0f ? q : 1.0f - q);
}
// v / (1 + exp(-e)) for an e of v's sign.
__device__ __forceinline__ float gated_exactly(float v, float e) {
  const float x = expf(-fabsf(e));
  return (v < 0.0f ? v * x : v) * near_rcp(1.0f + x);
}
template <bool kF32, st_act A>
__device__ __forceinline__ float activate1(float v) {
  if constexpr (A == ST_ACT_RELU) return v < 0.0f ? 0.0f : v;
  else if constexpr (kF32 && A == ST_ACT_SILU) return gated_exactly(v, v);
  else if constexpr (kF32 && A == ST_ACT_GELU_TANH) return gated_exactly(v, v * fmaf(v * v, kTanh3, kTanh1));
  else if constexpr (A == ST_ACT_SILU) return v * fast_rcp(1.0f + fast_exp2(-kLog2e * v));
  else if constexpr (A == ST_ACT_GELU) return gelu<kF32>(v);
  else if constexpr (A == ST_ACT_GELU_TANH)
    return v * fast_rcp(1.0f + fast_exp2(v * fmaf(v * v, -kTanh3 * kLog2e, -kTanh1 * kLog2e)));
  else return v;
}

template <bool kF32, int N>
__device__ __forceinline__ void activate(float (&v)[N], st_act act) {
  auto each = [&](auto tag) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate1<kF32, decltype(tag)::value>(v[i]);
  };
  switch (act) {
    case ST_ACT_RELU: return each(std::integral_constant<st_act, ST_ACT_RELU>{});
    case ST_ACT_SILU: return each(std::integral_constant<st_act, ST_ACT_SILU>{});
    case ST_ACT_GELU: return each(std::integral_constant<st_act, ST_ACT_GELU>{});
    case ST_ACT_GELU_TANH: return each(std::integral_constant<st_act, ST_ACT_GELU_TANH>{});
    default: return;
  }
}

// Whether a call's activation is one of those that differ for F32 outputs.
inline bool exact_act(st_act act, st_dtype y_dtype) { return y_dtype == ST_F32 && act > ST_ACT_RELU; }

// A kernel launched by launch() may start while the one before it in the
// stream still runs (programmatic dependent launch), so that its start-up
// overlaps that one's end.  It touches no global memory before
// wait_for_previous(), which returns when the previous kernel has ended and
// its writes are visible; let_next_start() lets the next one begin.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), unsigned blocks, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

}  // namespace stmat
