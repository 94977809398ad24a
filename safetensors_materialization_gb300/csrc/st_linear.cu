// st_linear.cu -- the matrix product with a checkpoint's weight, its scales,
// bias, activation and residual, for GB300 (sm_103a).
#include "st_ops_device.h"

namespace stmat {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

__device__ __forceinline__ float element(const void *p, st_dtype dtype, int64_t at) {
  switch (dtype) {
    case ST_BF16: return to_float(static_cast<const __nv_bfloat16 *>(p)[at]);
    case ST_F16: return to_float(static_cast<const __half *>(p)[at]);
    case ST_F8_E4M3: return static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(p)[at]);
    case ST_F8_E5M2: return static_cast<float>(static_cast<const __nv_fp8_e5m2 *>(p)[at]);
    default: return static_cast<const float *>(p)[at];
  }
}

// One 64 x 64 tile of y per block, 4 x 4 of it per thread, binary32 FMAs.
__global__ void __launch_bounds__(kThreads) linear_simple(const st_linear_args a) {
  __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
  const int64_t m0 = int64_t(blockIdx.y) * kTile, n0 = int64_t(blockIdx.x) * kTile;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < a.k; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      const int r = i / kStep, c = i % kStep;
      const bool kin = k0 + c < a.k;
      xs[c][r] = kin && m0 + r < a.m ? element(a.x, a.x_dtype, (m0 + r) * a.ldx + k0 + c) : 0.0f;
      ws[c][r] = kin && n0 + r < a.n ? element(a.w, a.w_dtype, (n0 + r) * a.ldw + k0 + c) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kStep; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[c][tm + 16 * i], ws[c][tn + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
      if (m >= a.m || n >= a.n) continue;
      float v = acc[i][j];
      if (a.x_scale) v *= a.x_scale[a.x_scale_count == 1 ? 0 : m];
      if (a.w_scale) v *= a.w_scale[a.w_scale_count == 1 ? 0 : n];
      if (a.bias) v += element(a.bias, a.bias_dtype, n);
      v = activate(v, a.act);
      if (a.residual) v += element(a.residual, a.y_dtype, m * a.ldr + n);
      const float out[1] = {v};
      store_any<1>(a.y, a.y_dtype, m * a.ldy + n, out);
    }
}

}  // namespace

st_status launch_linear(const st_linear_args &a, void *stream) {
  const dim3 grid(static_cast<unsigned>((a.n + kTile - 1) / kTile), static_cast<unsigned>((a.m + kTile - 1) / kTile));
  linear_simple<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return set_error(ST_E_CUDA, "st_linear launch (%lld x %lld x %lld): %s: %s", (long long)a.m, (long long)a.n,
                     (long long)a.k, cudaGetErrorName(e), cudaGetErrorString(e));
  return ST_OK;
}

}  // namespace stmat
