// st_rowops.cu -- row operators for GB300 (sm_103a): the root-mean-square
// norm with the residual's addition, and the gated activation, each with an
// output in 16 or 32 bits or in 8 bits with scales.
//
// Mathematics.  With h = x + r:
//   y = h w rstd,  rstd = 1 / sqrt(sum(h^2) / cols + eps)
// and for 8 bits the scale max|y| / 448.  rstd is one positive number per row
// and rounding is monotone, so max|y| = max|h w| * rstd exactly as computed:
// the row needs one pass and one joint reduction of (sum h^2, max |h w|), and
// the values stay in registers until they are written.  The gated activation
// z = act(g) u needs max|z| alone.
//
// Bound: HBM (norm, BF16 with residual to 8 bits: 7 bytes an element).
#include <string>

#include "st_ops_device.h"

namespace stmat {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kRowsPerBlock = 8;  // rows of one warp each
// A block brings the inputs of the row this far ahead into L2, so that HBM is
// kept busy while the rows on the SMs are reduced and written (8192 x 4096
// norm 37.9 -> 36.2 us, 8192 x 14336 gated activation 101 -> 95.5 us; the same
// within 1 % from 38 to 228 rows, slower from 456 rows of 48 KiB on).
constexpr int kAhead = 128;

// The largest block of a row kernel: its registers hold NV vectors a thread.
constexpr int block_threads(int v, int nv) { return v > 1 && nv >= 4 ? 512 : kMaxThreads; }

struct RowArgs {
  const void *x, *r, *w;  // norm: x, residual, weight; gate: gate, up
  void *h, *y;
  const float *scale;
  float *scales;
  int64_t ldx, ldr, ldh, ldy;
  int64_t rows;
  int cols;
  float eps;
  st_act act;
  st_dtype w_dtype, y_dtype;
};

struct Stat {
  float sum, top;  // sum of squares (norm), largest magnitude
};

__device__ __forceinline__ Stat warp_stat(Stat s) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    s.sum += __shfl_xor_sync(~0u, s.sum, d);
    s.top = max_nan(s.top, __shfl_xor_sync(~0u, s.top, d));
  }
  return s;
}

// The block's joint statistics, in a fixed order.
__device__ __forceinline__ Stat block_stat(Stat s) {
  __shared__ Stat part[kMaxThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  s = warp_stat(s);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  return warp_stat(lane < warps ? part[lane] : Stat{0.0f, 0.0f});
}

// What every value of the row is multiplied by before it is stored: rstd (1
// for the gated activation), then 1 / scale (1 unless 8 bits).  Two factors,
// since their product can leave binary32's range (a zero row: 1 / scale =
// 2^126).
struct Factor {
  float rstd, inv;
};

// The row's factors from its statistics; writes the row's scale.
template <bool kNorm>
__device__ __forceinline__ Factor row_factor(const RowArgs &a, Stat s, int64_t row, bool first) {
  Factor f{1.0f, 1.0f};
  if (kNorm) f.rstd = rsqrtf(s.sum / static_cast<float>(a.cols) + a.eps);
  if (a.y_dtype != ST_F8_E4M3) return f;
  float scale;
  if (a.scales) {
    scale = max_nan(s.top * f.rstd / kE4M3Max, kMinScale);
    if (first) a.scales[row] = scale;
  } else {
    scale = *a.scale;
  }
  f.inv = 1.0f / scale;
  return f;
}

template <bool kNorm>
__device__ __forceinline__ float scaled(float v, Factor f) {
  return (kNorm ? v * f.rstd : v) * f.inv;
}

template <class T>
constexpr st_dtype kDtype = sizeof(T) == 4 ? ST_F32 : std::is_same<T, __half>::value ? ST_F16 : ST_BF16;

// The values before the row's factors (h w, or z) of V elements at column c,
// from the elements as read, adding to the statistics and writing h.
template <class T, int V, bool kNorm, bool kWrite>
__device__ __forceinline__ void row_values(const RowArgs &a, int64_t row, int c, const Raw<T, V> &x, const Raw<T, V> &r,
                                           float (&v)[V], Stat &s) {
  unpack(x, v);
  float o[V];
  if (a.r) unpack(r, o);
  if constexpr (kNorm) {
    if (a.r) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += o[i];
      if (a.h && kWrite) store_any<V>(a.h, kDtype<T>, row * a.ldh + c, v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s.sum = fmaf(v[i], v[i], s.sum);
    if (a.w) {
      load_any<V>(a.w, a.w_dtype, c, o);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= o[i];
    }
  } else {
    activate(v, a.act);
    if (a.r) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= o[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s.top = max_nan(s.top, fabsf(v[i]));
}

template <class T, int V>
__device__ __forceinline__ Raw<T, V> row_read(const void *p, int64_t at) {
  return *reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(p) + at);
}

template <class T>
__device__ __forceinline__ void row_prefetch(const void *p, int64_t at, int cols) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const T *>(p) + at), "r"(cols * static_cast<int>(sizeof(T))) : "memory");
}

// One row in registers: a block (or, kWarpRow, a warp) per row, NV accesses
// of V elements per thread, all of them under way before the first is used.
template <class T, int V, int NV, bool kNorm, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerBlock : block_threads(V, NV)) row_kernel(const RowArgs a) {
  const int64_t row = kWarpRow ? int64_t(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5) : int64_t(blockIdx.x);
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x, nt = kWarpRow ? 32 : blockDim.x;
  wait_for_previous();
  let_next_start();
  if (kWarpRow && row >= a.rows) return;
  if (!kWarpRow && V > 1 && t == 0 && row + kAhead < a.rows) {
    row_prefetch<T>(a.x, (row + kAhead) * a.ldx, a.cols);
    if (a.r) row_prefetch<T>(a.r, (row + kAhead) * a.ldr, a.cols);
  }
  Raw<T, V> x[NV], r[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + t) * V;
    if (c < a.cols) x[i] = row_read<T, V>(a.x, row * a.ldx + c);
  }
  if (a.r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + t) * V;
      if (c < a.cols) r[i] = row_read<T, V>(a.r, row * a.ldr + c);
    }
  }
  float v[NV][V];
  Stat s{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + t) * V;
    if (c < a.cols) row_values<T, V, kNorm, true>(a, row, c, x[i], r[i], v[i], s);
  }
  s = kWarpRow ? warp_stat(s) : block_stat(s);
  const Factor f = row_factor<kNorm>(a, s, row, t == 0);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + t) * V;
    if (c < a.cols) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = scaled<kNorm>(v[i][j], f);
      store_any<V>(a.y, a.y_dtype, row * a.ldy + c, v[i]);
    }
  }
}

// A row too long for registers: the second pass reads the inputs again (each
// thread its own elements, so in-place outputs are read before they are
// written; h is written in the second pass).
template <class T, int V, bool kNorm>
__global__ void __launch_bounds__(kMaxThreads) row_loop_kernel(const RowArgs a) {
  const int64_t row = blockIdx.x;
  wait_for_previous();
  let_next_start();
  Stat s{0.0f, 0.0f}, unused{0.0f, 0.0f};
  Raw<T, V> x, r;
  float v[V];
  for (int64_t c = threadIdx.x * V; c < a.cols; c += kMaxThreads * V) {
    x = row_read<T, V>(a.x, row * a.ldx + c);
    if (a.r) r = row_read<T, V>(a.r, row * a.ldr + c);
    row_values<T, V, kNorm, false>(a, row, static_cast<int>(c), x, r, v, s);
  }
  s = block_stat(s);
  const Factor f = row_factor<kNorm>(a, s, row, threadIdx.x == 0);
  for (int64_t c = threadIdx.x * V; c < a.cols; c += kMaxThreads * V) {
    x = row_read<T, V>(a.x, row * a.ldx + c);
    if (a.r) r = row_read<T, V>(a.r, row * a.ldr + c);
    row_values<T, V, kNorm, true>(a, row, static_cast<int>(c), x, r, v, unused);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = scaled<kNorm>(v[j], f);
    store_any<V>(a.y, a.y_dtype, row * a.ldy + c, v);
  }
}

template <class T, int V, int NV, bool kNorm>
cudaError_t launch_rows(const RowArgs &a, int threads, cudaStream_t st) {
  if (threads == 32)
    return launch(row_kernel<T, V, NV, kNorm, true>, static_cast<unsigned>((a.rows + kRowsPerBlock - 1) / kRowsPerBlock),
                  32 * kRowsPerBlock, 0, 1, st, a);
  return launch(row_kernel<T, V, NV, kNorm, false>, static_cast<unsigned>(a.rows), threads, 0, 1, st, a);
}

// Accesses per thread: as few as blocks of 256 threads allow, so that several
// rows share an SM and one's loads overlap another's reduction; with too few
// rows for that, blocks of 1024, the shortest way through one row.
template <class T, int V, bool kNorm>
cudaError_t launch_typed(const RowArgs &a, cudaStream_t st) {
  const int64_t accesses = a.cols / V;
  const int64_t target = a.rows <= 256 ? kMaxThreads : 256;
  constexpr int kMost = V == 8 ? 4 : 8;
  auto threads = [&](int nv) { return static_cast<int>(((accesses + nv - 1) / nv + 31) / 32 * 32); };
  if (accesses <= target) return launch_rows<T, V, 1, kNorm>(a, threads(1), st);
  if (accesses <= 2 * target) return launch_rows<T, V, 2, kNorm>(a, threads(2), st);
  if (accesses <= 4 * block_threads(V, 4)) return launch_rows<T, V, 4, kNorm>(a, threads(4), st);
  if (accesses <= kMost * block_threads(V, kMost)) return launch_rows<T, V, kMost, kNorm>(a, threads(kMost), st);
  return launch(row_loop_kernel<T, V, kNorm>, static_cast<unsigned>(a.rows), kMaxThreads, 0, 1, st, a);
}

template <bool kNorm>
st_status launch_op(const RowArgs &a, st_dtype x_dtype, bool vec, void *stream, const char *op) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (x_dtype == ST_BF16) e = vec ? launch_typed<__nv_bfloat16, 8, kNorm>(a, st) : launch_typed<__nv_bfloat16, 1, kNorm>(a, st);
  else if (x_dtype == ST_F16) e = vec ? launch_typed<__half, 8, kNorm>(a, st) : launch_typed<__half, 1, kNorm>(a, st);
  else e = vec ? launch_typed<float, 4, kNorm>(a, st) : launch_typed<float, 1, kNorm>(a, st);
  if (e != cudaSuccess)
    return set_error(ST_E_CUDA, "%s launch (%lld rows): %s: %s", op, (long long)a.rows, cudaGetErrorName(e),
                     cudaGetErrorString(e));
  return ST_OK;
}

// Whether the accesses of a row of 16-byte input vectors are aligned in this
// matrix: 16 bytes, or eight (at least) of an 8-bit one.
bool vec_ok(const void *p, int64_t ld, st_dtype dtype) {
  if (!p) return true;
  const uint64_t item = dtype == ST_F8_E4M3 ? 1 : dtype == ST_F32 ? 4 : 2, need = item == 1 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(p) % need == 0 && (static_cast<uint64_t>(ld) * item) % need == 0;
}

}  // namespace

st_status launch_rms_norm(const st_rms_norm_args &p, void *stream) {
  RowArgs a{};
  a.x = p.x; a.r = p.residual; a.w = p.weight; a.h = p.h; a.y = p.y;
  a.ldx = p.ldx; a.ldr = p.ldr; a.ldh = p.ldh; a.ldy = p.ldy;
  a.scale = p.scale; a.scales = p.scales;
  a.rows = p.rows; a.cols = static_cast<int>(p.cols);
  a.eps = p.eps; a.act = ST_ACT_NONE; a.w_dtype = p.w_dtype; a.y_dtype = p.y_dtype;
  const bool vec = p.cols % 8 == 0 && vec_ok(p.x, p.ldx, p.x_dtype) && vec_ok(p.residual, p.ldr, p.x_dtype) &&
                   vec_ok(p.weight, 0, p.w_dtype) && vec_ok(p.h, p.ldh, p.x_dtype) && vec_ok(p.y, p.ldy, p.y_dtype);
  return launch_op<true>(a, p.x_dtype, vec, stream, "st_rms_norm");
}

st_status launch_gated_act(const st_gated_act_args &p, void *stream) {
  RowArgs a{};
  a.x = p.gate; a.r = p.up; a.y = p.y;
  a.ldx = p.ldg; a.ldr = p.ldu; a.ldy = p.ldy;
  a.scale = p.scale; a.scales = p.scales;
  a.rows = p.rows; a.cols = static_cast<int>(p.cols);
  a.act = p.act; a.w_dtype = ST_F32; a.y_dtype = p.y_dtype;
  const bool vec = p.cols % 8 == 0 && vec_ok(p.gate, p.ldg, p.x_dtype) && vec_ok(p.up, p.ldu, p.x_dtype) &&
                   vec_ok(p.y, p.ldy, p.y_dtype);
  return launch_op<false>(a, p.x_dtype, vec, stream, "st_gated_act");
}

}  // namespace stmat
