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
// Roundings: h is rounded to x's type where it is kept, but y is formed from
// the binary32 h, so that each output is rounded once.
//
// Bound: HBM.  Read + written, of the 6.74 TB/s a copy reaches: norm of 8192 x
// 4096 BF16 with residual to 8 bits (7 bytes an element) 36.2 us, 6.5 TB/s;
// of 4096 x 12288 to BF16 60.4 us, 6.7 TB/s; gated activation of 8192 x 14336
// BF16 to 8 bits 93.5 us, 6.3 TB/s.
#include <string>

#include "st_rows_device.h"

namespace stmat {
namespace {

constexpr int kRowsPerBlock = 8;  // rows of one warp each
// The operators: the norm, the gated activation, and that with an F32 output
// (exact_act).
enum Op { kNormOp, kActOp, kActF32Op };

// The largest block of a row kernel: its registers hold NV vectors a thread.
constexpr int block_threads(int nv) { return nv >= 4 ? 512 : kMaxThreads; }

// Blocks an SM has room for (0: as the compiler likes).  The exact activations
// otherwise take registers that leave a block alone on an SM (8192 x 14336
// silu from BF16 to F32 244 us, 163 with two; F32 gelu 303, 289 with one asked for).
constexpr int min_blocks(Op op, int v, int nv, bool warp_row) { return op != kActF32Op || warp_row ? 0 : v == 8 && nv == 4 ? 2 : 1; }

struct RowArgs {
  const void *x, *r, *w;  // norm: x, residual, weight; gate: gate, up
  void *h, *y;
  const float *scale;
  float *scales;
  int64_t ldx, ldr, ldh, ldy;
  int64_t rows;
  int cols;
  bool r_same, h_same, y_same;  // skewed rows: the matrix starts where x does, modulo V
  float eps;
  st_act act;
  st_dtype w_dtype, y_dtype;
};

// What every value of the row is multiplied by before it is stored: rstd (1
// for the gated activation), then 1 / scale (1 unless 8 bits).  Two factors,
// since their product can leave binary32's range (a zero row: 1 / scale =
// 2^126).  A given scale below binary32's normal range, whose reciprocal may
// be infinite, has 2^24 of it in the first.
struct Factor {
  float rstd, inv;
};

// The row's factors from its statistics; writes the row's scale.
template <Op kOp>
__device__ __forceinline__ Factor row_factor(const RowArgs &a, Stat s, int64_t row, bool first) {
  Factor f{1.0f, 1.0f};
  if (kOp == kNormOp) f.rstd = rsqrtf(s.sum / static_cast<float>(a.cols) + a.eps);
  if (a.y_dtype != ST_F8_E4M3) return f;
  float scale;
  if (a.scales) {
    scale = max_nan(s.top * f.rstd / kE4M3Max, kMinScale);
    if (first) a.scales[row] = scale;
  } else {
    scale = *a.scale;
    if (fabsf(scale) < kMinScale) f.rstd *= 0x1p24f, scale *= 0x1p24f;
  }
  f.inv = 1.0f / scale;
  return f;
}

// (The gated activation's first factor, seldom other than 1, is in the values.)
template <Op kOp>
__device__ __forceinline__ float scaled(float v, Factor f) {
  return (kOp == kNormOp ? v * f.rstd : v) * f.inv;
}

// Writes the elements of V values from column c on that the row has.
template <int V>
__device__ __forceinline__ void store_part(void *base, st_dtype dtype, int64_t at, int c, int cols, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float one[1] = {v[i]};
    if (c + i >= 0 && c + i < cols) store_any<1>(base, dtype, at + i, one);
  }
}

// The values before the row's factors (h w, or z) of V elements at column c,
// from the elements as read, adding to the statistics and writing h.  W: the
// weight's type; whole: the row has all of the elements.
template <class T, class W, int V, bool kSkew, Op kOp, bool kWrite>
__device__ __forceinline__ void row_values(const RowArgs &a, int64_t row, int c, bool whole, const Raw<T, V> &x,
                                           const Raw<T, V> &r, float (&v)[V], Stat &s) {
  unpack(x, v);
  float o[V];
  if (a.r) unpack(r, o);
  if constexpr (kOp == kNormOp) {
    if (a.r) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += o[i];
      if (a.h && kWrite) {
        if (!kSkew || (whole && a.h_same)) store_any<V>(a.h, kDtype<T>, row * a.ldh + c, v);
        else store_part<V>(a.h, kDtype<T>, row * a.ldh + c, c, a.cols, v);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s.sum = fmaf(v[i], v[i], s.sum);
    if (a.w) {
      const W *w = static_cast<const W *>(a.w) + c;
      if constexpr (kSkew) {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = whole || (c + i >= 0 && c + i < a.cols) ? to_float(w[i]) : 0.0f;
      } else {
        unpack(*reinterpret_cast<const Raw<W, V> *>(w), o);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= o[i];
    }
  } else {
    activate<kOp == kActF32Op>(v, a.act);
    if (a.r) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= o[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s.top = max_nan(s.top, fabsf(v[i]));
}

// V elements of which the row has those at columns 0 .. cols - 1; zeros else.
template <class T, int V>
__device__ __forceinline__ Raw<T, V> row_part(const void *p, int64_t at, int c, int cols) {
  Raw<T, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r.e[i] = T(0.0f);
    if (c + i >= 0 && c + i < cols) r.e[i] = static_cast<const T *>(p)[at + i];
  }
  return r;
}

// One row in registers: a block (or, kWarpRow, a warp) per row, NV accesses
// of V elements per thread, all of them under way before the first is used.
// kSkew: rows start anywhere; the accesses are aligned ones around the row of
// x, whose first and last may hold fewer of its elements, and of the other
// matrices where they start at the same place modulo V, else single elements.
template <class T, int V, int NV, bool kSkew, Op kOp, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerBlock : block_threads(NV), min_blocks(kOp, V, NV, kWarpRow)) row_kernel(const RowArgs a) {
  const int64_t row = kWarpRow ? int64_t(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5) : int64_t(blockIdx.x);
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x, nt = kWarpRow ? 32 : blockDim.x;
  wait_for_previous();
  let_next_start();
  if (kWarpRow && row >= a.rows) return;
  if (!kWarpRow && !kSkew && t == 0 && row + kAhead < a.rows) {
    row_prefetch<T>(a.x, (row + kAhead) * a.ldx, a.cols);
    if (a.r) row_prefetch<T>(a.r, (row + kAhead) * a.ldr, a.cols);
  }
  const int skip = kSkew ? static_cast<int>((reinterpret_cast<uintptr_t>(a.x) / sizeof(T) + row * a.ldx) & (V - 1)) : 0;
  auto column = [&](int i) { return (i * nt + t) * V - skip; };
  auto whole = [&](int c) { return !kSkew || (c >= 0 && c + V <= a.cols); };
  Raw<T, V> x[NV], r[NV];
  auto read = [&](Raw<T, V>(&to)[NV], const void *p, int64_t ld, bool same) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = column(i);
      if (c < a.cols && whole(c) && (!kSkew || same)) to[i] = row_read<T, V>(p, row * ld + c);
    }
    if constexpr (kSkew) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = column(i);
        if (c < a.cols && !(whole(c) && same)) to[i] = row_part<T, V>(p, row * ld + c, c, a.cols);
      }
    }
  };
  read(x, a.x, a.ldx, true);
  if (a.r) read(r, a.r, a.ldr, a.r_same);
  float v[NV][V];
  Stat s{0.0f, 0.0f};
  with_type(kOp == kNormOp ? a.w_dtype : kDtype<T>, [&](auto zero) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = column(i);
      if (c < a.cols) row_values<T, decltype(zero), V, kSkew, kOp, true>(a, row, c, whole(c), x[i], r[i], v[i], s);
    }
  });
  s = kWarpRow ? warp_stat(s) : block_stat(s);
  const Factor f = row_factor<kOp>(a, s, row, t == 0);
  if (kOp != kNormOp && f.rstd != 1.0f) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] *= f.rstd;
  }
  auto write = [&](st_dtype dtype) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = column(i);
      if (c < a.cols) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = scaled<kOp>(v[i][j], f);
        if (whole(c) && (!kSkew || a.y_same)) store_any<V>(a.y, dtype, row * a.ldy + c, v[i]);
        else store_part<V>(a.y, dtype, row * a.ldy + c, c, a.cols, v[i]);
      }
    }
  };
  if (a.y_dtype == ST_F8_E4M3) write(ST_F8_E4M3);
  else if (a.y_dtype == ST_BF16) write(ST_BF16);
  else if (a.y_dtype == ST_F16) write(ST_F16);
  else write(ST_F32);
}

// A row too long for registers: the second pass reads the inputs again (each
// thread its own elements, so in-place outputs are read before they are
// written; h is written in the second pass).
template <class T, int V, Op kOp>
__global__ void __launch_bounds__(kMaxThreads) row_loop_kernel(const RowArgs a) {
  const int64_t row = blockIdx.x;
  wait_for_previous();
  let_next_start();
  // (As the one loop over the row was unrolled, within 4 %: 4 x 2^22 BF16 583 ->
  // 598 us; by 4 in binary32 too 256 x 100000 with a residual 91 -> 107.)
  constexpr int kChainUnroll = V == 4 ? 2 : 4;
  Stat s{0.0f, 0.0f}, unused{0.0f, 0.0f};
  with_type(kOp == kNormOp ? a.w_dtype : kDtype<T>, [&](auto zero) {
    using W = decltype(zero);
    Raw<T, V> x, r;
    float v[V];
    auto add = [&](int64_t c) {
      x = row_read<T, V>(a.x, row * a.ldx + c);
      if (a.r) r = row_read<T, V>(a.r, row * a.ldr + c);
      row_values<T, W, V, false, kOp, false>(a, row, static_cast<int>(c), true, x, r, v, s);
    };
    if constexpr (kOp == kNormOp) {
      Two sum;
      for (int64_t c = threadIdx.x * V; c < a.cols;) {
        const int64_t end = min(int64_t(a.cols), c + kChain * kMaxThreads);
        s.sum = 0.0f;
#pragma unroll kChainUnroll
        for (; c < end; c += kMaxThreads * V) add(c);
        sum.add(s.sum);
      }
      s.sum = sum.value();
    } else {
      for (int64_t c = threadIdx.x * V; c < a.cols; c += kMaxThreads * V) add(c);
    }
    s = block_stat(s);
    const Factor f = row_factor<kOp>(a, s, row, threadIdx.x == 0);
    for (int64_t c = threadIdx.x * V; c < a.cols; c += kMaxThreads * V) {
      x = row_read<T, V>(a.x, row * a.ldx + c);
      if (a.r) r = row_read<T, V>(a.r, row * a.ldr + c);
      row_values<T, W, V, false, kOp, true>(a, row, static_cast<int>(c), true, x, r, v, unused);
      if (kOp != kNormOp && f.rstd != 1.0f) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= f.rstd;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = scaled<kOp>(v[j], f);
      store_any<V>(a.y, a.y_dtype, row * a.ldy + c, v);
    }
  });
}

// The scales of rows without columns, whose largest magnitude is 0.
__global__ void __launch_bounds__(kMaxThreads) empty_rows_kernel(float *scales, int64_t rows) {
  wait_for_previous();
  let_next_start();
  const int64_t row = int64_t(blockIdx.x) * kMaxThreads + threadIdx.x;
  if (row < rows) scales[row] = kMinScale;
}

// threads 0: a warp per row.
template <class T, int V, int NV, bool kSkew, Op kOp>
cudaError_t launch_rows(const RowArgs &a, int threads, cudaStream_t st) {
  if (threads)
    return launch(row_kernel<T, V, NV, kSkew, kOp, false>, static_cast<unsigned>(a.rows), threads, 0, 1, st, a);
  if constexpr (NV <= 4)
    return launch(row_kernel<T, V, NV, kSkew, kOp, true>, static_cast<unsigned>((a.rows + kRowsPerBlock - 1) / kRowsPerBlock),
                  32 * kRowsPerBlock, 0, 1, st, a);
  return cudaErrorInvalidValue;
}

// Accesses per thread: as few as blocks of 256 threads allow, so that several
// rows share an SM and one's loads overlap another's reduction; with too few
// rows for that, blocks of 1024, the shortest way through one row.  A warp
// takes a short row alone (16384 x 333 F16 norm with residual to 8 bits 16.5
// us; in blocks of two warps 19.4).
template <class T, int V, bool kSkew, Op kOp>
cudaError_t launch_typed(const RowArgs &a, cudaStream_t st) {
  const int64_t accesses = kSkew ? (a.cols + 2 * V - 2) / V : a.cols / V;
  const int64_t target = a.rows <= 256 ? kMaxThreads : 256;
  constexpr int kMost = V == 8 ? 4 : 8;
  auto threads = [&](int nv) { return static_cast<int>(((accesses + nv - 1) / nv + 31) / 32 * 32); };
  if (accesses <= 32) return launch_rows<T, V, 1, kSkew, kOp>(a, 0, st);
  if (accesses <= 64 && a.rows > 256) return launch_rows<T, V, 2, kSkew, kOp>(a, 0, st);
  if (accesses <= 128 && a.rows > 256) return launch_rows<T, V, 4, kSkew, kOp>(a, 0, st);
  if (accesses <= target) return launch_rows<T, V, 1, kSkew, kOp>(a, threads(1), st);
  if (accesses <= 2 * target) return launch_rows<T, V, 2, kSkew, kOp>(a, threads(2), st);
  if (accesses <= 4 * block_threads(4)) return launch_rows<T, V, 4, kSkew, kOp>(a, threads(4), st);
  if (accesses <= kMost * block_threads(kMost)) return launch_rows<T, V, kMost, kSkew, kOp>(a, threads(kMost), st);
  return launch(row_loop_kernel<T, kSkew ? 1 : V, kOp>, static_cast<unsigned>(a.rows), kMaxThreads, 0, 1, st, a);
}

template <class T, Op kOp>
cudaError_t launch_layout(const RowArgs &a, bool aligned, cudaStream_t st) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  return aligned ? launch_typed<T, V, false, kOp>(a, st) : launch_typed<T, V, true, kOp>(a, st);
}

template <Op kOp>
st_status launch_op(RowArgs &a, st_dtype x_dtype, void *stream, const char *op) {
  const int v = x_dtype == ST_F32 ? 4 : 8;
  const Place x = place(a.x, a.ldx, x_dtype, v), y = place(a.y, a.ldy, a.y_dtype, v);
  const Place r = a.r ? place(a.r, a.ldr, x_dtype, v) : x, h = a.h ? place(a.h, a.ldh, x_dtype, v) : x;
  a.r_same = r == x, a.h_same = h == x, a.y_same = y == x;
  const bool aligned = a.cols % v == 0 && x.aligned() && a.r_same && a.h_same && a.y_same &&
                       place(a.w, 0, a.w_dtype, v).aligned();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = x_dtype == ST_BF16  ? launch_layout<__nv_bfloat16, kOp>(a, aligned, st)
                        : x_dtype == ST_F16 ? launch_layout<__half, kOp>(a, aligned, st)
                                            : launch_layout<float, kOp>(a, aligned, st);
  if (e != cudaSuccess)
    return set_error(ST_E_CUDA, "%s launch (%lld rows): %s: %s", op, (long long)a.rows, cudaGetErrorName(e),
                     cudaGetErrorString(e));
  return ST_OK;
}

}  // namespace

st_status launch_empty_rows(float *scales, int64_t rows, void *stream, const char *op) {
  const cudaError_t e = launch(empty_rows_kernel, static_cast<unsigned>((rows + kMaxThreads - 1) / kMaxThreads), kMaxThreads, 0, 1,
                               static_cast<cudaStream_t>(stream), scales, rows);
  if (e != cudaSuccess)
    return set_error(ST_E_CUDA, "%s launch (%lld empty rows): %s: %s", op, (long long)rows, cudaGetErrorName(e), cudaGetErrorString(e));
  return ST_OK;
}

st_status launch_rms_norm(const st_rms_norm_args &p, void *stream) {
  RowArgs a{};
  a.x = p.x; a.r = p.residual; a.w = p.weight; a.h = p.h; a.y = p.y;
  a.ldx = p.ldx; a.ldr = p.ldr; a.ldh = p.ldh; a.ldy = p.ldy;
  a.scale = p.scale; a.scales = p.scales;
  a.rows = p.rows; a.cols = static_cast<int>(p.cols);
  a.eps = p.eps; a.act = ST_ACT_NONE; a.w_dtype = p.weight ? p.w_dtype : p.x_dtype; a.y_dtype = p.y_dtype;
  return launch_op<kNormOp>(a, p.x_dtype, stream, "st_rms_norm");
}

st_status launch_gated_act(const st_gated_act_args &p, void *stream) {
  RowArgs a{};
  a.x = p.gate; a.r = p.up; a.y = p.y;
  a.ldx = p.ldg; a.ldr = p.ldu; a.ldy = p.ldy;
  a.scale = p.scale; a.scales = p.scales;
  a.rows = p.rows; a.cols = static_cast<int>(p.cols);
  a.act = p.act; a.w_dtype = p.x_dtype; a.y_dtype = p.y_dtype;
  return exact_act(p.act, p.y_dtype) ? launch_op<kActF32Op>(a, p.x_dtype, stream, "st_gated_act")
                                     : launch_op<kActOp>(a, p.x_dtype, stream, "st_gated_act");
}

}  // namespace stmat
