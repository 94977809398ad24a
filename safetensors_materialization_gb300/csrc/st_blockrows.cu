// st_blockrows.cu -- the row operators with an 8-bit output that has a scale
// for every 128 columns of a row (GB300, sm_103a): what the product with a
// block-scaled weight takes.
//
// Mathematics.  With v the row operator's values (st_rowops.cu) and block b the
// columns 128 b .. 128 b + 127 of a row:
//   scale[b] = max(max over b of |v| / 448, 2^-126),  code = e4m3(v / scale[b]).
// A block is 16 (16-bit inputs) or 32 (binary32) neighbouring threads' vectors,
// so its largest magnitude is a reduction or two of a warp.  The norm's rstd is
// one positive number per row, known after the row's reduction: max|v| = max|h w|
// rstd as computed, and the row stays in registers between the two.  The gated
// activation has no reduction over the row: its rows are cut into pieces.
//
// Bound: HBM (7 bytes an element for a 16-bit norm with residual and h, 5 for a
// gated activation, and a scale's 4 bytes every 128).  A copy's rate is 6.7 TB/s:
// norm 8192 x 4096 BF16 38.3 us (6.2 TB/s), gated 8192 x 14336 with silu 92.8
// (6.4); a norm of one row is 1.9 us of latency.  Pieces instead of whole rows
// took the gated activation from 108 to 101 us, the rest cheaper scales.  Rows
// off 16-byte boundaries are bound by the instructions that shift them: gated
// 8192 x 1111 20.4 us (6.8 by its bytes), norm 16384 x 1111 47 (19).  Norms of
// more than 16384 columns read their row twice, an element a lane: 4096 x 20000
// with a residual 252 us (86).
#include "st_rows_device.h"

namespace stmat {
namespace {

constexpr int kBlock = 128;      // columns of a scale
constexpr int kWarps = 8;        // rows of one warp each, in a block
constexpr int kPieceThreads = 256;

enum Op { kNormOp, kActOp };

struct BlockRowArgs {
  const void *x, *r, *w;  // norm: x, residual, weight; gate: gate, up
  void *h;
  uint8_t *y;
  float *scales;
  int64_t ldx, ldr, ldh, ldy, blocks;
  int64_t rows;
  int cols, pieces;       // pieces of a row (gated activation)
  float eps;
  st_act act;
  st_dtype w_dtype;
};

// V elements from column c on of the row that starts at p, which may start at
// any element: two aligned accesses, shifted, where the row has neighbours to
// both sides (`inside`: up to 8 elements before and 16 behind it belong to the
// matrix), else single elements.  Zeros behind the row's end.
template <class T, int V>
__device__ __forceinline__ Raw<T, V> any_read(const T *p, int c, int cols, bool inside) {
  Raw<T, V> out;
  if (sizeof(T) == 2 && inside) {
    const uint32_t q = (reinterpret_cast<uintptr_t>(p) / 2) & 7;  // c is a multiple of 8
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (c < cols) {
      lo = *reinterpret_cast<const uint4 *>(p + c - q);
      if (q) hi = *reinterpret_cast<const uint4 *>(p + c - q + 8);
    }
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}, sh = 16 * (q & 1);
    uint32_t a[6], b[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) a[i] = q & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) b[i] = q & 2 ? a[i + 1] : a[i];
    uint32_t *u = reinterpret_cast<uint32_t *>(&out);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) u[i] = __funnelshift_r(b[i], b[i + 1], sh);
    if (c + V > cols) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i >= cols) out.e[i] = T(0.0f);
    }
    return out;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) out.e[i] = c + i < cols ? p[c + i] : T(0.0f);
  return out;
}

// The n lowest bytes of `bytes` (fewer than 8) to any address, by the largest
// aligned stores.
__device__ __forceinline__ void put_bytes(uint8_t *p, uint64_t bytes, int n) {
  auto put = [&](auto zero) {
    using U = decltype(zero);
    *reinterpret_cast<U *>(p) = static_cast<U>(bytes);
    p += sizeof(U), bytes >>= 8 * sizeof(U), n -= sizeof(U);
  };
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if ((at & 1) && n >= 1) put(uint8_t{});
  if ((reinterpret_cast<uintptr_t>(p) & 2) && n >= 2) put(uint16_t{});
  if (n >= 4) put(uint32_t{});
  if (n >= 2) put(uint16_t{});
  if (n >= 1) put(uint8_t{});
}

// Eight codes of every lane, from its column c on, in a row that starts at any
// byte: a lane writes the aligned word that its first codes lie in, with the
// last codes of the lane before.  The whole warp calls it, with consecutive
// columns.
__device__ __forceinline__ void put_codes8(uint8_t *row, int c, int cols, uint32_t lo, uint32_t hi, int lane) {
  const int q = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 7), left = cols - c;  // c is a multiple of 8
  const uint32_t lo_before = __shfl_up_sync(~0u, lo, 1), hi_before = __shfl_up_sync(~0u, hi, 1);
  // The word's bytes are those of the lane before's and this one's codes from
  // byte 8 - q on.
  const bool far = q > 4;
  const uint32_t a = far ? lo_before : hi_before, b = far ? hi_before : lo, e = far ? lo : hi, sh = 8 * ((8 - q) & 3);
  const uint32_t w0 = q ? __funnelshift_r(a, b, sh) : lo, w1 = q ? __funnelshift_r(b, e, sh) : hi;
  // The first byte that is this lane's to write, and how many they are.
  const int skip = lane > 0 ? 0 : q, n = min(8, left + q) - skip;
  uint8_t *const to = row + c - q;
  if (n == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(w0, w1);
  else if (n > 0) put_bytes(to + skip, (w0 | static_cast<uint64_t>(w1) << 32) >> (8 * skip), n);
  if (lane == 31 && q && left > 8 - q) put_bytes(to + 8, (lo | static_cast<uint64_t>(hi) << 32) >> (8 * (8 - q)), min(q, left - (8 - q)));
}

// V values of h from column c on, likewise: words of two 16-bit values, shifted
// by one where the row starts at an odd element.
template <class T, int V>
__device__ __forceinline__ void put_any(T *row, int c, int cols, const float (&v)[V], int lane) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < cols) row[c + i] = v[i];
  } else {
    uint32_t u[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      u[i] = kDtype<T> == ST_BF16 ? pack_bf16(v[2 * i], v[2 * i + 1]) : pack_f16(v[2 * i], v[2 * i + 1]);
    const uint32_t before = __shfl_up_sync(~0u, u[V / 2 - 1], 1);
    uint16_t *const p = reinterpret_cast<uint16_t *>(row + c);
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (at % 16 == 0 && c + V <= cols) {
      *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else if (at % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (c + 2 * i + 1 < cols) *reinterpret_cast<uint32_t *>(p + 2 * i) = u[i];
        else if (c + 2 * i < cols) p[2 * i] = static_cast<uint16_t>(u[i]);
      }
    } else {
      // Elements 2 i - 1 and 2 i.
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const uint32_t w = __funnelshift_r(i ? u[i - 1] : before, u[i], 16);
        const bool first = (i > 0 || lane > 0) && c + 2 * i - 1 < cols, second = c + 2 * i < cols;
        if (first && second) *reinterpret_cast<uint32_t *>(p + 2 * i - 1) = w;
        else if (first) p[2 * i - 1] = static_cast<uint16_t>(w);
        else if (second) p[2 * i] = static_cast<uint16_t>(w >> 16);
      }
      if (lane == 31 && c + V - 1 < cols) p[V - 1] = static_cast<uint16_t>(u[V / 2 - 1] >> 16);
    }
  }
}

// A block's scale from its largest magnitude, and the scale's inverse.  Both
// divisions in a few instructions, which every thread of the block takes: a
// quotient by the rounded 1 / 448 and a reciprocal, each with one step that
// takes its remainder in.  Both are then correctly rounded (compared with the
// division for every largest magnitude from 0 to infinity).
__device__ __forceinline__ float block_scale(float top, float *inv) {
  constexpr float kInv = 1.0f / kE4M3Max;
  const float q = top * kInv, exact = fmaf(fmaf(-kE4M3Max, q, top), kInv, q);
  // (An infinite q has no remainder.)
  const float s = max_nan(isinf(q) ? q : exact, kMinScale), r = fast_rcp(s);
  *inv = isinf(s) ? 0.0f : fmaf(r, fmaf(-s, r, 1.0f), r);
  return s;
}

// The largest of a block's magnitudes, in all of its threads: of numbers that
// are not negative the bits are in order, a NaN's above all.  (Two reductions of whole warps, of each half's
// block, for 16 bits; four shuffles took 1-4 % longer, five in binary32 5-10 %:
// 8192 x 4096 F32 norm 47.5 -> 42.5 us.)
template <int V>
__device__ __forceinline__ float block_top(float top, int lane) {
  const uint32_t u = __float_as_uint(top);
  if constexpr (kBlock / V == 32) return __uint_as_float(__reduce_max_sync(~0u, u));
  const bool low = lane < 16;
  const uint32_t a = __reduce_max_sync(~0u, low ? u : 0), b = __reduce_max_sync(~0u, low ? 0 : u);
  return __uint_as_float(low ? a : b);
}

// One row (kWarpRow: of a warp) in registers, NV accesses of V elements a
// thread; the gated activation's block has a piece of a row.  kAny: rows start
// anywhere, or end inside an access.
template <class T, int V, int NV, bool kAny, Op kOp, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kWarps : kOp == kActOp ? kPieceThreads : NV >= 4 ? 512 : kMaxThreads)
block_row_kernel(const BlockRowArgs a) {
  const bool piece = kOp == kActOp && !kWarpRow;
  const int64_t row = kWarpRow ? int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5) : piece ? blockIdx.x / a.pieces : blockIdx.x;
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x, nt = kWarpRow ? 32 : blockDim.x, lane = threadIdx.x & 31;
  const int first = piece ? static_cast<int>(blockIdx.x % a.pieces) * nt * V * NV : 0;
  wait_for_previous();
  let_next_start();
  if (kWarpRow && row >= a.rows) return;
  if (!kWarpRow && !kAny && t == 0 && row + kAhead < a.rows && first < a.cols) {
    const int n = min(a.cols - first, piece ? nt * V * NV : a.cols);
    row_prefetch<T>(a.x, (row + kAhead) * a.ldx + first, n);
    if (a.r) row_prefetch<T>(a.r, (row + kAhead) * a.ldr + first, n);
  }
  auto column = [&](int i) { return first + (i * nt + t) * V; };
  // Columns of the warp lie before the row's end or behind it: its lanes take
  // the same way.
  auto beyond = [&](int i) { return column(i) - lane * V >= a.cols; };
  const T *const px = static_cast<const T *>(a.x) + row * a.ldx, *const pr = static_cast<const T *>(a.r) + row * a.ldr;
  Raw<T, V> x[NV], r[NV];
  auto inside = [&](int64_t ld) { return row * ld >= 8 && (a.rows - 1 - row) * ld >= 16; };
  const bool x_inside = kAny && inside(a.ldx), r_inside = kAny && inside(a.ldr);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = column(i);
    if (beyond(i)) continue;
    if constexpr (kAny) {
      x[i] = any_read<T, V>(px, c, a.cols, x_inside);
      if (a.r) r[i] = any_read<T, V>(pr, c, a.cols, r_inside);
    } else if (c < a.cols) {
      x[i] = row_read<T, V>(px, c);
      if (a.r) r[i] = row_read<T, V>(pr, c);
    }
  }
  float v[NV][V], top[NV];
  Stat s{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = column(i);
    top[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) v[i][j] = 0.0f;
    if (kAny ? beyond(i) : c >= a.cols) continue;
    float o[V];
    unpack(x[i], v[i]);
    if (a.r) unpack(r[i], o);
    if constexpr (kOp == kNormOp) {
      if (a.r) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += o[j];
        if (a.h) {
          T *const ph = static_cast<T *>(a.h) + row * a.ldh;
          if constexpr (kAny) put_any<T, V>(ph, c, a.cols, v[i], lane);
          else store_any<V>(ph, kDtype<T>, c, v[i]);
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) s.sum = fmaf(v[i][j], v[i][j], s.sum);
      if (a.w) {
        with_type(a.w_dtype, [&](auto zero) {
          using W = decltype(zero);
          const W *w = static_cast<const W *>(a.w) + c;
          if (!kAny || (c + V <= a.cols && reinterpret_cast<uintptr_t>(w) % alignof(Raw<W, V>) == 0)) {
            unpack(*reinterpret_cast<const Raw<W, V> *>(w), o);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = c + j < a.cols ? to_float(w[j]) : 0.0f;
          }
        });
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] *= o[j];
      }
    } else {
      activate<false>(v[i], a.act);
      if (a.r) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] *= o[j];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) top[i] = max_nan(top[i], fabsf(v[i][j]));
  }
  float rstd = 1.0f;
  if constexpr (kOp == kNormOp) {
    s = kWarpRow ? warp_stat(s) : block_stat(s);
    rstd = rsqrtf(s.sum / static_cast<float>(a.cols) + a.eps);
  }
  uint8_t *const py = a.y + row * a.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = column(i);
    if (beyond(i)) continue;
    top[i] = block_top<V>(top[i], lane);
    float inv;
    const float scale = block_scale(top[i] * rstd, &inv);
    if (lane % (kBlock / V) == 0 && c < a.cols) a.scales[row * a.blocks + c / kBlock] = scale;
    uint32_t u[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      float2 lo = make_float2(v[i][4 * j], v[i][4 * j + 1]), hi = make_float2(v[i][4 * j + 2], v[i][4 * j + 3]);
      if constexpr (kOp == kNormOp) lo = __fmul2_rn(lo, make_float2(rstd, rstd)), hi = __fmul2_rn(hi, make_float2(rstd, rstd));
      lo = __fmul2_rn(lo, make_float2(inv, inv)), hi = __fmul2_rn(hi, make_float2(inv, inv));
      u[j] = pack_e4m3(lo.x, lo.y) | pack_e4m3(hi.x, hi.y) << 16;
    }
    if constexpr (V == 8) {
      if constexpr (kAny) put_codes8(py, c, a.cols, u[0], u[1], lane);
      else if (c < a.cols) *reinterpret_cast<uint2 *>(py + c) = make_uint2(u[0], u[1]);
    } else if (c < a.cols) {
      if (!kAny || (c + V <= a.cols && reinterpret_cast<uintptr_t>(py + c) % V == 0)) *reinterpret_cast<uint32_t *>(py + c) = u[0];
      else
        for (int j = 0; j < V && c + j < a.cols; ++j) py[c + j] = static_cast<uint8_t>(u[0] >> (8 * j));
    }
  }
}

// A norm's row too long for registers: a warp has a run of 32 columns of four
// elements, one block of a binary32 or 16-bit row, and the second pass reads
// the inputs again (each thread its own elements, so that an h in place of an
// input is written after its last use).  Reads of 16 bytes a lane, with the
// scales in groups of 16 lanes, were slower here.  The squares are added in
// chains of kChain (4096 x 20000 BF16 169 -> 161 us by the first pass's 32-bit
// columns, 252 with a residual; 4 x 2^22 1091).
template <class T>
__global__ void __launch_bounds__(kMaxThreads) block_row_loop_kernel(const BlockRowArgs a) {
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31;
  wait_for_previous();
  let_next_start();
  const T *const px = static_cast<const T *>(a.x) + row * a.ldx, *const pr = static_cast<const T *>(a.r) + row * a.ldr;
  T *const ph = static_cast<T *>(a.h) + row * a.ldh;
  uint8_t *const py = a.y + row * a.ldy;
  auto value = [&](auto c) {
    return c < a.cols ? to_float(px[c]) + (a.r ? to_float(pr[c]) : 0.0f) : 0.0f;
  };
  constexpr int kPass = kMaxThreads / 32 * kBlock;
  Stat s{0.0f, 0.0f};
  Two sum;
  for (int c0 = threadIdx.x / 32 * kBlock; c0 < a.cols;) {
    const int end = min(a.cols, c0 + kChain / 4 * kPass);
    s.sum = 0.0f;
#pragma unroll 2
    for (; c0 < end; c0 += kPass) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = value(c0 + 32 * j + lane);
        s.sum = fmaf(v, v, s.sum);
      }
    }
    sum.add(s.sum);
  }
  s.sum = sum.value();
  s = block_stat(s);
  const float rstd = rsqrtf(s.sum / static_cast<float>(a.cols) + a.eps);
  for (int64_t c0 = threadIdx.x / 32 * kBlock; c0 < a.cols; c0 += kMaxThreads / 32 * kBlock) {
    float v[4], top = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + 32 * j + lane;
      v[j] = value(c);
      if (c >= a.cols) continue;
      const float h[1] = {v[j]};
      if (a.h && a.r) store_any<1>(ph, kDtype<T>, c, h);
      float w[1] = {1.0f};
      if (a.w) load_any<1>(a.w, a.w_dtype, c, w);
      v[j] *= w[0];
      top = max_nan(top, fabsf(v[j]));
    }
    top = block_top<4>(top, lane);
    float inv;
    const float scale = block_scale(top * rstd, &inv);
    if (lane == 0) a.scales[row * a.blocks + c0 / kBlock] = scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + 32 * j + lane;
      if (c < a.cols) py[c] = static_cast<uint8_t>(pack_e4m3(v[j] * rstd * inv, 0.0f));
    }
  }
}

// Threads and accesses of a row: as for st_rowops.cu's kernels, a warp for a
// short row, else blocks of 256 threads so that several rows share an SM, or,
// with few rows, the shortest way through one.  Many rows of 16 bits without a
// residual are bound by instructions: half of the threads, with twice the
// elements, spare some (16384 x 1536 BF16 25.1 -> 21.9 us, 13308 x 2752 34.7 ->
// 31.5; with a residual 8192 x 4096 38.4 -> 39.0, F32 6095 x 1896 27.2 -> 28.7, and
// 300 x 4096 3.3 -> 4.1, so not there).
template <class T, int V, bool kAny>
cudaError_t launch_norm(const BlockRowArgs &a, cudaStream_t st) {
  const int64_t accesses = (int64_t(a.cols) + V - 1) / V;
  const unsigned rows = static_cast<unsigned>(a.rows), groups = static_cast<unsigned>((a.rows + kWarps - 1) / kWarps);
  auto threads = [&](int nv) { return static_cast<unsigned>(((accesses + nv - 1) / nv + 31) / 32 * 32); };
  const int64_t target = a.rows <= 256 ? kMaxThreads : a.rows <= 2048 || kAny || V == 4 || a.r ? 256 : 128;
  if (accesses <= 32) return launch(block_row_kernel<T, V, 1, kAny, kNormOp, true>, groups, 32 * kWarps, 0, 1, st, a);
  if (accesses <= 64 && a.rows > 256) return launch(block_row_kernel<T, V, 2, kAny, kNormOp, true>, groups, 32 * kWarps, 0, 1, st, a);
  if (accesses <= 128 && a.rows > 256) return launch(block_row_kernel<T, V, 4, kAny, kNormOp, true>, groups, 32 * kWarps, 0, 1, st, a);
  if (accesses <= target) return launch(block_row_kernel<T, V, 1, kAny, kNormOp, false>, rows, threads(1), 0, 1, st, a);
  if (accesses <= 2 * target) return launch(block_row_kernel<T, V, 2, kAny, kNormOp, false>, rows, threads(2), 0, 1, st, a);
  if (accesses <= 4 * 512) return launch(block_row_kernel<T, V, 4, kAny, kNormOp, false>, rows, threads(4), 0, 1, st, a);
  if constexpr (V == 4) {
    if (accesses <= 8 * 512) return launch(block_row_kernel<T, V, 8, kAny, kNormOp, false>, rows, threads(8), 0, 1, st, a);
  }
  return launch(block_row_loop_kernel<T>, rows, kMaxThreads, 0, 1, st, a);
}

template <class T, int V, int NV, bool kAny>
cudaError_t launch_pieces(BlockRowArgs a, int64_t accesses, cudaStream_t st) {
  const int64_t pieces = (accesses + kPieceThreads * NV - 1) / (kPieceThreads * NV);
  // The pieces' threads, as even as whole warps allow.
  const unsigned nt = static_cast<unsigned>(((accesses + pieces * NV - 1) / (pieces * NV) + 31) / 32 * 32);
  if (a.rows * pieces > 0x7fffffff) return cudaErrorInvalidConfiguration;
  a.pieces = static_cast<int>(pieces);
  return launch(block_row_kernel<T, V, NV, kAny, kActOp, false>, dim3(static_cast<unsigned>(a.rows * pieces)), nt, 0, 1, st, a);
}

// Pieces of 256 threads with one access a thread of each matrix, or two where
// there are more than 32 such blocks an SM (8192 x 14336 F32 without up 133 ->
// 119 us, BF16 83.3 -> 82.9, gated 93.1 -> 92.8; 608 x 14336 9.4 -> 10.3, 1216 x
// 2048 3.7 -> 4.4).  16-bit rows off 16-byte boundaries always have one: the
// instructions that shift them take longer in pairs (8192 x 1111 F16 20.4, 25.6;
// 60000 x 601 BF16 83, 114; F32 8192 x 2405 38.4, 35.7).
template <class T, int V, bool kAny>
cudaError_t launch_act(const BlockRowArgs &a, int sms, cudaStream_t st) {
  const int64_t accesses = (int64_t(a.cols) + V - 1) / V;
  const unsigned groups = static_cast<unsigned>((a.rows + kWarps - 1) / kWarps);
  if (accesses <= 32) return launch(block_row_kernel<T, V, 1, kAny, kActOp, true>, groups, 32 * kWarps, 0, 1, st, a);
  if (accesses <= 64) return launch(block_row_kernel<T, V, 2, kAny, kActOp, true>, groups, 32 * kWarps, 0, 1, st, a);
  if constexpr (!kAny || V == 4) {
    if (a.rows * accesses > int64_t(sms) * 32 * kPieceThreads) return launch_pieces<T, V, 2, kAny>(a, accesses, st);
  }
  return launch_pieces<T, V, 1, kAny>(a, accesses, st);
}

template <Op kOp>
st_status launch_blocks(const BlockRowArgs &a, st_dtype x_dtype, int sms, void *stream, const char *op) {
  const int v = x_dtype == ST_F32 ? 4 : 8;
  const bool aligned = a.cols % v == 0 && place(a.x, a.ldx, x_dtype, v).aligned() && place(a.y, a.ldy, ST_F8_E4M3, v).aligned() &&
                       (!a.r || place(a.r, a.ldr, x_dtype, v).aligned()) && (!a.h || place(a.h, a.ldh, x_dtype, v).aligned()) &&
                       (!a.w || place(a.w, 0, a.w_dtype, v).aligned());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&](auto zero, auto any) {
    using T = decltype(zero);
    constexpr int V = sizeof(T) == 4 ? 4 : 8;
    if constexpr (kOp == kNormOp) return launch_norm<T, V, decltype(any)::value>(a, st);
    else return launch_act<T, V, decltype(any)::value>(a, sms, st);
  };
  auto typed = [&](auto zero) { return aligned ? run(zero, std::false_type{}) : run(zero, std::true_type{}); };
  const cudaError_t e = x_dtype == ST_BF16 ? typed(__nv_bfloat16{}) : x_dtype == ST_F16 ? typed(__half{}) : typed(float{});
  if (e != cudaSuccess)
    return set_error(ST_E_CUDA, "%s launch (%lld rows): %s: %s", op, (long long)a.rows, cudaGetErrorName(e), cudaGetErrorString(e));
  return ST_OK;
}

}  // namespace

st_status launch_rms_norm_blocks(const st_rms_norm_args &p, void *stream) {
  BlockRowArgs a{};
  a.x = p.x; a.r = p.residual; a.w = p.weight; a.h = p.h;
  a.y = static_cast<uint8_t *>(p.y);
  a.scales = p.scales;
  a.ldx = p.ldx; a.ldr = p.ldr; a.ldh = p.ldh; a.ldy = p.ldy; a.blocks = (p.cols + kBlock - 1) / kBlock;
  a.rows = p.rows; a.cols = static_cast<int>(p.cols);
  a.eps = p.eps; a.act = ST_ACT_NONE; a.w_dtype = p.weight ? p.w_dtype : p.x_dtype;
  return launch_blocks<kNormOp>(a, p.x_dtype, 0, stream, "st_rms_norm_blocks");
}

st_status launch_gated_act_blocks(const st_gated_act_args &p, void *stream) {
  BlockRowArgs a{};
  a.x = p.gate; a.r = p.up;
  a.y = static_cast<uint8_t *>(p.y);
  a.scales = p.scales;
  a.ldx = p.ldg; a.ldr = p.ldu; a.ldy = p.ldy; a.blocks = (p.cols + kBlock - 1) / kBlock;
  a.rows = p.rows; a.cols = static_cast<int>(p.cols);
  a.act = p.act; a.w_dtype = p.x_dtype;
  int dev = 0, sms = 0;
  uint32_t *err = nullptr;
  const st_status s = product_device(&dev, &sms, &err);
  return s == ST_OK ? launch_blocks<kActOp>(a, p.x_dtype, sms, stream, "st_gated_act_blocks") : s;
}

}  // namespace stmat
