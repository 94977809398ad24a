// st_rows_device.h -- what the row kernels share (st_rowops.cu,
// st_blockrows.cu): statistics of a row, accesses, places of rows.
#pragma once

#include "st_ops_device.h"

namespace stmat {
namespace {

constexpr int kMaxThreads = 1024;
// A block brings the inputs of the row this far ahead into L2, so that HBM is
// kept busy while the rows on the SMs are reduced and written (8192 x 4096
// norm 37.9 -> 36.2 us, 8192 x 14336 gated activation 101 -> 95.5 us; the same
// within 1 % from 38 to 228 rows, slower from 456 rows of 48 KiB on).
constexpr int kAhead = 128;

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

// A thread's squares that are added in one chain.  A chain in binary32 is off
// by up to a unit of 2^-24 an addition, all the same way where the row's values
// are alike (7e-4 of the norm at 2^27 columns), so that long rows' chains end
// after so many, and are added in two words.  (Chains as an inner loop of their
// own: a test in every step of one loop took 4-10 % longer.)
constexpr int kChain = 64;

template <class T>
constexpr st_dtype kDtype = sizeof(T) == 4 ? ST_F32 : std::is_same<T, __half>::value ? ST_F16 : ST_BF16;

template <class T, int V>
__device__ __forceinline__ Raw<T, V> row_read(const void *p, int64_t at) {
  return *reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(p) + at);
}

template <class T>
__device__ __forceinline__ void row_prefetch(const void *p, int64_t at, int cols) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const T *>(p) + at), "r"(cols * static_cast<int>(sizeof(T))) : "memory");
}

// Where rows start, in elements modulo an access of V.  Contiguous rows of an
// odd length start at the same places in every matrix (5977 x 2407 BF16 norm
// to 8 bits 15.9 us; element by element 30.9).
struct Place {
  int64_t at, step;
  bool operator==(const Place &o) const { return at == o.at && step == o.step; }
  bool aligned() const { return at == 0 && step == 0; }
};
inline Place place(const void *p, int64_t ld, st_dtype dtype, int v) {
  return {static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) / st_dtype_size(dtype) % v), ld % v};
}

}  // namespace
}  // namespace stmat
