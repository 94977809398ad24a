// st_tensor_device.h -- what the kernels on the tensor cores share
// (st_linear.cu, st_block_linear.cu, st_moe.cu): barriers, TMA, tcgen05,
// clusters, outputs at any alignment, tensor maps.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "st_ops_device.h"

namespace stmat {

// One operand of the product.
struct Side {
  const uint8_t *p;
  int64_t pitch;   // bytes between rows
  int64_t span;    // bytes from the first row's start to the last row's end
  int64_t rows;
};
inline Side side_of(const void *ptr, int64_t ld, int64_t rows, int64_t k, int item) {
  return Side{static_cast<const uint8_t *>(ptr), ld * item, ld * item * (rows - 1) + k * item, rows};
}
// Copies the operands that TMA cannot read, rows of row_bytes, to aligned rows
// in the workspace, the weight's first, and points the sides at them.
st_status align_rows(Side *w, Side *x, int64_t row_bytes, void *workspace, void *stream, const char *op);

namespace {

constexpr int kStageK = 128;         // bytes of k per stage: one swizzle row
constexpr int kMaxStages = 12;       // ring slots
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr int kChunk = 32;           // columns an epilogue warp reads at a time

// What becomes of a product's sums.
struct OutArgs {
  int64_t m, n;
  int vec;                           // y and residual rows take the kernel's widest accesses
  st_act act;
  st_dtype y_dtype, bias_dtype;
  const void *bias, *residual;
  void *y;
  int64_t ldr, ldy;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void local_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// One thread of the (converged) warp, chosen so that the compiler knows that
// it runs alone: the tensor core's and TMA's operands then stay in uniform
// registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes;
}
// The polls allowed to a wait for a sum of `blocks` stages: kWaitLimit, which
// is room for one stage, and 256 a stage.  A poll takes 10 ns at the least, a
// stage 0.2 us, and under 1 us where every SM streams from HBM.  (Callers pass
// the whole sum's stages, which are no register of theirs: their own part's
// cost the readout 2834 x 1856 x 704 BF16 3 %.)
__device__ __forceinline__ uint32_t sum_limit(int blocks) {
  const uint64_t polls = kWaitLimit + 256ull * static_cast<uint32_t>(blocks);
  return polls < 0xffffffffu ? static_cast<uint32_t>(polls) : 0xffffffffu;
}
// Bounded: false after `limit` polls.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, uint32_t limit = kWaitLimit) {
  for (uint32_t it = 0; it < limit; ++it) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    if (ok) return true;
  }
  return false;
}
// The same for a whole warp that waits long: one lane polls, and pauses
// between polls, so that the threads that feed the tensor core are not held up.
__device__ __forceinline__ bool bar_wait_warp(uint64_t *bar, uint32_t parity, int lane, uint32_t limit) {
  int ok = 0;
  if (lane == 0) {
    for (uint32_t it = 0; it < limit && !ok; ++it) {
      asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                   : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
      if (!ok) __nanosleep(64);
    }
  }
  ok = __shfl_sync(~0u, ok, 0);
  __syncwarp();
  return ok;
}
__device__ __forceinline__ void tma_load(const CUtensorMap *map, void *dst, uint64_t *bar, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar)) : "memory");
}
// Shared-memory descriptor of a K-major tile in the 128-byte swizzle: rows of
// 128 bytes, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t tile_desc(const void *p) {
  return (static_cast<uint64_t>(smem_addr(p) >> 4) & 0x3fff) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
template <bool kEight>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if constexpr (kEight)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
               : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of this CTA's shared variable in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ void peer_store(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// A position in a ring of `stages` stages: its index, and the parity of its
// barriers' current phase.
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++at == stages) at = 0, phase ^= 1;
  }
};

// Pairs of CTAs.

// Orders what the CTA did before, not its global writes (a release to the
// cluster would wait for y to be written: 2000 cycles a tile).
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A tile of this CTA whose bytes count on a barrier that may be the peer's.
__device__ __forceinline__ void pair_load(const CUtensorMap *map, void *dst, uint32_t bar, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
template <bool kEight>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if constexpr (kEight)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
}
// Arrives on the barrier at this address in both CTAs of the pair whose first
// is `leader` once the MMAs so far are done.
__device__ __forceinline__ void pair_commit(uint64_t *bar, uint32_t leader) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(smem_addr(bar)), "h"(static_cast<uint16_t>(3u << leader)) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&f)[32]) {
  uint32_t v[32];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
                 "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
                 "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
               : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
}
__device__ __forceinline__ void ld32(const void *p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "l"(p) : "memory");
}
__device__ __forceinline__ void st32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}

// Residual and y of one token and kChunk columns, in 32-byte accesses.  A
// 16-bit residual is read (issued) well before it is added.
__device__ __forceinline__ void add16(const uint32_t (&u)[8], bool bf16, float *v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 f;
    if (bf16) f = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    else f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
    v[2 * i] += f.x;
    v[2 * i + 1] += f.y;
  }
}
__device__ __forceinline__ void add_row32(const void *base, int64_t at, float (&v)[kChunk]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ld32(static_cast<const float *>(base) + at + 8 * i, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * i + j] += __uint_as_float(u[j]);
  }
}
__device__ __forceinline__ void put_row(void *base, st_dtype dtype, int64_t at, const float (&v)[kChunk]) {
  uint32_t u[8];
  if (dtype == ST_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[8 * i + j]);
      st32(static_cast<float *>(base) + at + 8 * i, u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      u[j] = dtype == ST_BF16 ? pack_bf16(v[16 * i + 2 * j], v[16 * i + 2 * j + 1]) : pack_f16(v[16 * i + 2 * j], v[16 * i + 2 * j + 1]);
    st32(static_cast<uint16_t *>(base) + at + 16 * i, u);
  }
}

// Rows at any alignment, or a ragged last chunk.  A warp's 32 tokens x kChunk
// columns are turned in shared memory, so that a half-warp reads or writes one
// token's consecutive columns: half h has tokens 16 h + i, lane l of it the
// pair of columns 2 l, 2 l + 1, or, where a row of y starts at an odd place,
// 2 l + 1, 2 l + 2 (and the first column alone), so that a pair is one aligned
// word (5598 x 6526 x 391 BF16 with gelu and residual 145 us column by column,
// 103 so; 109 with gelu's present polynomial).
__device__ __forceinline__ int rows_from(const OutArgs &a, int64_t m) {
  return static_cast<int>(max(int64_t(0), min(int64_t(32), a.m - m)));
}
__device__ __forceinline__ void read_turned(const OutArgs &a, int64_t m0, int64_t n0, int lane, uint32_t (&old)[2][8]) {
  const int half = lane >> 4, l = lane & 15, rows = rows_from(a, m0);
  const int lim = static_cast<int>(min(int64_t(kChunk), a.n - n0));
  const uint16_t *p = static_cast<const uint16_t *>(a.residual) + (m0 + 16 * half) * a.ldr + n0 + 2 * l;
#pragma unroll
  for (int i = 0; i < 16; ++i, p += a.ldr) {
    uint32_t w = 0;
    if (i + 16 * half < rows) {
      if (2 * l + 1 < lim && reinterpret_cast<uintptr_t>(p) % 4 == 0) w = *reinterpret_cast<const uint32_t *>(p);
      else {
        if (2 * l < lim) w = p[0];
        if (2 * l + 1 < lim) w |= static_cast<uint32_t>(p[1]) << 16;
      }
    }
    old[i / 8][i % 8] = w;
  }
}
template <class T>
__device__ __forceinline__ void put_turned(uint32_t (&w)[32][17], const OutArgs &a, int64_t m0, int64_t n0, int lane,
                                           const uint32_t (&old)[2][8], float (&v)[kChunk]) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  const int half = lane >> 4, l = lane & 15, rows = rows_from(a, m0);
  const int lim = static_cast<int>(min(int64_t(kChunk), a.n - n0));
  if (a.residual) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i + 16 * half][l] = old[i / 8][i % 8];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = w[lane][8 * i + j];
      add16(u, kBf16, v + 16 * i);
    }
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 16; ++j) w[lane][j] = kBf16 ? pack_bf16(v[2 * j], v[2 * j + 1]) : pack_f16(v[2 * j], v[2 * j + 1]);
  __syncwarp();
  uint16_t *p = static_cast<uint16_t *>(a.y) + (m0 + 16 * half) * a.ldy + n0;
#pragma unroll
  for (int i = 0; i < 16; ++i, p += a.ldy) {
    if (i + 16 * half >= rows) break;
    const uint32_t *r = w[i + 16 * half];
    const uint32_t lo = r[l];
    if (reinterpret_cast<uintptr_t>(p) % 4 == 0) {
      if (2 * l + 1 < lim) *reinterpret_cast<uint32_t *>(p + 2 * l) = lo;
      else if (2 * l < lim) p[2 * l] = static_cast<uint16_t>(lo);
    } else {
      if (2 * l + 2 < lim) *reinterpret_cast<uint32_t *>(p + 2 * l + 1) = __funnelshift_r(lo, r[l + 1], 16);
      else if (2 * l + 1 < lim) p[2 * l + 1] = static_cast<uint16_t>(lo >> 16);
      if (l == 0) p[0] = static_cast<uint16_t>(lo);
    }
  }
}
// The same for binary32, 16 columns at a time.
__device__ __forceinline__ void put_turned32(uint32_t (&w)[32][17], const OutArgs &a, int64_t m0, int64_t n0, int lane,
                                             const float (&v)[kChunk]) {
  const int half = lane >> 4, rows = rows_from(a, m0);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) w[lane][j] = __float_as_uint(v[16 * h + j]);
    __syncwarp();
    const int64_t col = n0 + 16 * h + (lane & 15);
    if (col >= a.n) continue;
    const float *from = static_cast<const float *>(a.residual) + (m0 + 16 * half) * a.ldr + col;
    float *to = static_cast<float *>(a.y) + (m0 + 16 * half) * a.ldy + col;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + 16 * half >= rows) break;
      to[i * a.ldy] = __uint_as_float(w[i + 16 * half][lane & 15]) + (a.residual ? from[i * a.ldr] : 0.0f);
    }
  }
}

// ------------------------------------------------------------------- host

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline st_status encoder(EncodeFn *out, const char *op) {
  static std::mutex mu;
  static EncodeFn fn = nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || !p)
      return set_error(ST_E_CUDA, "%s: the driver has no cuTensorMapEncodeTiled (%s)", op, cudaGetErrorName(e));
    fn = reinterpret_cast<EncodeFn>(p);
  }
  *out = fn;
  return ST_OK;
}

// Whether TMA can read the matrix: address and row stride multiples of 16
// bytes, the stride under 2^40.
inline bool tma_ok(const Side &s) {
  return reinterpret_cast<uintptr_t>(s.p) % 16 == 0 && (s.rows == 1 || (s.pitch > 0 && s.pitch % 16 == 0 && s.pitch < (int64_t(1) << 40)));
}

// A matrix read in boxes of 128 bytes of k and box_rows rows.
inline st_status encode(CUtensorMap *map, const Side &s, int64_t k, int item, int box_rows, const char *op) {
  EncodeFn fn = nullptr;
  const st_status st = encoder(&fn, op);
  if (st != ST_OK) return st;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(s.rows)};
  const cuuint64_t stride[1] = {s.rows == 1 ? static_cast<cuuint64_t>((k * item + 15) / 16 * 16) : static_cast<cuuint64_t>(s.pitch)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kStageK / item), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  const CUresult r = fn(map, item == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                        const_cast<uint8_t *>(s.p), dims, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(ST_E_CUDA, "%s: tensor map of %lld x %lld refused (%d)", op, (long long)s.rows, (long long)k, static_cast<int>(r));
  return ST_OK;
}

constexpr int kMaxDevices = 256;

// Raises a kernel's limit of dynamic shared memory, once per kernel and device.
template <auto kKernel>
cudaError_t allow_smem(int dev, int bytes) {
  static std::atomic<bool> done[kMaxDevices];
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace
}  // namespace stmat
