// st_linear.cu -- the matrix product with a checkpoint's weight, its scales,
// bias, activation and residual, for GB300 (sm_103a).
//
//   y[i, j] = act(x_scale[i] w_scale[j] sum_l x[i, l] w[j, l] + bias[j]) + residual[i, j]
//
// split_kernel: the weight's rows are the MMA's rows (128 a tile), the tokens
// its columns, so that one token costs no more than the 16 columns of the
// narrowest MMA, and the weight streams through shared memory at the rate of
// HBM.  The sum's range is split over the CTAs of a cluster; each puts its
// binary32 partial sums into the shared memory of the CTA that joins them, in
// rank order (no workspace, no atomics, the same bits on every run).  Pushing
// them takes one cluster barrier where reading them from their makers took
// two (1 x 1024 x 4096 E4M3: 4.7 -> 3.3 us).  Bound by HBM: 1 x 28672 x 8192
// E4M3 36.5 us (6.4 TB/s), 1 x 14336 x 4096 11.8 us (5.0 TB/s, 3 us of it the
// chain from the last bytes to y).
//
// dense_kernel: many tokens.  A pair of CTAs (two SMs) computes 256 tokens x up
// to 256 weight rows with one MMA: each holds 128 tokens and half of the
// weight rows, so a stage's 32 KB per SM feed twice the products of a lone
// CTA's.  The pairs stay resident and take tiles in turn; a tile's sums are
// read out of one half of TMEM while the next tile's are formed in the other.
// Few tiles with long sums are shared by the pairs of a cluster, which join
// their sums as split_kernel's CTAs do.
// Bound by the power limit where sums are long: 4096 x 4096 x 14336 BF16 261
// us alone and 280 in a row (1.84 and 1.72 PFLOP/s, tensor pipe 93 % active),
// 8192 x 14336 x 4096 E4M3 with silu 267 and 296 us (3.60 and 3.25 PFLOP/s, 92
// %); where they are short, by the readout.
//
// Both operands are staged 128 bytes of k at a time in the 128-byte swizzled
// layout the MMA reads, by TMA.  A matrix whose address or row stride is not a
// multiple of 16 bytes, which TMA cannot read, is first copied to rows that
// are (align_kernel, 5.7 TB/s) in a workspace of the caller's.  Measured beside warps
// that realign rows on their way to shared memory, which take 1.2 us a stage
// (us, BF16): 4096 x 4097 x 4097 917, this 140; 256 x 4096 x 4097 85, this
// 34; 1 x 14336 x 4097 85, this 63.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "st_ops_device.h"

namespace stmat {
namespace {

constexpr int kTileN = 128;          // weight rows per tile: the MMA's M
constexpr int kStageK = 128;         // bytes of k per stage: one swizzle row
constexpr int kMaxStages = 12;       // ring slots
constexpr int kMaxSplit = 8;         // portable cluster size
constexpr int kEpilogueWarps = 4;    // one per 32 TMEM lanes
constexpr int kMmaWarp = 4, kCopyWarp = 5, kSplitThreads = 192;
constexpr uint32_t kWaitLimit = 1u << 22;

constexpr int kPairM = 256;          // tokens per pair of CTAs
constexpr int kMaxPairs = 4;         // pairs that share a tile's sum: portable clusters
constexpr int kPairMaxN = 256;       // weight rows per pair, a multiple of 32
// Three warps per 32 TMEM lanes, each with every third chunk of the columns: a
// product with a short sum is bound by its readout, whose chains of loads and
// arithmetic eight warps leave two thirds of the issue slots of; sixteen leave
// a thread 96 registers, twelve 128 (8192 x 4096 x 1024 E4M3: 39.0, 32.0, 28.2
// us).
constexpr int kDenseEpilogueWarps = 12;
constexpr int kDenseMmaWarp = 12, kDenseCopyWarp = 13, kDenseThreads = 448;
constexpr int kDenseSmem = 196 * 1024;  // the ring of stages; room for the rest of a CTA's 227 KB
constexpr int kChunk = 32;           // columns an epilogue warp reads at a time

// One operand of the product.
struct Side {
  const uint8_t *p;
  int64_t pitch;   // bytes between rows
  int64_t span;    // bytes from the first row's start to the last row's end
  int64_t rows;
};

struct LinArgs {
  Side w, x;
  int64_t m, n, kbytes;
  int k_blocks, splits, stages, m_tiles;
  int n_tiles, tile_n;               // dense_kernel: weight rows per tile
  int x_box;                         // token rows a TMA copy brings
  int vec;                           // y and residual rows take 32-byte (dense) or four-element (split) accesses
  uint32_t idesc;
  int eight;                         // 8-bit operands
  st_act act;
  st_dtype y_dtype, bias_dtype;
  const float *x_scale, *w_scale;
  int x_scale_step, w_scale_step;    // 0: one entry for all
  const void *bias, *residual;
  void *y;
  int64_t ldr, ldy;
  uint32_t *err;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
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

// --------------------------------------------------------- align_kernel

// Sixteen bytes of a matrix row at any alignment, read as the two aligned
// 16-byte words around them.  read() only issues loads, so that several
// chunks' can be under way; value() realigns.
struct Chunk {
  uint4 lo, hi;
  const uint8_t *p;
  int left;  // bytes of the row from p on (more than 16: 16); 0: zeros

  // The chunk `at` bytes into `row` of a side whose rows have row_bytes.
  __device__ __forceinline__ void read(const Side &s, int64_t row, int64_t at, int64_t row_bytes) {
    const int64_t rest = row < s.rows ? row_bytes - at : 0;
    left = rest >= 16 ? 16 : rest > 0 ? static_cast<int>(rest) : 0;
    p = s.p + row * s.pitch + at;
    const uint32_t r = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint8_t *a = p - r;
    // Words that leave the matrix are not read: such chunks go byte by byte.
    const bool whole = left == 16 && a >= s.p && a + (r ? 32 : 16) <= s.p + s.span;
    if (left && !whole) left |= 32;
    lo = hi = make_uint4(0, 0, 0, 0);
    if (whole) lo = *reinterpret_cast<const uint4 *>(a);
    if (whole && r) hi = *reinterpret_cast<const uint4 *>(a + 16);
  }

  __device__ __forceinline__ uint4 value() const {
    if (left & 32) {
      uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < (left & 31)) v[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
      return make_uint4(v[0], v[1], v[2], v[3]);
    }
    const uint32_t r = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15), sh = 8 * (r & 3);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t v[6], u[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = r & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) u[i] = r & 4 ? v[i + 1] : v[i];
    return make_uint4(__funnelshift_r(u[0], u[1], sh), __funnelshift_r(u[1], u[2], sh), __funnelshift_r(u[2], u[3], sh),
                      __funnelshift_r(u[3], u[4], sh));
  }
};

// Copies rows that TMA cannot read (an address or a stride that is no multiple
// of 16 bytes) to rows that it can.  A warp moves 2 KiB of a row, four chunks
// a lane, all of them under way before the first is stored.
struct AlignArgs {
  Side from[2];
  uint8_t *to[2];
  int64_t warps[2];  // warps for each matrix; 0: it stays where it is
  int64_t row_bytes, pitch;
  uint32_t segments;  // per row
};
constexpr int kAlignWarps = 8, kAlignEach = 4;

__global__ void __launch_bounds__(kAlignWarps * 32) align_kernel(const __grid_constant__ AlignArgs a) {
  wait_for_previous();
  let_next_start();
  int64_t w = int64_t(blockIdx.x) * kAlignWarps + (threadIdx.x >> 5);
  const int i = w >= a.warps[0];
  if (i) w -= a.warps[0];
  if (w >= a.warps[i]) return;
  const int64_t row = w / a.segments;
  const int64_t at0 = (w - row * a.segments) * (512 * kAlignEach) + (threadIdx.x & 31) * 16;
  Chunk c[kAlignEach];
#pragma unroll
  for (int e = 0; e < kAlignEach; ++e) c[e].read(a.from[i], row, at0 + 512 * e, a.row_bytes);
#pragma unroll
  for (int e = 0; e < kAlignEach; ++e)
    if (at0 + 512 * e < a.pitch) *reinterpret_cast<uint4 *>(a.to[i] + row * a.pitch + at0 + 512 * e) = c[e].value();
}

// ---------------------------------------------------------- split_kernel

template <int BM, bool kEight>
__global__ void __launch_bounds__(kSplitThreads)
split_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
             const __grid_constant__ LinArgs a) {
  constexpr int kStageBytes = (kTileN + BM) * kStageK;
  constexpr int kCols = BM < 32 ? 32 : BM;  // TMEM columns
  // The partial sums of 128 tokens (68 KB) lie over the stages, so that two
  // CTAs still share an SM; fewer tokens' have room of their own, and need not
  // wait for the whole cluster's MMAs.
  constexpr bool kOver = BM == 128;
  extern __shared__ uint8_t raw_smem[];
  uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_base;
  __shared__ int failed;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x % a.splits;
  const int64_t tile = blockIdx.x / a.splits;
  const int64_t m0 = tile % a.m_tiles * BM, n0 = tile / a.m_tiles * kTileN;
  const int first = static_cast<int>(int64_t(a.k_blocks) * rank / a.splits);
  const int blocks = static_cast<int>(int64_t(a.k_blocks) * (rank + 1) / a.splits) - first;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 1);
    }
    bar_init(&done, 1);
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "r"(kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  if (!kOver) cluster_arrive();
  wait_for_previous();
  let_next_start();

  Ring r;
  if (warp == kCopyWarp) {
    if (elect_one()) {
      int i = 0;
      constexpr int kStep = kEight ? kStageK : kStageK / 2;
      for (int at = first * kStep; i < blocks; ++i, at += kStep, r.next(a.stages)) {
        // Before its first use a stage counts as released.
        if (!bar_wait(&empty[r.at], r.phase ^ 1)) break;
        uint8_t *stage = smem + r.at * kStageBytes;
        bar_expect(&full[r.at], kTileN * kStageK + a.x_box * kStageK);
        tma_load(&wmap, stage, &full[r.at], at, static_cast<int32_t>(n0));
        tma_load(&xmap, stage + kTileN * kStageK, &full[r.at], at, static_cast<int32_t>(m0));
      }
      if (i < blocks) {  // a wait gave up: the copies in flight land before the CTA ends
        failed = 1;
        for (int j = i < a.stages ? 0 : i - a.stages; j < i; ++j) bar_wait(&full[j % a.stages], (j / a.stages) & 1);
      }
    }
  } else if (warp == kMmaWarp) {
    if (blocks > 0 && elect_one()) {
      uint32_t add = 0;
      for (int i = 0; i < blocks; ++i, r.next(a.stages)) {
        if (!bar_wait(&full[r.at], r.phase)) { failed = 1; break; }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t wd = tile_desc(smem + r.at * kStageBytes), xd = wd + (kTileN * kStageK >> 4);
#pragma unroll
        for (int j = 0; j < kStageK / 32; ++j, add = 1) mma<kEight>(tmem, wd + 2 * j, xd + 2 * j, a.idesc, add);
        mma_commit(&empty[r.at]);
      }
      mma_commit(&done);
    }
  }
  __syncwarp();

  // The tile's tokens are shared out: CTA r joins and writes `share` of them
  // from r * share on.  Every CTA puts its partial sums of a token into the
  // joining CTA's shared memory, [splits][share][kTileN].
  const int cols = static_cast<int>(a.m - m0 < BM ? a.m - m0 : BM), share = (cols + a.splits - 1) / a.splits;
  float *joined = reinterpret_cast<float *>(smem + (kOver ? 0 : a.stages * kStageBytes));
  // In the epilogue a lane has four consecutive weight rows, a warp every
  // fourth token.
  const int64_t n = n0 + 4 * lane;
  const int live = n < a.n ? static_cast<int>(min(int64_t(4), a.n - n)) : 0;
  const bool quad = live == 4 && a.vec;
  float ws[4], bias[4];
  if (warp < kEpilogueWarps) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float b[1] = {0.0f};
      if (a.bias && j < live) load_any<1>(a.bias, a.bias_dtype, n + j, b);
      ws[j] = a.w_scale && j < live ? a.w_scale[(n + j) * a.w_scale_step] : 1.0f;
      bias[j] = b[0];
    }
    if (blocks > 0 && !bar_wait(&done, 0, sum_limit(a.k_blocks))) failed = 1;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  }
  if (kOver) cluster_arrive();
  cluster_wait();  // every CTA runs (kOver: and is done with its stages)
  if (warp < kEpilogueWarps) {
    uint32_t owner = 0, to = peer_addr(joined + rank * share * kTileN + threadIdx.x, 0);
    int left = share;  // tokens of the owner's share to come
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (c + j >= cols) break;
        if (left == 0) {
          to = peer_addr(joined + rank * share * kTileN + threadIdx.x, ++owner);
          left = share;
        }
        peer_store(to, blocks > 0 ? __uint_as_float(v[j]) : 0.0f);
        to += kTileN * 4;
        --left;
      }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  cluster_arrive();

  // The residual may be y: a thread reads its values of a token, and one
  // token ahead, before it writes them.
  const int begin = static_cast<int>(rank) * share, mine = min(share, cols - begin);
  auto extras = [&](int c, float (&old)[4], float &xs) {
    const int64_t m = m0 + begin + c;
    xs = a.x_scale ? a.x_scale[m * a.x_scale_step] : 1.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) old[j] = 0.0f;
    if (!a.residual) return;
    if (quad) load_any<4>(a.residual, a.y_dtype, m * a.ldr + n, old);
    else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float o[1] = {0.0f};
        if (j < live) load_any<1>(a.residual, a.y_dtype, m * a.ldr + n + j, o);
        old[j] = o[0];
      }
    }
  };
  const bool writes = warp < kEpilogueWarps && warp < mine;
  float old[4], xs = 1.0f;
  if (writes) extras(warp, old, xs);
  cluster_wait();
  if (warp == kMmaWarp) {
    // The MMAs are done with the stages and TMEM, whatever the readout's wait
    // came to.
    if (blocks > 0 && !bar_wait(&done, 0, sum_limit(a.k_blocks))) failed = 1;
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
  }
  if (threadIdx.x == 0 && failed) atomicOr(a.err, kErrProduct);
  if (!writes) return;
#pragma unroll 1
  for (int c = warp; c < mine; c += kEpilogueWarps) {
    float next[4], next_xs = 1.0f;
    if (c + kEpilogueWarps < mine) extras(c + kEpilogueWarps, next, next_xs);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int r = 0; r < a.splits; ++r) {
      const float4 f = *reinterpret_cast<const float4 *>(joined + (r * share + c) * kTileN + 4 * lane);
      v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * xs * ws[j] + bias[j];
    if (a.y_dtype == ST_F32) activate<true>(v, a.act);
    else activate<false>(v, a.act);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += old[j], old[j] = next[j];
    xs = next_xs;
    const int64_t at = (m0 + begin + c) * a.ldy + n;
    if (quad) store_any<4>(a.y, a.y_dtype, at, v);
    else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float out[1] = {v[j]};
        if (j < live) store_any<1>(a.y, a.y_dtype, at + j, out);
      }
    }
  }
}

// ---------------------------------------------------------- dense_kernel

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
__device__ __forceinline__ int rows_from(const LinArgs &a, int64_t m) {
  return static_cast<int>(max(int64_t(0), min(int64_t(32), a.m - m)));
}
__device__ __forceinline__ void read_turned(const LinArgs &a, int64_t m0, int64_t n0, int lane, uint32_t (&old)[2][8]) {
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
__device__ __forceinline__ void put_turned(uint32_t (&w)[32][17], const LinArgs &a, int64_t m0, int64_t n0, int lane,
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
__device__ __forceinline__ void put_turned32(uint32_t (&w)[32][17], const LinArgs &a, int64_t m0, int64_t n0, int lane,
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

// Tile t of the launch: groups of eight token tiles, so that the tiles in
// flight share their operands in L2.
struct TileAt {
  int64_t m0, n0;
};
__device__ __forceinline__ TileAt tile_at(const LinArgs &a, int t) {
  constexpr int kGroup = 8;
  const int per = kGroup * a.n_tiles, g = t / per, in = t % per;
  const int rows = min(kGroup, a.m_tiles - g * kGroup);
  return {int64_t(g * kGroup + in % rows) * kPairM, int64_t(in / rows) * a.tile_n};
}

// kShared: one tile a cluster, its sum over k shared by the cluster's pairs.
// kF32: y's type, with an activation (exact_act).
template <bool kEight, bool kShared, bool kF32>
__global__ void __launch_bounds__(kDenseThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
             const __grid_constant__ LinArgs a) {
  extern __shared__ uint8_t raw_smem[];
  uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sums[2], taken[2];
  __shared__ uint32_t tmem_base;
  __shared__ int failed;
  __shared__ __align__(16) uint32_t turn[kDenseEpilogueWarps][32][17];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = kShared ? a.splits : 1;
  const uint32_t in_cluster = blockIdx.x % (2 * splits), rank = in_cluster & 1, leader = in_cluster & ~1u;
  const int split = static_cast<int>(in_cluster >> 1), tiles = a.m_tiles * a.n_tiles;
  const int pair = blockIdx.x / (2 * splits), pairs = gridDim.x / (2 * splits);
  const int half_n = a.tile_n / 2, stage_bytes = (128 + half_n) * kStageK;
  const int first = static_cast<int>(int64_t(a.k_blocks) * split / splits);
  const int blocks = static_cast<int>(int64_t(a.k_blocks) * (split + 1) / splits) - first;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sums[i], 1);
      bar_init(&taken[i], 2 * kDenseEpilogueWarps);
    }
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kDenseMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  wait_for_previous();
  let_next_start();

  const int quarter = warp & 3, chunks = a.tile_n / kChunk;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const bool columns_scaled = a.w_scale && a.w_scale_step;
  // The token's scale, and the weight's where it is a single one.
  auto scale_of = [&](int t) {
    const int64_t m = tile_at(a, t).m0 + rank * 128 + quarter * 32 + lane;
    float xs = m < a.m && a.x_scale ? a.x_scale[m * a.x_scale_step] : 1.0f;
    if (a.w_scale && !columns_scaled) xs *= *a.w_scale;
    return xs;
  };
  // Chunk c of a tile: its sums, read by `sums_of`, to y.
  auto finish = [&](const TileAt &at, int c, float xs, auto sums_of) {
    const int64_t mw = at.m0 + rank * 128 + quarter * 32, m = mw + lane, n0 = at.n0 + c * kChunk;
    const bool row = m < a.m, wide = a.vec && n0 + kChunk <= a.n;
    uint32_t old[2][8];
    if (a.residual && a.y_dtype != ST_F32) {
      if (!wide) read_turned(a, mw, n0, lane, old);
      else if (row) {
#pragma unroll
        for (int i = 0; i < 2; ++i) ld32(static_cast<const uint16_t *>(a.residual) + m * a.ldr + n0 + 16 * i, old[i]);
      }
    }
    // One column's scale and bias per lane, handed round below.
    float wl = 1.0f, bl[1] = {0.0f};
    if (n0 + lane < a.n) {
      if (columns_scaled) wl = a.w_scale[n0 + lane];
      if (a.bias) load_any<1>(a.bias, a.bias_dtype, n0 + lane, bl);
    }
    float v[kChunk];
    sums_of(v);
#pragma unroll
    for (int j = 0; j < kChunk; ++j) v[j] *= xs;
    if (columns_scaled) {
#pragma unroll
      for (int j = 0; j < kChunk; ++j) v[j] *= __shfl_sync(~0u, wl, j);
    }
    if (a.bias) {
      float *const all = reinterpret_cast<float *>(turn[warp]);
      __syncwarp();
      all[lane] = bl[0];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kChunk; j += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(all + j);
        v[j] += f.x, v[j + 1] += f.y, v[j + 2] += f.z, v[j + 3] += f.w;
      }
    }
    activate<kF32>(v, a.act);
    if (wide) {
      if (row) {
        if (a.residual && a.y_dtype != ST_F32) {
#pragma unroll
          for (int i = 0; i < 2; ++i) add16(old[i], a.y_dtype == ST_BF16, v + 16 * i);
        } else if (a.residual) add_row32(a.residual, m * a.ldr + n0, v);
        put_row(a.y, a.y_dtype, m * a.ldy + n0, v);
      }
    } else if (a.y_dtype == ST_BF16) put_turned<__nv_bfloat16>(turn[warp], a, mw, n0, lane, old, v);
    else if (a.y_dtype == ST_F16) put_turned<__half>(turn[warp], a, mw, n0, lane, old, v);
    else put_turned32(turn[warp], a, mw, n0, lane, v);
  };

  Ring r;
  if (warp == kDenseCopyWarp) {
    if (elect_one()) {
      // This CTA's tokens and its half of the weight rows; the bytes of both
      // CTAs count on the first one's barriers.
      const uint32_t bars = peer_addr(full, leader);
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const TileAt at = tile_at(a, t);
        const int32_t m = static_cast<int32_t>(at.m0 + rank * 128), n = static_cast<int32_t>(at.n0 + rank * half_n);
        constexpr int kStep = kEight ? kStageK : kStageK / 2;
        for (int b = 0, k = first * kStep; b < blocks; ++b, k += kStep, r.next(a.stages)) {
          // Before its first use a stage counts as released.
          if (!bar_wait(&empty[r.at], r.phase ^ 1)) { ok = false; break; }
          uint8_t *stage = smem + r.at * stage_bytes;
          if (rank == 0) bar_expect(&full[r.at], 2 * stage_bytes);
          pair_load(&xmap, stage, bars + 8 * r.at, k, m);
          pair_load(&wmap, stage + 128 * kStageK, bars + 8 * r.at, k, n);
        }
      }
      // The stages in flight are released (or, after a wait that gave up,
      // have had their time) before the CTA ends.
      for (int i = 0; i < a.stages; ++i, r.next(a.stages)) ok &= bar_wait(&empty[r.at], r.phase ^ 1);
      if (!ok) failed = 1;
    }
  } else if (warp == kDenseMmaWarp) {
    if (rank == 0 && elect_one()) {
      Ring sum;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, sum.next(2)) {
        if (!bar_wait(&taken[sum.at], sum.phase ^ 1)) { ok = false; break; }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + sum.at * kPairMaxN;
        uint32_t add = 0;
        for (int b = 0; b < blocks; ++b, r.next(a.stages)) {
          if (!bar_wait(&full[r.at], r.phase)) { ok = false; break; }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t xd = tile_desc(smem + r.at * stage_bytes), wd = xd + (128 * kStageK >> 4);
#pragma unroll
          for (int j = 0; j < kStageK / 32; ++j, add = 1) pair_mma<kEight>(d, xd + 2 * j, wd + 2 * j, a.idesc, add);
          pair_commit(&empty[r.at], leader);
        }
        pair_commit(&sums[sum.at], leader);
      }
      if (!ok) failed = 1;
    }
  } else if (!kShared) {
    const uint32_t taken_at = peer_addr(taken, leader);
    // A tile's scales are read while the one before it is written.
    float next_xs = pair < tiles ? scale_of(pair) : 1.0f;
    int n = 0;
    for (int t = pair; t < tiles; t += pairs, ++n) {
      const TileAt at = tile_at(a, t);
      const int buf = n & 1;
      const float xs = next_xs;
      if (t + pairs < tiles) next_xs = scale_of(t + pairs);
      // The half of TMEM is given back as soon as this warp has read its part.
      auto release = [&]() {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) peer_arrive(taken_at + 8 * buf);
      };
      const int live = static_cast<int>(min(int64_t(chunks), (a.n - at.n0 + kChunk - 1) / kChunk));
      if (!bar_wait_warp(&sums[buf], (n / 2) & 1, lane, sum_limit(a.k_blocks))) { failed = 1; break; }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      if (warp >> 2 >= live) release();
      for (int c = warp >> 2; c < live; c += kDenseEpilogueWarps / 4)
        finish(at, c, xs, [&](float(&v)[kChunk]) {
          tmem_ld32(lanes + buf * kPairMaxN + c * kChunk, v);
          if (c + kDenseEpilogueWarps / 4 >= live) release();
        });
    }
  }
  __syncwarp();
  if constexpr (kShared) {
    // Once every pair is done with its stages, each CTA
    // puts its partial sums of a chunk of columns into the CTA that joins it:
    // pair s has chunks [s per, (s + 1) per), from every pair's CTA with the
    // same tokens, [splits][per][column][token] over the stages.
    const int per = chunks / splits;
    float *joined = reinterpret_cast<float *>(smem);
    const bool reads = warp < kDenseEpilogueWarps;
    float xs = 1.0f;
    if (reads) {
      xs = scale_of(pair);
      if (!bar_wait_warp(&sums[0], 0, lane, sum_limit(a.k_blocks))) failed = 1;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    cluster_arrive();
    cluster_wait();
    if (reads) {
      for (int c = warp >> 2; c < chunks; c += kDenseEpilogueWarps / 4) {
        float v[kChunk];
        tmem_ld32(lanes + c * kChunk, v);
        const uint32_t to = peer_addr(joined + ((split * per + c % per) * kChunk * 128 + quarter * 32 + lane), 2 * (c / per) + rank);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) peer_store(to + j * 128 * 4, v[j]);
      }
    }
    cluster_arrive();
    cluster_wait();
    if (reads) {
      const TileAt at = tile_at(a, pair);
      const int live = static_cast<int>(min(int64_t(chunks), (a.n - at.n0 + kChunk - 1) / kChunk));
      for (int c = warp >> 2; c < per && split * per + c < live; c += kDenseEpilogueWarps / 4)
        finish(at, split * per + c, xs, [&](float(&v)[kChunk]) {
          const float *from = joined + c * kChunk * 128 + quarter * 32 + lane;
#pragma unroll
          for (int j = 0; j < kChunk; ++j) v[j] = from[j * 128];
          for (int s = 1; s < splits; ++s) {
            from += per * kChunk * 128;
#pragma unroll
            for (int j = 0; j < kChunk; ++j) v[j] += from[j * 128];
          }
        });
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kDenseMmaWarp) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if (threadIdx.x == 0 && failed) atomicOr(a.err, kErrProduct);
}

// ------------------------------------------------------------------- host

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

st_status encoder(EncodeFn *out) {
  static std::mutex mu;
  static EncodeFn fn = nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || !p)
      return set_error(ST_E_CUDA, "st_linear: the driver has no cuTensorMapEncodeTiled (%s)", cudaGetErrorName(e));
    fn = reinterpret_cast<EncodeFn>(p);
  }
  *out = fn;
  return ST_OK;
}

// Whether TMA can read the matrix: address and row stride multiples of 16
// bytes, the stride under 2^40.
bool tma_ok(const Side &s) {
  return reinterpret_cast<uintptr_t>(s.p) % 16 == 0 && (s.rows == 1 || (s.pitch > 0 && s.pitch % 16 == 0 && s.pitch < (int64_t(1) << 40)));
}

st_status encode(CUtensorMap *map, const Side &s, int64_t k, int item, int box_rows) {
  EncodeFn fn = nullptr;
  const st_status st = encoder(&fn);
  if (st != ST_OK) return st;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(s.rows)};
  const cuuint64_t stride[1] = {s.rows == 1 ? static_cast<cuuint64_t>((k * item + 15) / 16 * 16) : static_cast<cuuint64_t>(s.pitch)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kStageK / item), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  const CUresult r = fn(map, item == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                        const_cast<uint8_t *>(s.p), dims, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(ST_E_CUDA, "st_linear: tensor map of %lld x %lld refused (%d)", (long long)s.rows, (long long)k, static_cast<int>(r));
  return ST_OK;
}

// What launches on a device need, looked up on its first one.
constexpr int kMaxDevices = 256;
struct Device {
  int sms = 0;
  int clusters[kMaxPairs + 1] = {};  // clusters of so many pairs that dense_kernel runs at a time
  uint32_t *err = nullptr;
};

void cluster_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, unsigned blocks, unsigned threads, size_t smem, unsigned cluster) {
  cfg->gridDim = dim3(blocks);
  cfg->blockDim = dim3(threads);
  cfg->dynamicSmemBytes = smem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

st_status device(int *index, const Device **out) {
  static std::mutex mu;
  static Device known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev >= kMaxDevices) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) return set_error(ST_E_CUDA, "st_linear: the current device: %s", cudaGetErrorName(e));
  std::lock_guard<std::mutex> lock(mu);
  Device &d = known[dev];
  if (!d.err) {
    void *scratch = nullptr;
    const st_status s = static_scratch(&scratch);
    if (s != ST_OK) return s;
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(dense_kernel<true, true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDenseSmem + 1024);
    for (int pairs = 1; pairs <= kMaxPairs && e == cudaSuccess; pairs *= 2) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      cluster_config(&cfg, attr, 2 * pairs, kDenseThreads, kDenseSmem + 1024, 2 * pairs);
      e = cudaOccupancyMaxActiveClusters(&d.clusters[pairs], dense_kernel<true, true, false>, &cfg);
    }
    if (e != cudaSuccess) return set_error(ST_E_CUDA, "st_linear: counting SMs and clusters: %s", cudaGetErrorName(e));
    d.err = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(scratch) + kStaticErrOffset);
  }
  *index = dev;
  *out = &d;
  return ST_OK;
}

// Raises a kernel's limit of dynamic shared memory, once per kernel and device.
template <auto kKernel>
cudaError_t allow_smem(int dev, int bytes) {
  static std::atomic<bool> done[kMaxDevices];
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

// How a kernel would cut a product, and its time in units of one 128-byte
// row brought into an SM (1.2 ns, measured), without what every launch costs.
struct Shape {
  int64_t m_tiles, n_tiles;
  int width, splits;  // as in st_linear_form
  double cost;
};

// dense_kernel: rounds of tiles over the pairs; a stage takes as long as its
// rows (1.08 units each: 64 columns wide, 0.207 us a stage) or its MMAs,
// whichever is longer, and a tile as long as its stages or its readout (1500
// units and 8 a column).  The width of a tile is the one with the shortest rounds in
// all (4096 x 4096 x 14336 BF16: 224 columns, four full rounds, 285 us; 256
// columns, 314).  Few tiles with long sums are each shared by a cluster of pairs,
// if all of the clusters run at a time, for 18 units a column of joining (us,
// without and with: 256 x 4096 x 14336 E4M3 23.8, 19.6, BF16 35.8, 31.0; 256 x
// 1024 x 4096 E4M3 10.5, 8.7; 512 x 4096 x 4096 BF16 18.4, 20.3).  The cost
// compared with split_kernel's is that of the shortest stages and the joining,
// without the start and the readout, which count for a few tokens only
// (choose).
Shape dense_shape(int64_t m, int64_t n, int k_blocks, const Device &gpu) {
  Shape best{};
  double shortest = 0, cost = 0;
  const int64_t m_tiles = (m + kPairM - 1) / kPairM;
  for (int pairs = 1; pairs <= kMaxPairs; pairs *= 2) {
    for (int w = kPairMaxN; w >= 32 * pairs; w -= 32) {
      const int64_t n_tiles = (n + w - 1) / w, tiles = m_tiles * n_tiles;
      if (pairs > 1 && (w % (32 * pairs) || tiles > gpu.clusters[pairs] || k_blocks < 4 * pairs)) continue;
      const double rounds = pairs > 1 ? 1 : static_cast<double>((tiles + gpu.sms / 2 - 1) / (gpu.sms / 2));
      const double stages = (k_blocks + pairs - 1) / pairs * std::max(1.08 * (128 + w / 2), 0.87 * w);
      const double join = pairs > 1 ? 18.0 * w : 0, all = rounds * std::max(stages, 1500 + 8.0 * w) + join;
      cost = best.width == 0 ? rounds * stages + join : std::min(cost, rounds * stages + join);
      if (best.width == 0 || all < shortest) best = Shape{m_tiles, n_tiles, w, pairs, 0}, shortest = all;
    }
  }
  best.cost = cost;
  return best;
}

// split_kernel: the MMA's columns are the tokens, up to 128; the sum is split
// until the CTAs fill the SMs twice, each with at least four stages.  Joining
// and writing a tile costs 26 units per column, and a part of a round of CTAs
// costs about half of a whole one.  (Device time in us, this and dense_kernel:
// 64 x 4096 x 4096 E4M3 8.8, 11.3; 128 x 4096 x 4096 14.3, 10.6; 128 x 4096 x
// 14336 20.4, 25.9; 384 x 4096 x 14336 BF16 56, 46.)
Shape split_shape(int64_t m, int64_t n, int k_blocks, int sms) {
  Shape s{};
  s.width = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  s.m_tiles = (m + s.width - 1) / s.width;
  s.n_tiles = (n + kTileN - 1) / kTileN;
  const int64_t tiles = s.m_tiles * s.n_tiles;
  s.splits = 1;
  while (s.splits < kMaxSplit && tiles * s.splits <= sms && k_blocks / (s.splits * 2) >= 4) s.splits *= 2;
  const int64_t ctas = tiles * s.splits, rounds = (ctas + sms - 1) / sms;
  s.cost = 0.5 * (static_cast<double>(rounds) + (ctas > sms ? static_cast<double>(ctas) / sms : 1.0)) * ((k_blocks + s.splits - 1) / s.splits * (kTileN + s.width) + 26.0 * s.width);
  return s;
}

// For up to so many tokens dense_kernel's start and readout, 1300 units and 8 a
// column more than split_kernel's, outweigh its shorter stages wherever sums are
// short (device time in us, split_kernel and dense_kernel: 1 x 28672 x 64 BF16
// 2.9, 6.5; 1 x 304 x 256 3.6, 4.1; 8 x 4096 x 256 3.9, 5.7; 8 x 64 x 448 4.7,
// 4.7; 0.7 of the time in the middle of 276 sizes with up to 1 KB of k).  With
// 16 tokens split_kernel's readout has caught up (16 x 64 x 256 BF16 5.4, 4.2;
// 16 x 4096 x 448 5.3, 5.9).
constexpr int64_t kFewTokens = 8;

st_status launch_error(const LinArgs &a, cudaError_t e) {
  return set_error(ST_E_CUDA, "st_linear launch (%lld x %lld, %lld bytes of k): %s: %s", (long long)a.m, (long long)a.n,
                   (long long)a.kbytes, cudaGetErrorName(e), cudaGetErrorString(e));
}

template <int BM, bool kEight>
st_status launch_split(LinArgs &a, const CUtensorMap &wmap, const CUtensorMap &xmap, int64_t tiles, int dev, cudaStream_t st) {
  constexpr int kStageBytes = (kTileN + BM) * kStageK;
  // About half of the SM's shared memory, so that two CTAs share one.
  constexpr int kJoined = (BM + kMaxSplit) * kTileN * 4, kBudget = 109 * 1024;
  constexpr int kStages = BM == 128 ? 3 : (kBudget - kJoined) / kStageBytes;
  static_assert(kStages >= 3 && kStages <= kMaxStages && (BM < 128 || kJoined <= kStages * kStageBytes), "a ring of stages");
  a.stages = kStages;
  constexpr int smem = kStages * kStageBytes + (BM == 128 ? 0 : kJoined) + 1024;
  constexpr auto kernel = split_kernel<BM, kEight>;
  cudaError_t e = allow_smem<kernel>(dev, smem);
  if (e == cudaSuccess)
    e = launch(kernel, static_cast<unsigned>(tiles * a.splits), kSplitThreads, smem, a.splits, st, wmap, xmap, a);
  return e == cudaSuccess ? ST_OK : launch_error(a, e);
}

template <bool kEight, bool kShared, bool kF32>
st_status launch_dense(LinArgs &a, const CUtensorMap &xmap, const CUtensorMap &wmap, int dev, int sms, cudaStream_t st) {
  // As many stages as fit: a narrow tile's are smaller, and need more of them
  // under way to cover the memory's latency.
  const int stage_bytes = (128 + a.tile_n / 2) * kStageK;
  a.stages = kDenseSmem / stage_bytes < kMaxStages ? kDenseSmem / stage_bytes : kMaxStages;
  cudaError_t e = allow_smem<dense_kernel<kEight, kShared, kF32>>(dev, kDenseSmem + 1024);
  if (e == cudaSuccess) {
    const int pairs = sms / 2, tiles = a.m_tiles * a.n_tiles;
    e = launch(dense_kernel<kEight, kShared, kF32>, 2 * (kShared ? tiles * a.splits : std::min(tiles, pairs)), kDenseThreads,
               a.stages * stage_bytes + 1024, 2 * a.splits, st, xmap, wmap, a);
  }
  return e == cudaSuccess ? ST_OK : launch_error(a, e);
}

}  // namespace

namespace {

int item_of(const st_linear_args &p) { return p.x_dtype == ST_BF16 || p.x_dtype == ST_F16 ? 2 : 1; }

Side side_of(const void *ptr, int64_t ld, int64_t rows, int64_t k, int item) {
  return Side{static_cast<const uint8_t *>(ptr), ld * item, ld * item * (rows - 1) + k * item, rows};
}

// Copies the operands that TMA cannot read to aligned rows in the workspace
// and points the arguments at them.
st_status align(LinArgs &a, uint8_t *workspace, cudaStream_t st) {
  AlignArgs al{};
  al.row_bytes = a.kbytes;
  al.pitch = (a.kbytes + 15) / 16 * 16;
  al.segments = static_cast<uint32_t>((al.pitch + 512 * kAlignEach - 1) / (512 * kAlignEach));
  Side *sides[2] = {&a.w, &a.x};
  for (int i = 0; i < 2; ++i) {
    Side &s = *sides[i];
    if (a.kbytes == 0 || tma_ok(s)) continue;
    al.from[i] = s;
    al.to[i] = workspace;
    al.warps[i] = s.rows * al.segments;
    workspace += s.rows * al.pitch;
    s.p = al.to[i];
    s.pitch = al.pitch;
  }
  const int64_t blocks = (al.warps[0] + al.warps[1] + kAlignWarps - 1) / kAlignWarps;
  if (blocks == 0) return ST_OK;
  if (blocks > 0x7fffffff) return set_error(ST_E_INVAL, "st_linear: too many rows to align in one launch");
  const cudaError_t e = launch(align_kernel, static_cast<unsigned>(blocks), kAlignWarps * 32, 0, 1, st, al);
  if (e != cudaSuccess) return set_error(ST_E_CUDA, "st_linear: aligning rows: %s: %s", cudaGetErrorName(e), cudaGetErrorString(e));
  return ST_OK;
}

}  // namespace

int64_t linear_workspace(const st_linear_args &p) {
  const int item = item_of(p);
  const int64_t pitch = (p.k * item + 15) / 16 * 16;
  int64_t bytes = 0;
  if (p.k > 0 && !tma_ok(side_of(p.w, p.ldw, p.n, p.k, item))) bytes += p.n * pitch;
  if (p.k > 0 && !tma_ok(side_of(p.x, p.ldx, p.m, p.k, item))) bytes += p.m * pitch;
  return bytes;
}

namespace {

int blocks_of(const st_linear_args &p) { return static_cast<int>((p.k * item_of(p) + kStageK - 1) / kStageK); }

// The cheaper kernel's shape.
Shape choose(const st_linear_args &p, const Device &gpu, bool *dense) {
  const int k_blocks = blocks_of(p);
  const Shape d = dense_shape(p.m, p.n, k_blocks, gpu), c = split_shape(p.m, p.n, k_blocks, gpu.sms);
  const double more = p.m <= kFewTokens ? 1300 + 8.0 * d.width : 0;
  *dense = p.k > 0 && d.cost + more < c.cost;
  return *dense ? d : c;
}

Shape shape_of(const st_linear_args &p, const st_linear_form &f) {
  const bool dense = f.kernel == ST_LINEAR_DENSE;
  const int64_t rows = dense ? kPairM : f.width, columns = dense ? f.width : kTileN;
  return Shape{(p.m + rows - 1) / rows, (p.n + columns - 1) / columns, f.width, f.splits, 0};
}

}  // namespace

st_status check_linear_form(const st_linear_args &p, const st_linear_form &f) {
  const bool dense = f.kernel == ST_LINEAR_DENSE;
  const int most = dense ? kMaxPairs : kMaxSplit;
  bool ok = (dense || f.kernel == ST_LINEAR_SPLIT) && f.splits >= 1 && f.splits <= most && !(f.splits & (f.splits - 1));
  ok = ok && (dense ? f.width >= 32 && f.width <= kPairMaxN && f.width % (32 * f.splits) == 0
                    : f.width == 16 || f.width == 32 || f.width == 64 || f.width == 128);
  if (!ok) return set_error(ST_E_INVAL, "st_linear: no kernel %d has tiles of width %d and sums in %d parts", f.kernel, f.width, f.splits);
  if (f.splits > std::max(1, blocks_of(p)) || (dense && p.k == 0))
    return set_error(ST_E_INVAL, "st_linear: a sum of %d runs of 128 bytes in %d parts", blocks_of(p), f.splits);
  return ST_OK;
}

st_linear_form choose_linear_form(const st_linear_args &p, int sms, int clusters_of_2, int clusters_of_4) {
  Device gpu{};
  gpu.sms = sms;
  gpu.clusters[1] = sms / 2;
  gpu.clusters[2] = clusters_of_2;
  gpu.clusters[4] = clusters_of_4;
  bool dense = false;
  const Shape s = choose(p, gpu, &dense);
  return {dense ? ST_LINEAR_DENSE : ST_LINEAR_SPLIT, s.width, s.splits};
}

st_status launch_linear(const st_linear_args &p, const st_linear_form *form, void *stream) {
  const int item = item_of(p);
  LinArgs a{};
  a.m = p.m; a.n = p.n; a.kbytes = p.k * item;
  a.eight = item == 1;
  a.act = p.act; a.y_dtype = p.y_dtype; a.bias_dtype = p.bias_dtype;
  a.x_scale = p.x_scale; a.w_scale = p.w_scale;
  a.x_scale_step = p.x_scale_count > 1; a.w_scale_step = p.w_scale_count > 1;
  a.bias = p.bias; a.residual = p.residual; a.y = p.y;
  a.ldr = p.ldr; a.ldy = p.ldy;
  a.x = side_of(p.x, p.ldx, p.m, p.k, item);
  a.w = side_of(p.w, p.ldw, p.n, p.k, item);
  int dev = 0;
  const Device *gpu = nullptr;
  st_status s = device(&dev, &gpu);
  if (s != ST_OK) return s;
  a.err = gpu->err;
  const int sms = gpu->sms;
  a.k_blocks = blocks_of(p);
  // Instruction descriptor: binary32 accumulators; formats of A and B, both
  // K-major; rows and columns of one MMA.
  const uint32_t fw = item == 2 ? (p.w_dtype == ST_BF16) : (p.w_dtype == ST_F8_E5M2), fx = item == 2 ? (p.x_dtype == ST_BF16) : 0;
  auto idesc = [](uint32_t fa, uint32_t fb, uint32_t rows, uint32_t cols) {
    return (1u << 4) | (fa << 7) | (fb << 10) | ((cols / 8) << 17) | ((rows / 16) << 24);
  };
  CUtensorMap wmap{}, xmap{};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  s = align(a, static_cast<uint8_t *>(p.workspace), st);
  if (s != ST_OK) return s;

  const int64_t out = static_cast<int64_t>(st_dtype_size(p.y_dtype));
  auto aligned = [&](int64_t to) {
    auto one = [&](const void *q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % to == 0 && ld * out % to == 0; };
    return one(p.y, p.ldy) && (!p.residual || one(p.residual, p.ldr));
  };

  bool dense = form && form->kernel == ST_LINEAR_DENSE;
  const Shape shape = form ? shape_of(p, *form) : choose(p, *gpu, &dense);
  const int64_t tiles = shape.m_tiles * shape.n_tiles;
  a.splits = shape.splits;
  if (dense) {
    if (2 * tiles * a.splits > 0x7fffffff)
      return set_error(ST_E_INVAL, "st_linear: %lld x %lld needs more tiles than one launch has", (long long)p.m, (long long)p.n);
    a.m_tiles = static_cast<int>(shape.m_tiles);
    a.n_tiles = static_cast<int>(shape.n_tiles);
    a.tile_n = shape.width;
    a.idesc = idesc(fx, fw, kPairM, a.tile_n);
    a.vec = aligned(32);
    s = encode(&xmap, a.x, p.k, item, 128);
    if (s == ST_OK) s = encode(&wmap, a.w, p.k, item, a.tile_n / 2);
    if (s != ST_OK) return s;
    auto with = [](bool yes, auto &&f) { return yes ? f(std::true_type{}) : f(std::false_type{}); };
    return with(a.eight, [&](auto eight) {
      return with(a.splits > 1, [&](auto shared) {
        return with(exact_act(a.act, a.y_dtype), [&](auto f32) {
          return launch_dense<decltype(eight)::value, decltype(shared)::value, decltype(f32)::value>(a, xmap, wmap, dev, sms, st);
        });
      });
    });
  }

  a.vec = aligned(4 * out);
  a.m_tiles = static_cast<int>(shape.m_tiles);
  const int bm = shape.width;
  if (tiles * a.splits > 0x7fffffff)
    return set_error(ST_E_INVAL, "st_linear: %lld x %lld needs more tiles than one launch has", (long long)p.m, (long long)p.n);
  a.idesc = idesc(fw, fx, kTileN, bm);
  if (p.k > 0) {
    s = encode(&wmap, a.w, p.k, item, kTileN);
    // Fewer tokens than the MMA's columns: only they are copied (what the other
    // columns hold reaches no sum that is read).
    a.x_box = p.m < bm ? static_cast<int>(p.m) : bm;
    if (s == ST_OK) s = encode(&xmap, a.x, p.k, item, a.x_box);
    if (s != ST_OK) return s;
  }
#define ST_SPLIT(BM) \
  (a.eight ? launch_split<BM, true>(a, wmap, xmap, tiles, dev, st) : launch_split<BM, false>(a, wmap, xmap, tiles, dev, st))
  switch (bm) {
    case 16: return ST_SPLIT(16);
    case 32: return ST_SPLIT(32);
    case 64: return ST_SPLIT(64);
    default: return ST_SPLIT(128);
  }
#undef ST_SPLIT
}

}  // namespace stmat
