// st_block_linear.cu -- the product of 8-bit rows that have a scale for every
// 128 columns with an 8-bit weight that has one for every 128 x 128 block, for
// GB300 (sm_103a).
//
//   y[i, j] = act(sum_b xs[i, b] ws[j / 128, b] sum_{l in b} x[i, l] w[j, l] + bias[j]) + residual[i, j]
//
// A block's scales are binary32 numbers, which the tensor core cannot apply: a
// stage of 128 columns is one block, its products are summed by the tensor
// core alone (four MMAs), and the block's sums go from TMEM through one
// multiplication and addition each into registers, while the next blocks'
// are formed elsewhere in TMEM.
//
// block_split_kernel, few tokens: as st_linear's split_kernel the weight's rows
// (128 a tile, so one scale a block) are the MMA's rows and the tokens its
// columns, and the sum is split over the CTAs of a cluster, which put their
// partial sums into the shared memory of the CTA that joins them, in rank
// order (no workspace, no atomics, the same bits on every run).
//
// block_dense_kernel, many tokens: a pair of CTAs computes 256 tokens x up to
// 256 weight rows.  A thread of the eight readout warps has a token's sums for
// half of the columns in registers (128 of them), so that its scale of a block
// is one number, or two where its columns meet two of the weight's blocks.
//
// Bound, few tokens: HBM, behind a launch's chain of first copies, last MMAs
// and join (1 x 14336 x 4096 13.1 us, 8.8 by the weight's bytes; 64 x 4096 x 14336
// 17.1, 9.1).  Many: a block's chain.  Its four MMAs take 1100-1300 clocks from
// their issue to their signal, their sums' way out of TMEM about 450, and TMEM
// holds two blocks of 256 columns, so that a block is not done in less than
// about 840, where the MMAs alone would take 512: 8192 x 14336 x 4096 374 us
// (2.6 PFLOP/s; 244 at the tensor core's measured rate), the tensor pipe half
// active.  With silu 417: its exponential and reciprocal, on the one unit that
// has them, add 2400 clocks a tile to the 3800 that writes it.  Registers are
// full: 64 bytes of spill in the loop over blocks cost 12 %.
#include "st_tensor_device.h"

namespace stmat {
namespace {

constexpr int kTileN = 128;          // weight rows per tile of block_split_kernel: the MMA's M
constexpr int kBlockK = 128;         // columns of a scale: one stage
constexpr int kMaxSplit = 8;         // portable cluster size
constexpr int kSumWarps = 4;         // block_split_kernel: one per 32 TMEM lanes
constexpr int kMmaWarp = 4, kCopyWarp = 5, kSplitThreads = 192;

constexpr int kPairM = 256;          // tokens per pair of CTAs
constexpr int kPairMaxN = 256;       // weight rows per pair, a multiple of 64
constexpr int kDenseSumWarps = 8;
constexpr int kDenseMmaWarp = 8, kDenseCopyWarp = 9, kDenseThreads = 384;
// Three warpgroups start with 168 registers a thread; the two that hold sums
// take 240, the third gives the rest (2 x 240 + 24 = 3 x 168).
constexpr int kSumRegisters = 240, kFeedRegisters = 24;
constexpr int kDenseSmem = 224 * 1024;  // the ring of stages, and y's tile
// A readout warp's part of y's tile in 16 bits, or what rows at any place are
// turned in.
__host__ __device__ constexpr int part_bytes(int w) { return w * 32 > 3 * 1024 ? w * 32 : 3 * 1024; }

struct BlockArgs : OutArgs {
  Side w, x;
  int64_t kbytes;
  int k_blocks, splits, stages, m_tiles, n_tiles;
  int x_box;                         // token rows a TMA copy brings
  uint32_t idesc;
  int tma_store;                     // y is written, and the residual read, by TMA
  const float *x_scale, *w_scale;
  int64_t ldxs, ldws;
  uint32_t *err;
};

// --------------------------------------------------- block_split_kernel

template <int BM>
__global__ void __launch_bounds__(kSplitThreads)
block_split_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const __grid_constant__ BlockArgs a) {
  constexpr int kStageBytes = (kTileN + BM) * kStageK;
  constexpr int kCols = BM;                           // TMEM columns of a block's sums
  constexpr bool kOver = BM == 128;                   // partial sums lie over the stages
  extern __shared__ uint8_t raw_smem[];
  uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sums[2], taken[2];
  __shared__ uint32_t tmem_base;
  __shared__ int failed;
  __shared__ __align__(16) float scales[kSumWarps][2][BM];

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
    for (int i = 0; i < 2; ++i) {
      bar_init(&sums[i], 1);
      bar_init(&taken[i], kSumWarps);
    }
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "r"(2 * kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  if (!kOver) cluster_arrive();
  wait_for_previous();
  let_next_start();

  const int cols = static_cast<int>(a.m - m0 < BM ? a.m - m0 : BM);
  Ring r;
  float acc[BM];
  if (warp == kCopyWarp) {
    if (elect_one()) {
      bool ok = true;
      for (int i = 0; i < blocks; ++i, r.next(a.stages)) {
        // Before its first use a stage counts as released.
        if (!bar_wait(&empty[r.at], r.phase ^ 1)) { ok = false; break; }
        uint8_t *stage = smem + r.at * kStageBytes;
        bar_expect(&full[r.at], kTileN * kStageK + a.x_box * kStageK);
        tma_load(&wmap, stage, &full[r.at], (first + i) * kStageK, static_cast<int32_t>(n0));
        tma_load(&xmap, stage + kTileN * kStageK, &full[r.at], (first + i) * kStageK, static_cast<int32_t>(m0));
      }
      // The stages in flight are released (or, after a wait that gave up,
      // have had their time) before the CTA ends.
      for (int i = 0; i < a.stages; ++i, r.next(a.stages)) ok &= bar_wait(&empty[r.at], r.phase ^ 1);
      if (!ok) failed = 1;
    }
  } else if (warp == kMmaWarp) {
    if (elect_one()) {
      Ring sum;
      for (int i = 0; i < blocks; ++i, r.next(a.stages), sum.next(2)) {
        if (!bar_wait(&taken[sum.at], sum.phase ^ 1) || !bar_wait(&full[r.at], r.phase)) { failed = 1; break; }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t wd = tile_desc(smem + r.at * kStageBytes), xd = wd + (kTileN * kStageK >> 4);
#pragma unroll
        for (int j = 0; j < kStageK / 32; ++j) mma<true>(tmem + sum.at * kCols, wd + 2 * j, xd + 2 * j, a.idesc, j > 0);
        mma_commit(&empty[r.at]);
        mma_commit(&sums[sum.at]);
      }
    }
  } else {
    // The tokens' scales of a block, times the weight's, one block ahead: lane
    // l has the tokens l, l + 32 ... .
    constexpr int kEach = (BM + 31) / 32;
    const float *ws = a.w_scale + n0 / kBlockK * a.ldws + first, *xs = a.x_scale + m0 * a.ldxs + first;
    float next[kEach], next_w = 0.0f;
    auto fetch = [&](int b) {
      next_w = ws[b];
#pragma unroll
      for (int e = 0; e < kEach; ++e) next[e] = lane + 32 * e < cols ? xs[(lane + 32 * e) * a.ldxs + b] : 0.0f;
    };
    if (blocks > 0) fetch(0);
#pragma unroll
    for (int j = 0; j < BM; ++j) acc[j] = 0.0f;
    Ring sum;
    for (int b = 0; b < blocks; ++b, sum.next(2)) {
      float *const sc = scales[warp][b & 1];
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (BM >= 32 || lane < BM) sc[lane + 32 * e] = next[e] * next_w;
      if (b + 1 < blocks) fetch(b + 1);
      __syncwarp();
      if (!bar_wait(&sums[sum.at], sum.phase, sum_limit(a.k_blocks))) { failed = 1; break; }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t from = tmem + (static_cast<uint32_t>(warp * 32) << 16) + sum.at * kCols;
#pragma unroll
      for (int c = 0; c < BM; c += 16) {
        if (c >= cols) continue;
        uint32_t v[16];
        tmem_ld16(from + c, v);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(sc + c + j);
          acc[c + j] = fmaf(__uint_as_float(v[j]), f.x, acc[c + j]);
          acc[c + j + 1] = fmaf(__uint_as_float(v[j + 1]), f.y, acc[c + j + 1]);
          acc[c + j + 2] = fmaf(__uint_as_float(v[j + 2]), f.z, acc[c + j + 2]);
          acc[c + j + 3] = fmaf(__uint_as_float(v[j + 3]), f.w, acc[c + j + 3]);
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&taken[sum.at])) : "memory");
    }
  }
  __syncwarp();

  // The tile's tokens are shared out: CTA r joins and writes `share` of them
  // from r * share on.  Every CTA puts its partial sums of a token into the
  // joining CTA's shared memory, [splits][share][kTileN].
  const int share = (cols + a.splits - 1) / a.splits;
  float *joined = reinterpret_cast<float *>(smem + (kOver ? 0 : a.stages * kStageBytes));
  const int64_t n = n0 + 4 * lane;
  const int live = n < a.n ? static_cast<int>(min(int64_t(4), a.n - n)) : 0;
  const bool quad = live == 4 && a.vec;
  float bias[4];
  if (warp < kSumWarps) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float b[1] = {0.0f};
      if (a.bias && j < live) load_any<1>(a.bias, a.bias_dtype, n + j, b);
      bias[j] = b[0];
    }
  }
  if (kOver) cluster_arrive();
  cluster_wait();  // every CTA runs (kOver: and is done with its stages)
  if (warp < kSumWarps) {
    uint32_t owner = 0, to = peer_addr(joined + rank * share * kTileN + threadIdx.x, 0);
    int left = share;  // tokens of the owner's share to come
#pragma unroll
    for (int c = 0; c < BM; c += 16) {
      if (c >= cols) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (c + j >= cols) continue;
        if (left == 0) {
          to = peer_addr(joined + rank * share * kTileN + threadIdx.x, ++owner);
          left = share;
        }
        peer_store(to, acc[c + j]);
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
  auto residual = [&](int c, float (&old)[4]) {
    const int64_t at = (m0 + begin + c) * a.ldr + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) old[j] = 0.0f;
    if (!a.residual) return;
    if (quad) load_any<4>(a.residual, a.y_dtype, at, old);
    else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float o[1] = {0.0f};
        if (j < live) load_any<1>(a.residual, a.y_dtype, at + j, o);
        old[j] = o[0];
      }
    }
  };
  const bool writes = warp < kSumWarps && warp < mine;
  float old[4];
  if (writes) residual(warp, old);
  cluster_wait();
  if (warp == kMmaWarp) {
    // The sums have been read, and with them the MMAs are done (or a wait
    // gave up and had its time).
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kCols));
  }
  if (threadIdx.x == 0 && failed) atomicOr(a.err, kErrProduct);
  if (!writes) return;
#pragma unroll 1
  for (int c = warp; c < mine; c += kSumWarps) {
    float next[4];
    if (c + kSumWarps < mine) residual(c + kSumWarps, next);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float4 f = *reinterpret_cast<const float4 *>(joined + (s * share + c) * kTileN + 4 * lane);
      v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += bias[j];
    if (a.y_dtype == ST_F32) activate<true>(v, a.act);
    else activate<false>(v, a.act);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += old[j], old[j] = next[j];
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

// --------------------------------------------------- block_dense_kernel

// Tile t of the launch: groups of eight token tiles, so that the tiles in
// flight share their operands in L2.
struct TileAt {
  int64_t m0, n0;
};
template <int W>
__device__ __forceinline__ TileAt tile_at(const BlockArgs &a, int t) {
  constexpr int kGroup = 8;
  const int per = kGroup * a.n_tiles, g = t / per, in = t % per;
  const int rows = min(kGroup, a.m_tiles - g * kGroup);
  return {int64_t(g * kGroup + in % rows) * kPairM, int64_t(in / rows) * W};
}

// Issues the read of 32 columns; they are there after tmem_wait32().
__device__ __forceinline__ void tmem_issue32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
                 "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]),
                 "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
                 "=r"(v[30]), "=r"(v[31])
               : "r"(addr));
}
// (The values pass through the wait, so that no use of them is moved before it.)
__device__ __forceinline__ void tmem_wait32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :: "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(smem_addr(src)) : "memory");
}

// W: weight rows of a tile.  kF32: y's type, with an activation (exact_act).
template <int W, bool kF32>
__global__ void __launch_bounds__(kDenseThreads, 1)
block_dense_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap rmap, const __grid_constant__ BlockArgs a) {
  // Narrow tiles' stores would hold up the copies of the next stages (8192 x
  // 14336 x 4096 by tiles of 128: 567 us, 472 from registers).
  const bool tma_y = W > 128 && a.tma_store;
  constexpr int kHalf = W / 2;       // columns of a thread; weight rows of a CTA's stage
  constexpr int kStageBytes = (128 + kHalf) * kStageK;
  // Blocks whose sums TMEM holds: as many as fit (8192 x 14336 x 4096 by tiles of
  // 128: four instead of two 519 -> 481 us).
  constexpr int kBuffers = W <= 128 ? 4 : 2, kBufferColumns = 512 / kBuffers;
  extern __shared__ uint8_t raw_smem[];
  uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sums[kBuffers], taken[kBuffers], residuals[kDenseSumWarps];
  __shared__ uint32_t tmem_base;
  __shared__ int failed;
  __shared__ __align__(16) float biases[kDenseSumWarps][kChunk];
  uint8_t *const tile = smem + a.stages * kStageBytes;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;
  const int tiles = a.m_tiles * a.n_tiles, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      bar_init(&sums[i], 1);
      bar_init(&taken[i], 2 * kDenseSumWarps);
    }
    for (int i = 0; i < kDenseSumWarps; ++i) bar_init(&residuals[i], 1);
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

  if (warp < kDenseSumWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegisters));
    const int quarter = warp & 3, left = (warp >> 2) * kHalf;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + left;
    const uint32_t taken_at = peer_addr(taken, 0);
    // This warp's part of y's tile: chunks of 32 columns, rows of 64 bytes whose
    // 16-byte parts are swizzled as TMA reads them.
    uint8_t *const box = tile + warp * part_bytes(W);
    uint32_t(&turn)[32][17] = *reinterpret_cast<uint32_t(*)[32][17]>(box);
    bool stored = false;
    uint32_t residual_phase = 0;
    // The stores so far have left shared memory.
    auto drain = [&]() {
      if (lane == 0) asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
    };
    Ring sum;
    bool ok = true;
    // Whether the columns can lie in two of the weight's blocks.
    constexpr bool kTwo = kHalf > kBlockK / 2 && kBlockK % kHalf != 0;
    for (int t = pair; t < tiles && ok; t += pairs) {
      const TileAt at = tile_at<W>(a, t);
      const int64_t mw = at.m0 + rank * 128 + quarter * 32, m = mw + lane, first = at.n0 + left;
      const bool row = m < a.m;
      // The scales of a block, read one block ahead: the token's, and the weight
      // block's (kTwo: and those of the next one, for the columns from `edge` on).
      const int edge = kBlockK - static_cast<int>(first % kBlockK);
      const bool two = kTwo && edge < kHalf && first + edge < a.n;
      const float *const xs = a.x_scale + (row ? m : 0) * a.ldxs, *const ws = a.w_scale + (first < a.n ? first / kBlockK : 0) * a.ldws;
      float nx = xs[0], n0 = ws[0], n1 = two ? ws[a.ldws] : 0.0f;
      // The residual's boxes take the place of y's while the sums are formed.
      const int boxes = mw < a.m ? static_cast<int>(max(int64_t(0), min(int64_t(kHalf / kChunk), (a.n - first + kChunk - 1) / kChunk))) : 0;
      if (tma_y && a.residual && boxes > 0) {
        if (stored) drain();
        if (lane == 0) {
          bar_expect(&residuals[warp], boxes * 32 * 64);
          for (int i = 0; i < boxes; ++i)
            tma_load(&rmap, box + i * 32 * 64, &residuals[warp], static_cast<int32_t>(first + i * kChunk), static_cast<int32_t>(mw));
        }
      }
      float acc[kHalf];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) acc[j] = 0.0f;
      for (int b = 0; b < a.k_blocks; ++b, sum.next(kBuffers)) {
        const float s0 = nx * n0, s1 = nx * n1;
        if (b + 1 < a.k_blocks) {
          nx = xs[b + 1], n0 = ws[b + 1];
          if (two) n1 = ws[a.ldws + b + 1];
        }
        if (!bar_wait(&sums[sum.at], sum.phase, sum_limit(a.k_blocks))) { ok = false; break; }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t from = lanes + sum.at * kBufferColumns;
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
          tmem_issue32(from + c, v);
          tmem_wait32(v);
          if (c + 32 >= kHalf) {
            // The buffer is given back as soon as this warp has read its part.
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) peer_arrive(taken_at + 8 * sum.at);
          }
          const float s = kTwo && c >= edge ? s1 : s0;
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(__uint_as_float(v[j]), s, acc[c + j]);
        }
      }
      if (!ok) break;
      if (tma_y) {
        if (boxes > 0 && a.residual) {
          if (!bar_wait(&residuals[warp], residual_phase)) { ok = false; break; }
          residual_phase ^= 1;
        } else if (stored) drain();
      }
#pragma unroll
      for (int c = 0; c < kHalf; c += kChunk) {
        const int64_t n0c = first + c;
        if (n0c >= a.n) break;
        const bool wide = a.vec && n0c + kChunk <= a.n;
        uint32_t old[2][8];
        if (a.residual && !tma_y && a.y_dtype != ST_F32) {
          if (!wide) read_turned(a, mw, n0c, lane, old);
          else if (row) {
#pragma unroll
            for (int i = 0; i < 2; ++i) ld32(static_cast<const uint16_t *>(a.residual) + m * a.ldr + n0c + 16 * i, old[i]);
          }
        }
        float v[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] = acc[c + j];
        if (a.bias) {
          float bl[1] = {0.0f};
          if (n0c + lane < a.n) load_any<1>(a.bias, a.bias_dtype, n0c + lane, bl);
          __syncwarp();
          biases[warp][lane] = bl[0];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < kChunk; j += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(biases[warp] + j);
            v[j] += f.x, v[j + 1] += f.y, v[j + 2] += f.z, v[j + 3] += f.w;
          }
        }
        activate<kF32>(v, a.act);
        if (tma_y) {
          uint8_t *const at_row = box + c * 64 + lane * 64;
          auto part = [&](int i) { return reinterpret_cast<uint4 *>(at_row + ((i ^ (lane >> 1 & 3)) << 4)); };
          if (a.residual) {
            uint32_t o[2][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(&o[i / 2][i % 2 * 4]) = *part(i);
#pragma unroll
            for (int i = 0; i < 2; ++i) add16(o[i], a.y_dtype == ST_BF16, v + 16 * i);
          }
          uint32_t u[16];
          if (a.y_dtype == ST_BF16) {
#pragma unroll
            for (int j = 0; j < 16; ++j) u[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) u[j] = pack_f16(v[2 * j], v[2 * j + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) *part(i) = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0 && mw < a.m) tma_store(&ymap, box + c * 64, static_cast<int32_t>(n0c), static_cast<int32_t>(mw));
        } else if (wide) {
          if (row) {
            if (a.residual && a.y_dtype != ST_F32) {
#pragma unroll
              for (int i = 0; i < 2; ++i) add16(old[i], a.y_dtype == ST_BF16, v + 16 * i);
            } else if (a.residual) add_row32(a.residual, m * a.ldr + n0c, v);
            put_row(a.y, a.y_dtype, m * a.ldy + n0c, v);
          }
        } else if (a.y_dtype == ST_BF16) put_turned<__nv_bfloat16>(turn, a, mw, n0c, lane, old, v);
        else if (a.y_dtype == ST_F16) put_turned<__half>(turn, a, mw, n0c, lane, old, v);
        else put_turned32(turn, a, mw, n0c, lane, v);
      }
      stored = tma_y;
    }
    if (stored && lane == 0) asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok) {  // a residual under way lands before the CTA ends
      if (tma_y && a.residual) bar_wait(&residuals[warp], residual_phase);
      failed = 1;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFeedRegisters));
    if (warp == kDenseCopyWarp) {
      if (elect_one()) {
        // This CTA's tokens and its half of the weight rows; the bytes of both
        // CTAs count on the first one's barriers.
        Ring r;
        const uint32_t bars = peer_addr(full, 0);
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
          const TileAt at = tile_at<W>(a, t);
          const int32_t m = static_cast<int32_t>(at.m0 + rank * 128), n = static_cast<int32_t>(at.n0 + rank * kHalf);
          for (int b = 0; b < a.k_blocks; ++b, r.next(a.stages)) {
            // Before its first use a stage counts as released.
            if (!bar_wait(&empty[r.at], r.phase ^ 1)) { ok = false; break; }
            uint8_t *stage = smem + r.at * kStageBytes;
            if (rank == 0) bar_expect(&full[r.at], 2 * kStageBytes);
            pair_load(&xmap, stage, bars + 8 * r.at, b * kStageK, m);
            pair_load(&wmap, stage + 128 * kStageK, bars + 8 * r.at, b * kStageK, n);
          }
        }
        // The stages in flight are released (or, after a wait that gave up,
        // have had their time) before the CTA ends.
        for (int i = 0; i < a.stages; ++i, r.next(a.stages)) ok &= bar_wait(&empty[r.at], r.phase ^ 1);
        if (!ok) failed = 1;
      }
    } else if (warp == kDenseMmaWarp) {
      if (rank == 0 && elect_one()) {
        Ring r, sum;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
          for (int b = 0; b < a.k_blocks; ++b, r.next(a.stages), sum.next(kBuffers)) {
            if (!bar_wait(&full[r.at], r.phase) || !bar_wait(&taken[sum.at], sum.phase ^ 1)) { ok = false; break; }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint64_t xd = tile_desc(smem + r.at * kStageBytes), wd = xd + (128 * kStageK >> 4);
  #pragma unroll
            for (int j = 0; j < kStageK / 32; ++j) pair_mma<true>(tmem + sum.at * kBufferColumns, xd + 2 * j, wd + 2 * j, a.idesc, j > 0);
            pair_commit(&empty[r.at], 0);
            pair_commit(&sums[sum.at], 0);
          }
        }
        if (!ok) failed = 1;
      }
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

st_status launch_error(const BlockArgs &a, cudaError_t e) {
  return set_error(ST_E_CUDA, "st_block_linear launch (%lld x %lld x %lld): %s: %s", (long long)a.m, (long long)a.n,
                   (long long)a.kbytes, cudaGetErrorName(e), cudaGetErrorString(e));
}

template <int BM>
st_status launch_split(BlockArgs &a, const CUtensorMap &wmap, const CUtensorMap &xmap, int64_t tiles, int dev, cudaStream_t st) {
  constexpr int kStageBytes = (kTileN + BM) * kStageK;
  // About half of the SM's shared memory, so that two CTAs share one.
  constexpr int kJoined = (BM + kMaxSplit) * kTileN * 4, kBudget = 109 * 1024;
  constexpr int kStages = BM == 128 ? 3 : (kBudget - kJoined) / kStageBytes;
  static_assert(kStages >= 3 && kStages <= kMaxStages && (BM < 128 || kJoined <= kStages * kStageBytes), "a ring of stages");
  a.stages = kStages;
  constexpr int smem = kStages * kStageBytes + (BM == 128 ? 0 : kJoined) + 1024;
  constexpr auto kernel = block_split_kernel<BM>;
  cudaError_t e = allow_smem<kernel>(dev, smem);
  if (e == cudaSuccess)
    e = launch(kernel, dim3(static_cast<unsigned>(tiles * a.splits)), kSplitThreads, smem, a.splits, st, wmap, xmap, a);
  return e == cudaSuccess ? ST_OK : launch_error(a, e);
}

template <int W, bool kF32>
st_status launch_dense(BlockArgs &a, const CUtensorMap &xmap, const CUtensorMap &wmap, const CUtensorMap &ymap, const CUtensorMap &rmap, int dev, int sms,
                       cudaStream_t st) {
  constexpr int kStageBytes = (128 + W / 2) * kStageK, kFit = (kDenseSmem - kDenseSumWarps * part_bytes(W)) / kStageBytes;
  constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  a.stages = kStages;
  constexpr int smem = kStages * kStageBytes + kDenseSumWarps * part_bytes(W) + 1024;
  constexpr auto kernel = block_dense_kernel<W, kF32>;
  cudaError_t e = allow_smem<kernel>(dev, smem);
  if (e == cudaSuccess)
    e = launch(kernel, dim3(2u * static_cast<unsigned>(std::min(a.m_tiles * a.n_tiles, sms / 2))), kDenseThreads, smem, 2, st, xmap, wmap, ymap, rmap, a);
  return e == cudaSuccess ? ST_OK : launch_error(a, e);
}

// Rows of 16-bit values, in boxes of 32 x 32.
st_status encode_rows(CUtensorMap *map, const Side &s, int64_t n, const char *op) {
  EncodeFn fn = nullptr;
  const st_status st = encoder(&fn, op);
  if (st != ST_OK) return st;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(s.rows)};
  const cuuint64_t stride[1] = {s.rows == 1 ? static_cast<cuuint64_t>((n * 2 + 15) / 16 * 16) : static_cast<cuuint64_t>(s.pitch)};
  const cuuint32_t box[2] = {kChunk, 32}, step[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<uint8_t *>(s.p), dims, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(ST_E_CUDA, "%s: tensor map of rows of %lld x %lld refused (%d)", op, (long long)s.rows, (long long)n, static_cast<int>(r));
  return ST_OK;
}

int blocks_of(const st_block_linear_args &p) { return static_cast<int>((p.k + kBlockK - 1) / kBlockK); }

}  // namespace

int64_t block_linear_workspace(const st_block_linear_args &p) {
  const int64_t pitch = (p.k + 15) / 16 * 16;
  int64_t bytes = 0;
  if (p.k > 0 && !tma_ok(side_of(p.w, p.ldw, p.n, p.k, 1))) bytes += p.n * pitch;
  if (p.k > 0 && !tma_ok(side_of(p.x, p.ldx, p.m, p.k, 1))) bytes += p.m * pitch;
  return bytes;
}

st_status check_block_linear_form(const st_block_linear_args &p, const st_linear_form &f) {
  const bool dense = f.kernel == ST_LINEAR_DENSE;
  bool ok = (dense || f.kernel == ST_LINEAR_SPLIT) && f.splits >= 1 && f.splits <= (dense ? 1 : kMaxSplit) && !(f.splits & (f.splits - 1));
  ok = ok && (dense ? f.width >= 64 && f.width <= kPairMaxN && f.width % 64 == 0 : f.width == 16 || f.width == 32 || f.width == 64 || f.width == 128);
  if (!ok) return set_error(ST_E_INVAL, "st_block_linear: no kernel %d has tiles of width %d and sums in %d parts", f.kernel, f.width, f.splits);
  if (f.splits > std::max(1, blocks_of(p)) || (dense && p.k == 0))
    return set_error(ST_E_INVAL, "st_block_linear: a sum of %d blocks in %d parts", blocks_of(p), f.splits);
  return ST_OK;
}

// Either kernel's time in us, by what was measured of it, and the least of
// them.  block_split_kernel: 4.5, and 0.33, 0.44 or 0.47 a block of its part of
// the sum for tiles of 16, 32 and 64 tokens, 1.8 times as long for two CTAs an
// SM, and again for each round of those.  (1 x 4096 x 14336 in 1, 2, 4, 8 parts: 39.8, 21.5, 13.7, 13.7; 64
// tokens 53.7, 32.3, 19.2, 16.4; tiles of 128 tokens were slower than two of 64
// or the other kernel.)  block_dense_kernel: 2.5, and a round of tiles 0.1 and
// 0.008 a weight row of a tile to write it, and 0.265, 0.307, 0.43 or 0.487 a
// block by 64, 128, 192 and 256 weight rows (8192 x 14336 x 4096: 828, 472, 440,
// 374; 8192 x 4096 x 1024 77, 54, 53, 46; 256 x 4096 x 4096 12.7, 13.5, 16.8, 18.5).
// Writing takes longer with an activation, and where rows off 32-byte boundaries
// are turned in shared memory, and the longer the wider the tile: less of it lies
// beside the next tile's sums (7178 x 1056 x 528 18.1, 14.8, 15.4, 13.6, with gelu
// 21.8, 20.6, 23.9, 22.2; 7178 x 1053 x 528 26.1, 25.5, 28.7, 26.9, with gelu 31.2,
// 31.4, 41.4, 41.1).  It counts among these widths alone: block_split_kernel's
// own writing takes longer too, and is not in its time (5549 x 7887 x 99 with gelu
// 122, and 285 by block_split_kernel).
st_linear_form choose_block_linear_form(const st_block_linear_args &p, int sms) {
  const int k_blocks = blocks_of(p);
  const int tokens = p.m <= 16 ? 16 : p.m <= 32 ? 32 : 64;
  const int64_t tiles = (p.m + tokens - 1) / tokens * ((p.n + kTileN - 1) / kTileN);
  st_linear_form best{ST_LINEAR_SPLIT, tokens, 1};
  double least = 0;
  for (int splits = 1; splits <= kMaxSplit; splits *= 2) {
    if (splits > 1 && k_blocks < 2 * splits) break;
    const int64_t ctas = tiles * splits;
    const double rounds = static_cast<double>((ctas + 2 * sms - 1) / (2 * sms)), block = tokens == 16 ? 0.33 : tokens == 32 ? 0.44 : 0.47;
    const double us = rounds * (4.5 + (k_blocks + splits - 1) / splits * block * (ctas <= sms ? 1.0 : 1.8));
    if (splits == 1 || us < least) best.splits = splits, least = us;
  }
  if (p.m <= 16 || p.k == 0) return best;
  static constexpr double kBlock[] = {0.265, 0.307, 0.43, 0.487};
  const int64_t item = static_cast<int64_t>(st_dtype_size(p.y_dtype));
  auto off = [&](int64_t to) {
    auto one = [&](const void *q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % to || (p.m > 1 && ld * item % to); };
    return one(p.y, p.ldy) || (p.residual && one(p.residual, p.ldr));
  };
  const double act = p.act == ST_ACT_GELU ? 1.0 : p.act == ST_ACT_SILU || p.act == ST_ACT_GELU_TANH ? 0.4 : 0.0;
  const bool tma = item == 2 && !off(16), turned = off(32);
  double wide = 0;  // of block_dense_kernel's widths, what writing takes counted
  int width = 0;
  for (int w = kPairMaxN; w >= 64; w -= 64) {
    const int64_t dense = (p.m + kPairM - 1) / kPairM * ((p.n + w - 1) / w);
    const double write = 0.008 + act * (0.006 + 0.00005 * w) + (turned && !(tma && w > 128) ? 0.015 + 0.00005 * w : 0.0);
    const double rounds = static_cast<double>((dense + sms / 2 - 1) / (sms / 2)), us = 2.5 + rounds * (0.1 + 0.008 * w + k_blocks * kBlock[w / 64 - 1]);
    const double whole = us + rounds * (write - 0.008) * w;
    if (us < least) best.kernel = ST_LINEAR_DENSE, least = us;
    if (!width || whole < wide) width = w, wide = whole;
  }
  if (best.kernel == ST_LINEAR_DENSE) best.width = width, best.splits = 1;
  return best;
}

st_status launch_block_linear(const st_block_linear_args &p, const st_linear_form *form, void *stream) {
  const char *op = "st_block_linear";
  BlockArgs a{};
  a.m = p.m; a.n = p.n; a.kbytes = p.k;
  a.act = p.act; a.y_dtype = p.y_dtype; a.bias_dtype = p.bias_dtype;
  a.bias = p.bias; a.residual = p.residual; a.y = p.y;
  a.ldr = p.ldr; a.ldy = p.ldy;
  a.x_scale = p.x_scale; a.w_scale = p.w_scale; a.ldxs = p.ldxs; a.ldws = p.ldws;
  a.x = side_of(p.x, p.ldx, p.m, p.k, 1);
  a.w = side_of(p.w, p.ldw, p.n, p.k, 1);
  int dev = 0, sms = 0;
  st_status s = product_device(&dev, &sms, &a.err);
  if (s == ST_OK) s = align_rows(&a.w, &a.x, p.k, p.workspace, stream, op);
  if (s != ST_OK) return s;
  a.k_blocks = blocks_of(p);
  const st_linear_form f = form ? *form : choose_block_linear_form(p, sms);
  const bool dense = f.kernel == ST_LINEAR_DENSE;
  const int64_t rows = dense ? kPairM : f.width, columns = dense ? f.width : kTileN;
  const int64_t m_tiles = (p.m + rows - 1) / rows, n_tiles = (p.n + columns - 1) / columns, tiles = m_tiles * n_tiles;
  if (2 * tiles * f.splits > 0x7fffffff)
    return set_error(ST_E_INVAL, "%s: %lld x %lld needs more tiles than one launch has", op, (long long)p.m, (long long)p.n);
  a.m_tiles = static_cast<int>(m_tiles);
  a.n_tiles = static_cast<int>(n_tiles);
  a.splits = f.splits;
  const int64_t out = static_cast<int64_t>(st_dtype_size(p.y_dtype)), to = dense ? 32 : 4 * out;
  auto one = [&](const void *q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % to == 0 && ld * out % to == 0; };
  a.vec = one(p.y, p.ldy) && (!p.residual || one(p.residual, p.ldr));
  // Instruction descriptor: binary32 accumulators; formats of A and B, both
  // K-major; rows and columns of one MMA.
  const uint32_t e5m2 = p.w_dtype == ST_F8_E5M2;
  auto idesc = [](uint32_t fa, uint32_t fb, uint32_t r, uint32_t c) {
    return (1u << 4) | (fa << 7) | (fb << 10) | ((c / 8) << 17) | ((r / 16) << 24);
  };
  CUtensorMap wmap{}, xmap{}, ymap{}, rmap{};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dense) {
    a.idesc = idesc(0, e5m2, kPairM, f.width);
    s = encode(&xmap, a.x, p.k, 1, 128, op);
    if (s == ST_OK) s = encode(&wmap, a.w, p.k, 1, f.width / 2, op);
    // y and the residual in boxes of a warp's 32 rows and 32 columns.
    const Side y = side_of(p.y, p.ldy, p.m, p.n, 2), res = side_of(p.residual, p.ldr, p.m, p.n, 2);
    a.tma_store = out == 2 && tma_ok(y) && (!p.residual || tma_ok(res));
    if (s == ST_OK && a.tma_store) s = encode_rows(&ymap, y, p.n, op);
    if (s == ST_OK && a.tma_store && p.residual) s = encode_rows(&rmap, res, p.n, op);
    if (s != ST_OK) return s;
    auto run = [&](auto w) {
      constexpr int W = decltype(w)::value;
      return exact_act(a.act, a.y_dtype) ? launch_dense<W, true>(a, xmap, wmap, ymap, rmap, dev, sms, st) : launch_dense<W, false>(a, xmap, wmap, ymap, rmap, dev, sms, st);
    };
    switch (f.width) {
      case 64: return run(std::integral_constant<int, 64>{});
      case 128: return run(std::integral_constant<int, 128>{});
      case 192: return run(std::integral_constant<int, 192>{});
      default: return run(std::integral_constant<int, 256>{});
    }
  }
  a.idesc = idesc(e5m2, 0, kTileN, f.width);
  if (p.k > 0) {
    s = encode(&wmap, a.w, p.k, 1, kTileN, op);
    // Fewer tokens than the MMA's columns: only they are copied (what the other
    // columns hold reaches no sum that is read).
    a.x_box = p.m < f.width ? static_cast<int>(p.m) : f.width;
    if (s == ST_OK) s = encode(&xmap, a.x, p.k, 1, a.x_box, op);
    if (s != ST_OK) return s;
  }
  switch (f.width) {
    case 16: return launch_split<16>(a, wmap, xmap, tiles, dev, st);
    case 32: return launch_split<32>(a, wmap, xmap, tiles, dev, st);
    case 64: return launch_split<64>(a, wmap, xmap, tiles, dev, st);
    default: return launch_split<128>(a, wmap, xmap, tiles, dev, st);
  }
}

}  // namespace stmat
