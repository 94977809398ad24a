// st_moe.cu -- a mixture-of-experts layer for a few tokens, from its router to
// the sum of its experts, for GB300 (sm_103a).
//
//   l = x router^T,  s = softmax(l) or sigmoid(l)
//   chosen: the top_k experts with the largest s + router_bias,  p = factor s / (sum of the chosen s, or 1)
//   y = sum over the chosen e of  p_e down_e (act(gate_e x) (up_e x))  + residual
//
// A few tokens choose most of a batch's experts once or twice, so the layer is
// as long as the chosen experts' weights take to come from HBM.  Four launches,
// each of which starts while the one before it ends:
//   logits_kernel  the router's product, and x in the columns (below) that the
//                  tensor core takes
//   route_kernel   the choice, its weights, and the list of the chosen experts
//                  with their tokens ("slots", ordered by expert and token)
//   up_kernel      h = p act(gate x) (up x): 128 rows of one expert's gate and
//                  up, of its tokens alone
//   down_kernel    128 rows of y: every chosen expert's down in turn
// As in st_linear's split_kernel the weight's rows are the MMA's rows, the
// tokens its columns (as many as the expert has, in steps of 16), and the sum
// is split over the CTAs of a cluster that join in rank order: no atomics, the
// same bits on every run.
//
// Eight-bit experts.  The weights go to the tensor core as they are stored, and
// it multiplies eight bits with eight; x and h are not rounded to eight bits
// for that.  A run of 128 values is divided by a power of two to below 256 and
// written as two or three columns of E4M3 codes, each the rounding error of
// those before it: c0, 2^-4 c1, 2^-9 c2.  Four significant bits a column hold a
// BF16's eight in two, an F16's eleven (and 12 of h, a binary32) in three, down
// to 2^-21 of the run's largest.  The extra columns cost no time while the
// weights come from HBM.  Sixteen-bit experts take x as it is and h as two
// columns of their type.
//
// The choice turns on the last digits of the logits: they are summed in two
// binary32 words with the rounding errors kept (Knuth's two-sum).
//
// Bound: HBM, behind the router.  64 tokens, 6 of 64 experts 4096 -> 1408 in 8
// bits: 182 us, 135 by the bytes of the 52 experts chosen (logits 17, the choice
// 9, up and down at 5.6 and 4.9 TB/s, each alone and cold); 7 tokens, 2 of 8
// experts 4096 -> 14336 BF16 368 and 419 (7 and 8 experts: 368, 421).  One token,
// 8 of 128 experts 2048 -> 768 in 8 bits: 24.4 us (5.7), four kernels' latencies
// of 4 to 6 each, overlapped.  Bringing the experts' weights into L2 while the
// router runs was slower in all of seven cases (its reads wait behind them: 8
// tokens, 4 of 8 experts 2048 -> 1024 BF16 32.5 -> 37.8 us).
#include "st_tensor_device.h"

namespace stmat {
namespace {

constexpr int kRows = 128;           // weight rows of a tile: the MMA's M
constexpr int kRun = 128;            // values with a common scale
constexpr int kMaxTokens = ST_MOE_MAX_TOKENS;
static_assert(kMaxTokens <= 64, "bits of an expert's mask");
constexpr int kMaxTop = 32;
constexpr int kMaxExperts = 1024;
constexpr int kMaxSplit = 8;         // portable cluster size
constexpr int kSumWarps = 4;         // one per 32 TMEM lanes
constexpr int kMmaWarp = 4, kCopyWarp = 5, kScaleWarp = 6, kThreads = 224;
constexpr int kMaxBuffers = 8;       // stages' sums that TMEM holds
constexpr int kScaleSlots = 8, kScaleRun = 4;  // stages whose scales are ready, and brought in together
constexpr int kLogitWarps = 8, kLogitTokens = 4;
constexpr int kRouteWarps = 8;       // tokens of a CTA of route_kernel
constexpr int kGroup = 32;           // tokens of an expert that are multiplied at a time
// Stages and sums: under half of an SM's shared memory, and at most half of its
// TMEM, so that one CTA's start and end lie beside another's copies, and no CTA
// of a cluster waits for TMEM that another cluster's holds.
constexpr int kSmem = 106 * 1024;

// What route_kernel finds.  Arrays of as many entries as can be needed.
struct Lists {
  int *count;         // groups: chosen experts with up to kGroup of their tokens
  int *most;          // tokens of the largest group
  int *expert;        // [i]: the i-th group's expert, ascending
  int *first;         // [i]: its first slot; [count]: the number of slots
  int *token;         // [slot]
  float *weight;      // [slot]
};

struct MoeArgs {
  const void *x, *router, *residual;
  const float *bias;
  void *y;
  int *chosen;
  float *weights;
  int64_t ldx, ld_router, ldr, ldy;
  int tokens, hidden, inter, experts, top_k;
  int sigmoid, normalize;
  float factor;
  st_act act;
  st_dtype x_dtype, router_dtype, y_dtype, w_dtype;
  int has_up;
  // Block scales of gate, up and down (8 bits): [expert, row block, block].
  const float *scale[3];
  int64_t scale_expert[3], scale_row[3], scale_col[3];
  // Workspace.
  double *logits, *keys;  // keys: what is compared, where that is not the logit
  uint8_t *xq, *hq;       // columns of x and h, rows of pitch bytes
  float *xs, *hs;         // their runs' scales (x: 8 bits alone)
  int64_t x_pitch, h_pitch;
  int h_blocks, in_blocks, h_runs, in_runs;  // stages and runs of hidden and inter
  Lists list;
  uint32_t idesc;         // without the number of columns
  int splits, tiles;
  uint32_t *err;
};

// ------------------------------------------------------------ columns

// The power of two that takes a run's largest magnitude below 2^below (8 bits:
// 256, BF16: 4, F16: 2^15); NaN where that is not finite.
__device__ __forceinline__ float run_scale(float top, int below) {
  if (!(top < __int_as_float(0x7f800000))) return __int_as_float(0x7fffffff);
  const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - (below - 1), 1);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}
__device__ __forceinline__ float exact_inverse(float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); }

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half *>(&h));
}
// The codes of v's columns.
template <int C>
__device__ __forceinline__ void columns8(float v, uint32_t (&c)[C]) {
  constexpr float kUp[3] = {1.0f, 16.0f, 512.0f};
#pragma unroll
  for (int i = 0; i < C; ++i) {
    c[i] = pack_e4m3(v * kUp[i], 0.0f) & 0xff;
    v -= e4m3_value(c[i]) * (1.0f / kUp[i]);
  }
}

__device__ __forceinline__ float warp_top(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = max_nan(v, __shfl_xor_sync(~0u, v, d));
  return v;
}

// ------------------------------------------------------- logits_kernel

// A block has an expert and up to four tokens; its warps share the sum.
template <class X, class R>
__device__ __forceinline__ void logits(const MoeArgs &a, int expert, int t0) {
  __shared__ float part[kLogitWarps][kLogitTokens][2];
  const int live = min(kLogitTokens, a.tokens - t0), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kThreadsHere = 32 * kLogitWarps;
  const R *const w = static_cast<const R *>(a.router) + expert * a.ld_router;
  // Fewer than four: the last one again, so that all four's steps interleave.
  const X *x[kLogitTokens];
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t) x[t] = static_cast<const X *>(a.x) + (t0 + min(t, live - 1)) * a.ldx;
  Two sum[kLogitTokens];
  auto step = [&](int t, float xv, float wv) {
    const float p = __fmul_rn(xv, wv);
    // Two 16-bit numbers' product is exact.
    if (sizeof(R) == 4) sum[t].lo += fmaf(xv, wv, -p);
    sum[t].add(p);
  };
  constexpr int V = sizeof(R) == 4 ? 4 : 8;
  const bool wide = a.hidden % V == 0 && a.ldx % V == 0 && a.ld_router % V == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.router) % 16 == 0;
  if (wide) {
    for (int c = threadIdx.x * V; c < a.hidden; c += kThreadsHere * V) {
      float wv[V], xv[kLogitTokens][V];
      unpack(*reinterpret_cast<const Raw<R, V> *>(w + c), wv);
#pragma unroll
      for (int t = 0; t < kLogitTokens; ++t) unpack(*reinterpret_cast<const Raw<X, V> *>(x[t] + c), xv[t]);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int t = 0; t < kLogitTokens; ++t) step(t, xv[t][i], wv[i]);
    }
  } else {
    for (int c = threadIdx.x; c < a.hidden; c += kThreadsHere) {
      const float wv = to_float(w[c]);
#pragma unroll
      for (int t = 0; t < kLogitTokens; ++t) step(t, to_float(x[t][c]), wv);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1)
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t) {
      const float hi = __shfl_xor_sync(~0u, sum[t].hi, d), lo = __shfl_xor_sync(~0u, sum[t].lo, d);
      sum[t].lo += lo;
      sum[t].add(hi);
    }
  Two mine;  // lane t's: token t's
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t)
    if (lane == t) mine = sum[t];
  if (lane < live) part[warp][lane][0] = mine.hi, part[warp][lane][1] = mine.lo;
  __syncthreads();
  if (threadIdx.x < live) {
    mine = Two{};
#pragma unroll
    for (int i = 0; i < kLogitWarps; ++i) {
      mine.lo += part[i][lane][1];
      mine.add(part[i][lane][0]);
    }
    // Where the sum has left binary32's range its error has no meaning.
    const double l = isfinite(mine.hi) ? static_cast<double>(mine.hi) + mine.lo : mine.hi;
    const int64_t at = int64_t(t0 + lane) * a.experts + expert;
    a.logits[at] = l;
    if (a.bias && a.sigmoid) a.keys[at] = 1.0 / (1.0 + exp(-l)) + a.bias[expert];
  }
}

// A block has a token's columns.
template <class X>
__device__ __forceinline__ void x_columns(const MoeArgs &a, int token) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const X *const x = static_cast<const X *>(a.x) + token * a.ldx;
  if (a.w_dtype == ST_BF16 || a.w_dtype == ST_F16) {
    X *const to = reinterpret_cast<X *>(a.xq + token * a.x_pitch);
    if (a.hidden % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0) {
      for (int c = threadIdx.x * 8; c < a.hidden; c += 256 * kLogitWarps)
        *reinterpret_cast<uint4 *>(to + c) = *reinterpret_cast<const uint4 *>(x + c);
    } else {
#pragma unroll 8
      for (int c = threadIdx.x; c < a.hidden; c += 32 * kLogitWarps) to[c] = x[c];
    }
    return;
  }
  constexpr int C = std::is_same<X, __half>::value ? 3 : 2;
  uint8_t *const to = a.xq + int64_t(token) * C * a.x_pitch;
  for (int run = warp; run < a.h_runs; run += kLogitWarps) {
    const int c0 = run * kRun + 4 * lane;
    float v[4], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = c0 + i < a.hidden ? to_float(x[c0 + i]) : 0.0f;
      top = max_nan(top, fabsf(v[i]));
    }
    const float s = run_scale(warp_top(top), 8), inv = exact_inverse(s);
    if (lane == 0) a.xs[token * a.h_runs + run] = s;
    uint32_t packed[C] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c[C];
      columns8<C>(v[i] * inv, c);
#pragma unroll
      for (int j = 0; j < C; ++j) packed[j] |= c[j] << (8 * i);
    }
    if (c0 < a.x_pitch) {
#pragma unroll
      for (int j = 0; j < C; ++j) *reinterpret_cast<uint32_t *>(to + j * a.x_pitch + c0) = packed[j];
    }
  }
}

// A block for a token's columns, or an expert and four tokens.
__global__ void __launch_bounds__(32 * kLogitWarps) logits_kernel(const __grid_constant__ MoeArgs a) {
  wait_for_previous();
  let_next_start();
  const int groups = (a.tokens + kLogitTokens - 1) / kLogitTokens, item = blockIdx.x - a.tokens;
  auto with_x = [&](auto &&f) {
    if (a.x_dtype == ST_BF16) f(__nv_bfloat16{});
    else f(__half{});
  };
  with_x([&](auto x) {
    if (item < 0) x_columns<decltype(x)>(a, blockIdx.x);
    else with_type(a.router_dtype, [&](auto r) { logits<decltype(x), decltype(r)>(a, item / groups, item % groups * kLogitTokens); });
  });
}

// -------------------------------------------------------- route_kernel

// A whole number in the order of the choice: by size, a NaN above all.  (The
// SM compares 64 whole numbers in the time of one pair of binary64 ones: 1 of
// 128 experts' choice of 8 took 19 us so.)
__device__ __forceinline__ int64_t order(double v) {
  int64_t b = __double_as_longlong(v);
  if ((b & 0x7fffffffffffffffll) > 0x7ff0000000000000ll) return 0x7fffffffffffffffll;
  if (b == static_cast<int64_t>(0x8000000000000000ull)) b = 0;  // -0
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double ordered(int64_t k) { return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll)); }

// A warp chooses for a token; kPer of the experts a lane (expert 32 j + lane).
// kScores: what is compared is softmax's scores and a bias.
template <int kPer, bool kScores>
__device__ __forceinline__ void choose_experts(const MoeArgs &a, int token, int lane, int *chosen, float *weight) {
  constexpr int64_t kNone = static_cast<int64_t>(0x8000000000000000ull);  // below every number
  const double *const l = a.logits + int64_t(token) * a.experts;
  int64_t key[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) key[j] = 32 * j + lane < a.experts ? order(l[32 * j + lane]) : kNone;
  // Softmax: relative to the largest logit.
  double top = 0.0;
  float all = 0.0f;
  if (!a.sigmoid) {
    int64_t best = kNone;
#pragma unroll
    for (int j = 0; j < kPer; ++j) best = max(best, key[j]);
#pragma unroll
    for (int d = 16; d; d >>= 1) best = max(best, static_cast<int64_t>(__shfl_xor_sync(~0u, best, d)));
    top = ordered(best);
    if (!a.normalize) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (32 * j + lane < a.experts) all += expf(static_cast<float>(ordered(key[j]) - top));
#pragma unroll
      for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(~0u, all, d);
    }
    if constexpr (kScores) {
      double sum = 0.0, s[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (32 * j + lane < a.experts) s[j] = exp(ordered(key[j]) - top), sum += s[j];
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (32 * j + lane < a.experts) key[j] = order(s[j] / sum + a.bias[32 * j + lane]);
    }
  } else if (a.bias) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (32 * j + lane < a.experts) key[j] = order(a.keys[int64_t(token) * a.experts + 32 * j + lane]);
  }
  // Taken experts leave with a key of none; an expert's own is above it.
  int mine = 0;
  for (int i = 0; i < a.top_k; ++i) {
    int64_t best = kNone;
    int best_e = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (key[j] > best) best = key[j], best_e = 32 * j + lane;
    // The warp's largest key by its two halves, then the lowest index.
    const int high = static_cast<int>(best >> 32), top_high = __reduce_max_sync(~0u, high);
    const uint32_t low = high == top_high ? static_cast<uint32_t>(best) : 0, top_low = __reduce_max_sync(~0u, low);
    best_e = __reduce_min_sync(~0u, high == top_high && static_cast<uint32_t>(best) == top_low ? best_e : 0x7fffffff);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (32 * j + lane == best_e) key[j] = kNone;
    if (lane == i) mine = best_e;
  }
  // Lane i has the i-th chosen expert.  Scores that their own sum divides are
  // relative to the chosen ones' largest (a bias may have chosen experts, and
  // sigmoid's scores may all lie, where exp leaves binary32's range).
  const double v = lane < a.top_k ? l[mine] : __longlong_as_double(0xfff0000000000000ll);
  if (a.normalize && (kScores || a.sigmoid)) {
    float most = static_cast<float>(v);
#pragma unroll
    for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
    top = a.sigmoid ? fminf(most, 0.0f) : most;
  }
  float s = 0.0f;
  if (lane < a.top_k) {
    s = expf(static_cast<float>(v - top));
    if (a.sigmoid) s = v < 0.0 ? s / (1.0f + expf(static_cast<float>(v))) : 1.0f / (1.0f + expf(static_cast<float>(-v)));
  }
  float sum = s;
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  const float p = a.factor * (a.normalize ? s / sum : a.sigmoid ? s : s / all);
  if (lane < a.top_k) {
    chosen[lane] = mine;
    weight[lane] = p;
    if (a.chosen) a.chosen[int64_t(token) * a.top_k + lane] = mine;
    if (a.weights) a.weights[int64_t(token) * a.top_k + lane] = p;
  }
}

// The CTAs of one cluster have eight tokens each; each places its own in the
// lists, and the first lists the groups.
template <int kPer, bool kScores>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ MoeArgs a) {
  __shared__ struct {
    uint64_t mask[kMaxExperts];             // tokens of an expert
    int slots[kMaxExperts], totals[kRouteWarps][3];
    int chosen[kRouteWarps][kMaxTop];
    float weight[kRouteWarps][kMaxTop];
  } s;
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, token = cta * kRouteWarps + warp;
  constexpr int kThreadsHere = 32 * kRouteWarps;
  for (int e = threadIdx.x; e < a.experts; e += kThreadsHere) s.mask[e] = 0;
  wait_for_previous();
  let_next_start();
  if (token < a.tokens) choose_experts<kPer, kScores>(a, token, lane, s.chosen[warp], s.weight[warp]);
  cluster_arrive();
  __syncthreads();
  cluster_wait();
  // Every CTA reads all CTAs' choices, so that each can place its own.
  for (int i = threadIdx.x; i < a.tokens * a.top_k; i += kThreadsHere) {
    const int t = i / a.top_k;
    int e;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(e) : "r"(peer_addr(&s.chosen[t % kRouteWarps][i % a.top_k], t / kRouteWarps)) : "memory");
    atomicOr(reinterpret_cast<unsigned long long *>(&s.mask[e]), 1ull << t);
  }
  cluster_arrive();
  __syncthreads();
  // Slots, and places in the list: running counts over the experts, kEach a
  // thread.
  const int each = (a.experts + kThreadsHere - 1) / kThreadsHere;
  int all_n = 0, all_used = 0, most = 0;
  for (int i = 0; i < each; ++i) {
    const int e = threadIdx.x * each + i, n = e < a.experts ? __popcll(s.mask[e]) : 0;
    all_n += n, all_used += (n + kGroup - 1) / kGroup;
    most = max(most, min(n, kGroup));
  }
  int before_n = all_n, before_used = all_used;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, before_n, d), u = __shfl_up_sync(~0u, before_used, d);
    if (lane >= d) before_n += o, before_used += u;
  }
  most = __reduce_max_sync(~0u, most);
  if (lane == 31) s.totals[warp][0] = before_n, s.totals[warp][1] = before_used, s.totals[warp][2] = most;
  __syncthreads();
  before_n -= all_n, before_used -= all_used;
#pragma unroll
  for (int w = 0; w < kRouteWarps; ++w) {
    if (w < warp) before_n += s.totals[w][0], before_used += s.totals[w][1];
    most = max(most, s.totals[w][2]);
  }
  for (int i = 0; i < each; ++i) {
    const int e = threadIdx.x * each + i;
    if (e >= a.experts) break;
    const int n = __popcll(s.mask[e]);
    s.slots[e] = before_n;
    for (int g = 0; g < n; g += kGroup, ++before_used) {
      if (cta > 0) continue;
      a.list.expert[before_used] = e;
      a.list.first[before_used] = before_n + g;
    }
    before_n += n;
  }
  if (cta == 0 && threadIdx.x == kThreadsHere - 1) {
    *a.list.count = before_used;
    *a.list.most = most;
    a.list.first[before_used] = before_n;
  }
  __syncthreads();
  if (token < a.tokens && lane < a.top_k) {
    const int e = s.chosen[warp][lane], slot = s.slots[e] + __popcll(s.mask[e] & ((1ull << token) - 1));
    a.list.token[slot] = token;
    a.list.weight[slot] = s.weight[warp][lane];
  }
  cluster_wait();  // no CTA ends while another reads its choices
}

// -------------------------------------------------- the experts' products

__device__ __forceinline__ void tma_load3(const CUtensorMap *map, void *dst, uint64_t *bar, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)) : "memory");
}

// The TMEM columns of eight tokens, C each.
template <int C>
__device__ __forceinline__ void read_tokens(uint32_t addr, uint32_t (&v)[8 * C]) {
  if constexpr (C != 2)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "r"(addr));
  if constexpr (C != 1) {
    constexpr int o = C == 3 ? 8 : 0;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7]),
                   "=r"(v[o + 8]), "=r"(v[o + 9]), "=r"(v[o + 10]), "=r"(v[o + 11]), "=r"(v[o + 12]), "=r"(v[o + 13]), "=r"(v[o + 14]), "=r"(v[o + 15])
                 : "r"(addr + o));
  }
  if constexpr (C == 1)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]) :: "memory");
  if constexpr (C > 1)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]),
                   "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]) :: "memory");
  if constexpr (C == 3)
    asm volatile("" : "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]) :: "memory");
}
// A token's sum of its columns' sums.
template <int C, bool kEight>
__device__ __forceinline__ float of_columns(const uint32_t (&v)[8 * C], int t) {
  float s = __uint_as_float(v[C * t]);
  if constexpr (C > 1) s = fmaf(__uint_as_float(v[C * t + 1]), kEight ? 0x1p-4f : 1.0f, s);
  if constexpr (C > 2) s = fmaf(__uint_as_float(v[C * t + 2]), 0x1p-9f, s);
  return s;
}

__host__ __device__ constexpr int round16(int n) { return (n + 15) / 16 * 16; }
__host__ __device__ constexpr int buffers_of(int columns) { return 256 / columns < kMaxBuffers ? 256 / columns : kMaxBuffers; }
__host__ __device__ constexpr int tmem_columns(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512; }

// What both kernels' CTAs have.
struct Pipe {
  uint64_t full[kMaxStages], empty[kMaxStages], sums[kMaxBuffers], taken[kMaxBuffers], ready[kScaleSlots], used[kScaleSlots];
  uint32_t tmem;
  int failed;
};
__device__ __forceinline__ void pipe_start(Pipe &p, int warp, int columns) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      bar_init(&p.full[i], 1);
      bar_init(&p.empty[i], 1);
    }
    for (int i = 0; i < kMaxBuffers; ++i) {
      bar_init(&p.sums[i], 1);
      bar_init(&p.taken[i], kSumWarps);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      bar_init(&p.ready[i], 1);
      bar_init(&p.used[i], kSumWarps);
    }
    p.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&p.tmem)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void pipe_end(Pipe &p, int warp, int columns, uint32_t *err) {
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(p.tmem), "r"(columns));
  if (threadIdx.x == 0 && p.failed) atomicOr(err, kErrProduct);
}
// The four summing warps.
__device__ __forceinline__ void sum_warps_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Adds eight tokens' sums of a stage, times their scales.
template <int C, bool kEight, int BT>
__device__ __forceinline__ void add_tokens(float (&to)[BT], int t, uint32_t from, const float *scale) {
  uint32_t v[8 * C];
  read_tokens<C>(from + t * C, v);
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 1.0f;
  if (scale) {
    *reinterpret_cast<float4 *>(f) = *reinterpret_cast<const float4 *>(scale + t);
    *reinterpret_cast<float4 *>(f + 4) = *reinterpret_cast<const float4 *>(scale + t + 4);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) to[t + j] = fmaf(of_columns<C, kEight>(v, j), f[j], to[t + j]);
}

// h of 128 rows of one group.  BT: tokens that a group may have; C: columns of
// an x.  Gate's and up's sums of a stage lie side by side in TMEM.
template <int BT, int C, bool kEight>
__global__ void __launch_bounds__(kThreads) up_kernel(const __grid_constant__ CUtensorMap gate, const __grid_constant__ CUtensorMap up,
                                                      const __grid_constant__ CUtensorMap xmap, const __grid_constant__ MoeArgs a) {
  // Sixteen bits have no scales: their sums stay in TMEM to the end.
  constexpr int kN = round16(BT * C), kBuffers = kEight ? buffers_of(2 * kN) : 1, kColumns = tmem_columns(kBuffers * 2 * kN);
  constexpr int kStep = kEight ? kStageK : kStageK / 2, kOutColumns = kEight ? 3 : 2;
  static_assert(kColumns <= 256 && 2 * (2 * kRows + kN) * kStageK <= kSmem && (BT + kMaxSplit) * 2 * kRows * 4 <= kSmem, "half of an SM");
  extern __shared__ uint8_t raw_smem[];
  uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  __shared__ Pipe pipe;
  __shared__ __align__(16) float scales[kScaleSlots][2][BT];
  __shared__ float tops[kSumWarps][BT], weights[BT];
  __shared__ int tokens[BT];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x % a.splits;
  const int item = blockIdx.x / a.splits, which = item / a.tiles, n0 = item % a.tiles * kRows;
  const int first = static_cast<int>(int64_t(a.h_blocks) * rank / a.splits);
  const int blocks = static_cast<int>(int64_t(a.h_blocks) * (rank + 1) / a.splits) - first;
  pipe_start(pipe, warp, kColumns);
  wait_for_previous();
  let_next_start();
  if (which >= *a.list.count) {  // every CTA of the cluster
    pipe_end(pipe, warp, kColumns, a.err);
    return;
  }
  const int expert = a.list.expert[which], slot0 = a.list.first[which], count = a.list.first[which + 1] - slot0;
  const int columns = round16(count * C), stage_bytes = (2 * kRows + columns) * kStageK;
  const int stages = min(kMaxStages, kSmem / stage_bytes);
  const uint32_t tmem = pipe.tmem;

  Ring r;
  float g[BT], u[BT];
  if (warp == kCopyWarp) {
    if (lane < count) tokens[lane] = a.list.token[slot0 + lane];
    __syncwarp();
    if (elect_one()) {
      bool ok = true;
      const uint32_t bytes = (a.has_up ? 2 : 1) * kRows * kStageK + count * C * kStageK;
      for (int i = 0; i < blocks; ++i, r.next(stages)) {
        // Before its first use a stage counts as released.
        if (!bar_wait(&pipe.empty[r.at], r.phase ^ 1)) { ok = false; break; }
        uint8_t *stage = smem + r.at * stage_bytes;
        const int k = (first + i) * kStep;
        bar_expect(&pipe.full[r.at], bytes);
        tma_load3(&gate, stage, &pipe.full[r.at], k, n0, expert);
        if (a.has_up) tma_load3(&up, stage + kRows * kStageK, &pipe.full[r.at], k, n0, expert);
        for (int t = 0; t < count; ++t) tma_load(&xmap, stage + (2 * kRows + t * C) * kStageK, &pipe.full[r.at], k, tokens[t] * C);
      }
      // The stages in flight are released (or, after a wait that gave up,
      // have had their time) before the CTA ends.
      for (int i = 0; i < stages; ++i, r.next(stages)) ok &= bar_wait(&pipe.empty[r.at], r.phase ^ 1);
      if (!ok) pipe.failed = 1;
    }
  } else if (warp == kMmaWarp) {
    if (elect_one()) {
      Ring sum;
      const uint32_t idesc = a.idesc | static_cast<uint32_t>(columns / 8) << 17;
      for (int i = 0; i < blocks; ++i, r.next(stages), sum.next(kBuffers)) {
        if ((kEight && !bar_wait(&pipe.taken[sum.at], sum.phase ^ 1)) || !bar_wait(&pipe.full[r.at], r.phase)) { pipe.failed = 1; break; }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t gd = tile_desc(smem + r.at * stage_bytes), ud = gd + (kRows * kStageK >> 4), xd = ud + (kRows * kStageK >> 4);
        const uint32_t d = tmem + sum.at * 2 * kN;
        const bool add = !kEight && i > 0;
#pragma unroll
        for (int j = 0; j < kStageK / 32; ++j) mma<kEight>(d, gd + 2 * j, xd + 2 * j, idesc, add || j > 0);
        if (a.has_up) {
#pragma unroll
          for (int j = 0; j < kStageK / 32; ++j) mma<kEight>(d + kN, ud + 2 * j, xd + 2 * j, idesc, add || j > 0);
        }
        mma_commit(&pipe.empty[r.at]);
        if (kEight || i == blocks - 1) mma_commit(&pipe.sums[sum.at]);
      }
    }
  } else if (warp == kScaleWarp) {
    // Scales of several stages at a time, well ahead: lane l has the token l.
    // (Brought one stage ahead by the summing warps they took L2's latency a
    // stage.)
    if (kEight) {
      const int block_row = n0 / kRun, token = lane < count ? a.list.token[slot0 + lane] : 0;
      const float *const gs = a.scale[0] + expert * a.scale_expert[0] + block_row * a.scale_row[0];
      const float *const us = a.scale[1] + expert * a.scale_expert[1] + block_row * a.scale_row[1];
      const float *const xs = a.xs + token * a.h_runs;
      bool ok = true;
      float gv[2][kScaleRun], uv[2][kScaleRun], xv[2][kScaleRun];
      auto fetch = [&](int at, int i0) {
#pragma unroll
        for (int i = 0; i < kScaleRun; ++i) {
          const int b = first + min(i0 + i, blocks - 1);
          gv[at][i] = gs[b * a.scale_col[0]];
          uv[at][i] = a.has_up ? us[b * a.scale_col[1]] : 0.0f;
          xv[at][i] = lane < count ? xs[b] : 0.0f;
        }
      };
      auto put = [&](int at, int i0) {
#pragma unroll
        for (int i = 0; i < kScaleRun; ++i) {
          if (i0 + i >= blocks || !ok) continue;
          if (!bar_wait(&pipe.used[r.at], r.phase ^ 1, sum_limit(a.h_blocks))) { ok = false; continue; }
          if (lane < BT) scales[r.at][0][lane] = xv[at][i] * gv[at][i], scales[r.at][1][lane] = xv[at][i] * uv[at][i];
          __syncwarp();
          if (lane == 0) local_arrive(&pipe.ready[r.at]);
          r.next(kScaleSlots);
        }
      };
      fetch(0, 0);
      for (int i0 = 0; i0 < blocks && ok; i0 += 2 * kScaleRun) {
        fetch(1, i0 + kScaleRun);
        put(0, i0);
        fetch(0, i0 + 2 * kScaleRun);
        put(1, i0 + kScaleRun);
      }
      if (!ok) pipe.failed = 1;
    }
  } else {
    if (threadIdx.x < count) weights[threadIdx.x] = a.list.weight[slot0 + threadIdx.x];
#pragma unroll
    for (int t = 0; t < BT; ++t) g[t] = u[t] = 0.0f;
    Ring sum;
    for (int b = 0; b < (kEight ? blocks : 1); ++b, sum.next(kBuffers), r.next(kScaleSlots)) {
      if ((kEight && !bar_wait(&pipe.ready[r.at], r.phase, sum_limit(a.h_blocks))) || !bar_wait(&pipe.sums[sum.at], sum.phase, sum_limit(a.h_blocks))) {
        pipe.failed = 1;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t from = tmem + (static_cast<uint32_t>(warp * 32) << 16) + sum.at * 2 * kN;
#pragma unroll
      for (int t = 0; t < BT; t += 8) {
        if (t >= count) continue;
        add_tokens<C, kEight>(g, t, from, kEight ? scales[r.at][0] : nullptr);
        if (a.has_up) add_tokens<C, kEight>(u, t, from + kN, kEight ? scales[r.at][1] : nullptr);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        local_arrive(&pipe.taken[sum.at]);
        if (kEight) local_arrive(&pipe.used[r.at]);
      }
    }
  }
  __syncwarp();

  // h and its columns.  The CTAs of a cluster share the tokens out: CTA r joins
  // and writes `share` of them from r * share on, whose partial sums every CTA
  // puts into its shared memory, [splits][share][gate, up][kRows] over the
  // stages.
  const int share = (count + a.splits - 1) / a.splits;
  const int begin = static_cast<int>(rank) * share, own = max(0, min(share, count - begin));
  float *const joined = reinterpret_cast<float *>(smem);
  const int row = threadIdx.x, n = n0 + row;
  if (a.splits > 1) {
    cluster_arrive();
    cluster_wait();  // every CTA is done with its stages
  } else if (warp < kSumWarps) {
    sum_warps_sync();  // the last MMAs are done, and with them the stages
  }
  if (warp < kSumWarps) {
    uint32_t owner = 0, to = peer_addr(joined + rank * share * 2 * kRows + row, 0);
    int left = share;
#pragma unroll
    for (int t = 0; t < BT; ++t) {
      if (t >= count) continue;
      if (left == 0) {
        to = peer_addr(joined + rank * share * 2 * kRows + row, ++owner);
        left = share;
      }
      peer_store(to, g[t]);
      peer_store(to + kRows * 4, u[t]);
      to += 2 * kRows * 4;
      --left;
    }
  }
  if (a.splits > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (warp < kSumWarps) {
    for (int t = 0; t < own; ++t) {
      float v[1] = {0.0f}, uv = 0.0f;
      for (int s = 0; s < a.splits; ++s) {
        const float *from = joined + (s * share + t) * 2 * kRows + row;
        v[0] += from[0], uv += from[kRows];
      }
      activate<false>(v, a.act);
      if (a.has_up) v[0] *= uv;
      v[0] *= weights[begin + t];
      joined[t * 2 * kRows + row] = v[0];
      const float top = warp_top(fabsf(v[0]));
      if (lane == 0) tops[warp][t] = top;
    }
    sum_warps_sync();
#pragma unroll 2
    for (int t = 0; t < own; ++t) {
      const int64_t slot = slot0 + begin + t;
      float top = 0.0f;
#pragma unroll
      for (int w = 0; w < kSumWarps; ++w) top = max_nan(top, tops[w][t]);
      const float s = run_scale(top, kEight ? 8 : a.w_dtype == ST_BF16 ? 2 : 15), v = joined[t * 2 * kRows + row] * exact_inverse(s);
      if (row == 0) a.hs[slot * a.in_runs + n0 / kRun] = s;
      if (n >= a.inter) continue;
      uint8_t *const to = a.hq + slot * kOutColumns * a.h_pitch;
      if constexpr (kEight) {
        uint32_t c[kOutColumns];
        columns8<kOutColumns>(v, c);
#pragma unroll
        for (int i = 0; i < kOutColumns; ++i) to[i * a.h_pitch + n] = static_cast<uint8_t>(c[i]);
      } else {
        const float hi[1] = {a.w_dtype == ST_BF16 ? to_float(__float2bfloat16_rn(v)) : to_float(__float2half_rn(v))}, lo[1] = {v - hi[0]};
        store_any<1>(to, a.w_dtype, n, hi);
        store_any<1>(to + a.h_pitch, a.w_dtype, n, lo);
      }
    }
  }
  pipe_end(pipe, warp, kColumns, a.err);
}

// A walk over (group, run of its sum), with the next group's entries read ahead.
struct Walk {
  int groups, which, run, expert, slot0, count, next_expert, next_end;
  __device__ __forceinline__ void begin(const MoeArgs &a, int n, int64_t at) {
    groups = n;
    which = static_cast<int>(at / a.in_runs);
    run = static_cast<int>(at % a.in_runs);
    expert = slot0 = count = next_expert = next_end = 0;
    if (which >= groups) return;
    next_expert = __ldcg(&a.list.expert[which]);
    slot0 = __ldcg(&a.list.first[which]);
    next_end = __ldcg(&a.list.first[which + 1]);
    enter(a);
  }
  __device__ __forceinline__ void enter(const MoeArgs &a) {
    expert = next_expert;
    slot0 += count;
    count = next_end - slot0;
    if (which + 1 >= groups) return;
    next_expert = __ldcg(&a.list.expert[which + 1]);
    next_end = __ldcg(&a.list.first[which + 2]);
  }
  // Whether the next run is another group's.
  __device__ __forceinline__ bool next(const MoeArgs &a) {
    if (++run < a.in_runs) return false;
    run = 0;
    if (++which < groups) enter(a);
    return true;
  }
};

// 128 rows of y.  The runs of all groups, one after the other, are shared out
// over the cluster's CTAs; each keeps the tokens' sums of its part in shared
// memory.  A run is one stage of eight bits, two of sixteen (one, where a last
// run is short), whose sums are read out together.
template <int BT, bool kEight>
__global__ void __launch_bounds__(kThreads) down_kernel(const __grid_constant__ CUtensorMap down, const __grid_constant__ CUtensorMap hmap,
                                                        const __grid_constant__ MoeArgs a) {
  constexpr int C = kEight ? 3 : 2, kN = round16(BT * C), kBuffers = buffers_of(kN), kColumns = tmem_columns(kBuffers * kN);
  constexpr int kStep = kEight ? kStageK : kStageK / 2, kPerRun = kRun / kStep;
  static_assert(kColumns <= 256 && 2 * (kRows + kN) * kStageK + kMaxTokens * kRows * 4 <= kSmem, "half of an SM");
  extern __shared__ uint8_t raw_smem[];
  uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  __shared__ Pipe pipe;
  __shared__ __align__(16) float scales[kScaleSlots][BT];
  float *const total = reinterpret_cast<float *>(smem);  // [token][kRows]
  uint8_t *const ring = smem + (a.tokens * kRows * 4 + 1023) / 1024 * 1024;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x % a.splits;
  const int n0 = static_cast<int>(blockIdx.x / a.splits) * kRows;
  pipe_start(pipe, warp, kColumns);
  // The lists are the router's, which has ended: up_kernel's CTAs waited for
  // that before any let this kernel start.  So the first stages' weights are
  // under way before h is there.  (Read from L2: an L1 may hold an earlier
  // call's lists until this kernel's own wait.)
  const int groups = __ldcg(a.list.count);
  const int64_t all = int64_t(groups) * a.in_runs, begin = all * rank / a.splits, end = all * (rank + 1) / a.splits;
  const int runs = static_cast<int>(end - begin);
  // Stages before run r of all.
  auto stages_before = [&](int64_t r) { return r / a.in_runs * a.in_blocks + r % a.in_runs * kPerRun; };
  const int64_t blocks = stages_before(end) - stages_before(begin);
  const uint32_t limit = sum_limit(static_cast<int>(min(all * kPerRun, int64_t(0x7fffffff))));
  const int stage_bytes = (kRows + round16(__ldcg(a.list.most) * C)) * kStageK;
  const int stages = min(kMaxStages, static_cast<int>(kSmem - (ring - smem)) / stage_bytes);
  const uint32_t tmem = pipe.tmem;
  auto stages_of = [&](const Walk &w) { return min(kPerRun, a.in_blocks - w.run * kPerRun); };
  Walk at;
  at.begin(a, groups, begin);
  Ring r;
  if (warp == kCopyWarp) {
    if (elect_one()) {
      bool ok = true;
      auto weights = [&](const Walk &w, int part, int slot) {
        bar_expect(&pipe.full[slot], (kRows + round16(w.count * C)) * kStageK);
        tma_load3(&down, ring + slot * stage_bytes, &pipe.full[slot], (w.run * kPerRun + part) * kStep, n0, w.expert);
      };
      Walk early = at;
      for (int i = 0, part = 0; i < min(int64_t(stages), blocks); ++i) {
        weights(early, part, i);
        if (++part == stages_of(early)) part = 0, early.next(a);
      }
      wait_for_previous();
      let_next_start();
      int part = 0;
      for (int64_t i = 0; i < blocks; ++i, r.next(stages)) {
        if (i >= stages) {
          if (!bar_wait(&pipe.empty[r.at], r.phase ^ 1)) { ok = false; break; }
          weights(at, part, r.at);
        }
        uint8_t *const h = ring + r.at * stage_bytes + kRows * kStageK;
        const int columns = round16(at.count * C);
        for (int c = 0; c < columns; c += 16)
          tma_load(&hmap, h + c * kStageK, &pipe.full[r.at], (at.run * kPerRun + part) * kStep, at.slot0 * C + c);
        if (++part == stages_of(at)) part = 0, at.next(a);
      }
      // The stages in flight are released (or, after a wait that gave up,
      // have had their time) before the CTA ends.
      for (int i = 0; i < stages; ++i, r.next(stages)) ok &= bar_wait(&pipe.empty[r.at], r.phase ^ 1);
      if (!ok) pipe.failed = 1;
    }
  } else if (warp == kMmaWarp) {
    if (elect_one()) {
      Ring sum;
      bool ok = true;
      wait_for_previous();
      for (int i = 0; i < runs && ok; ++i, sum.next(kBuffers), at.next(a)) {
        if (!bar_wait(&pipe.taken[sum.at], sum.phase ^ 1)) { ok = false; break; }
        const uint32_t idesc = a.idesc | static_cast<uint32_t>(round16(at.count * C) / 8) << 17;
        const int parts = stages_of(at);
        for (int part = 0; part < parts; ++part, r.next(stages)) {
          if (!bar_wait(&pipe.full[r.at], r.phase)) { ok = false; break; }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t wd = tile_desc(ring + r.at * stage_bytes), hd = wd + (kRows * kStageK >> 4);
#pragma unroll
          for (int j = 0; j < kStageK / 32; ++j) mma<kEight>(tmem + sum.at * kN, wd + 2 * j, hd + 2 * j, idesc, part > 0 || j > 0);
          mma_commit(&pipe.empty[r.at]);
        }
        mma_commit(&pipe.sums[sum.at]);
      }
      if (!ok) pipe.failed = 1;
    }
  } else if (warp == kScaleWarp) {
    // As in up_kernel: lane l has the group's slot l.
    wait_for_previous();
    let_next_start();
    bool ok = true;
    float w[2][kScaleRun], h[2][kScaleRun];
    auto fetch = [&](float(&wv)[kScaleRun], float(&hv)[kScaleRun], int i0) {
#pragma unroll
      for (int i = 0; i < kScaleRun; ++i) {
        if (i0 + i >= runs) continue;
        wv[i] = kEight ? a.scale[2][at.expert * a.scale_expert[2] + n0 / kRun * a.scale_row[2] + at.run * a.scale_col[2]] : 1.0f;
        hv[i] = lane < at.count ? a.hs[int64_t(at.slot0 + lane) * a.in_runs + at.run] : 0.0f;
        at.next(a);
      }
    };
    auto put = [&](const float(&wv)[kScaleRun], const float(&hv)[kScaleRun], int i0) {
#pragma unroll
      for (int i = 0; i < kScaleRun; ++i) {
        if (i0 + i >= runs || !ok) continue;
        if (!bar_wait(&pipe.used[r.at], r.phase ^ 1, limit)) { ok = false; continue; }
        if (lane < BT) scales[r.at][lane] = wv[i] * hv[i];
        __syncwarp();
        if (lane == 0) local_arrive(&pipe.ready[r.at]);
        r.next(kScaleSlots);
      }
    };
    fetch(w[0], h[0], 0);
    for (int i0 = 0; i0 < runs && ok; i0 += 2 * kScaleRun) {
      fetch(w[1], h[1], i0 + kScaleRun);
      put(w[0], h[0], i0);
      fetch(w[0], h[0], i0 + 2 * kScaleRun);
      put(w[1], h[1], i0 + kScaleRun);
    }
    if (!ok) pipe.failed = 1;
  } else {
    const int row = threadIdx.x;
    for (int t = 0; t < a.tokens; ++t) total[t * kRows + row] = 0.0f;
    wait_for_previous();
    let_next_start();
    // Lane l has the token of the group's slot l.
    int token = runs > 0 && lane < at.count ? a.list.token[at.slot0 + lane] : 0;
    float acc[BT];
#pragma unroll
    for (int t = 0; t < BT; ++t) acc[t] = 0.0f;
    Ring sum;
    for (int b = 0; b < runs; ++b, sum.next(kBuffers), r.next(kScaleSlots)) {
      if (!bar_wait(&pipe.ready[r.at], r.phase, limit) || !bar_wait(&pipe.sums[sum.at], sum.phase, limit)) { pipe.failed = 1; break; }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t from = tmem + (static_cast<uint32_t>(warp * 32) << 16) + sum.at * kN;
#pragma unroll
      for (int t = 0; t < BT; t += 8)
        if (t < at.count) add_tokens<C, kEight>(acc, t, from, scales[r.at]);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        local_arrive(&pipe.taken[sum.at]);
        local_arrive(&pipe.used[r.at]);
      }
      if (at.run == a.in_runs - 1 || b == runs - 1) {
        // The group's part of its tokens' sums.  (Columns that are no token's
        // have had anything added.)
#pragma unroll
        for (int t = 0; t < BT; t += 8) {
          if (t >= at.count) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int to = __shfl_sync(~0u, token, t + j);
            if (t + j < at.count) total[to * kRows + row] += acc[t + j];
            acc[t + j] = 0.0f;
          }
        }
      }
      if (at.next(a) && b + 1 < runs) token = lane < at.count ? a.list.token[at.slot0 + lane] : 0;
    }
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  const int n = n0 + static_cast<int>(threadIdx.x);
  if (warp < kSumWarps) {
    const int share = (a.tokens + a.splits - 1) / a.splits, t0 = static_cast<int>(rank) * share, t1 = min(a.tokens, t0 + share);
    // A token's residual and parts are under way while the one before is summed.
    float part[kMaxSplit], next[kMaxSplit], old[1] = {0.0f}, next_old[1] = {0.0f};
    auto read = [&](int t, float(&to)[kMaxSplit], float(&res)[1]) {
      if (a.residual && n < a.hidden) load_any<1>(a.residual, a.y_dtype, t * a.ldr + n, res);
#pragma unroll
      for (int s = 0; s < kMaxSplit; ++s)
        if (s < a.splits) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(to[s]) : "r"(peer_addr(total + t * kRows + threadIdx.x, s)) : "memory");
    };
    if (t0 < t1) read(t0, part, old);
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) read(t + 1, next, next_old);
      float v[1] = {0.0f};
#pragma unroll
      for (int s = 0; s < kMaxSplit; ++s) {
        if (s < a.splits) v[0] += part[s];
        part[s] = next[s];
      }
      v[0] += old[0];
      old[0] = next_old[0];
      if (n < a.hidden) store_any<1>(a.y, a.y_dtype, t * a.ldy + n, v);
    }
  }
  cluster_arrive();
  cluster_wait();
  pipe_end(pipe, warp, kColumns, a.err);
}

// ------------------------------------------------------------------- host

int item_of(const st_moe_args &p) { return p.w_dtype == ST_BF16 || p.w_dtype == ST_F16 ? 2 : 1; }
int x_columns_of(const st_moe_args &p) { return item_of(p) == 2 ? 1 : p.x_dtype == ST_F16 ? 3 : 2; }
int h_columns_of(const st_moe_args &p) { return item_of(p) == 2 ? 2 : 3; }

// The workspace's parts, at multiples of 256 bytes.
struct Space {
  int64_t at = 0;
  int64_t take(int64_t bytes) {
    const int64_t from = at;
    at += (bytes + 255) / 256 * 256;
    return from;
  }
};
// Groups at most: chosen experts, and those with more than kGroup tokens again.
int64_t groups_of(const st_moe_args &p) { return std::min(p.tokens * p.top_k, p.experts + p.tokens * p.top_k / (kGroup + 1)); }
int64_t lay_out(const st_moe_args &p, MoeArgs *a) {
  const int item = item_of(p);
  const int64_t slots = p.tokens * p.top_k, most = groups_of(p);
  const int64_t x_pitch = (p.hidden * item + 15) / 16 * 16, h_pitch = (p.inter * item + 15) / 16 * 16;
  const int64_t h_runs = (p.hidden + kRun - 1) / kRun, in_runs = (p.inter + kRun - 1) / kRun;
  Space s;
  const int64_t logits = s.take(8 * p.tokens * p.experts), keys = s.take(p.router_bias && p.score == ST_MOE_SIGMOID ? 8 * p.tokens * p.experts : 0);
  const int64_t xq = s.take(p.tokens * x_columns_of(p) * x_pitch), xs = s.take(item == 1 ? 4 * p.tokens * h_runs : 0);
  const int64_t hq = s.take(slots * h_columns_of(p) * h_pitch), hs = s.take(4 * slots * in_runs);
  const int64_t count = s.take(8), expert = s.take(4 * most), first = s.take(4 * (most + 1)), token = s.take(4 * slots), weight = s.take(4 * slots);
  if (a) {
    uint8_t *const base = static_cast<uint8_t *>(p.workspace);
    a->logits = reinterpret_cast<double *>(base + logits);
    a->keys = reinterpret_cast<double *>(base + keys);
    a->xq = base + xq;
    a->xs = reinterpret_cast<float *>(base + xs);
    a->hq = base + hq;
    a->hs = reinterpret_cast<float *>(base + hs);
    a->x_pitch = x_pitch, a->h_pitch = h_pitch;
    a->h_runs = static_cast<int>(h_runs), a->in_runs = static_cast<int>(in_runs);
    a->list = {reinterpret_cast<int *>(base + count), reinterpret_cast<int *>(base + count) + 1, reinterpret_cast<int *>(base + expert), reinterpret_cast<int *>(base + first),
               reinterpret_cast<int *>(base + token), reinterpret_cast<float *>(base + weight)};
  }
  return s.at;
}

// All experts' [rows, k] matrices, read in boxes of 128 rows and 128 bytes of k.
st_status encode_experts(CUtensorMap *map, const void *p, int64_t k, int64_t rows, int64_t experts, int64_t ld, int64_t step, int item, const char *op) {
  EncodeFn fn = nullptr;
  const st_status st = encoder(&fn, op);
  if (st != ST_OK) return st;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(experts)};
  const int64_t row = rows == 1 ? (k * item + 15) / 16 * 16 : ld * item;
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(experts == 1 ? (rows * row + 15) / 16 * 16 : step * item)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kStageK / item), kRows, 1}, each[3] = {1, 1, 1};
  const CUresult r = fn(map, item == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(p), dims, stride, box,
                        each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(ST_E_CUDA, "%s: tensor map of %lld x %lld x %lld refused (%d)", op, (long long)experts, (long long)rows, (long long)k, static_cast<int>(r));
  return ST_OK;
}

struct Maps {
  CUtensorMap gate, up, down, x, h;
};

template <class... P, class... A>
st_status start(const char *what, void (*kernel)(P...), int64_t blocks, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st, const A &...args) {
  const cudaError_t e = launch(kernel, dim3(static_cast<unsigned>(blocks)), threads, smem, cluster, st, args...);
  return e == cudaSuccess ? ST_OK : set_error(ST_E_CUDA, "st_moe: %s launch: %s: %s", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Parts of the sum: as many as let all CTAs run at a time, each with at least
// four stages.
int parts(int64_t items, int64_t blocks, int most, int64_t room) {
  int splits = 1;
  while (splits < most && items * splits * 2 <= room && blocks / (splits * 2) >= 4) splits *= 2;
  return splits;
}

template <int BT, int C, bool kEight>
st_status launch_up(MoeArgs a, const Maps &maps, int64_t groups, int dev, int sms, cudaStream_t st) {
  a.tiles = (a.inter + kRows - 1) / kRows;
  a.splits = parts(groups * a.tiles, a.h_blocks, kMaxSplit, 2 * sms);
  constexpr auto kernel = up_kernel<BT, C, kEight>;
  const cudaError_t e = allow_smem<kernel>(dev, kSmem + 1024);
  if (e != cudaSuccess) return set_error(ST_E_CUDA, "st_moe: %s", cudaGetErrorString(e));
  return start("up", kernel, groups * a.tiles * a.splits, kThreads, kSmem + 1024, a.splits, st, maps.gate, maps.up, maps.x, a);
}

template <int BT, bool kEight>
st_status launch_down(MoeArgs a, const Maps &maps, int dev, int sms, cudaStream_t st) {
  a.tiles = (a.hidden + kRows - 1) / kRows;
  a.splits = parts(a.tiles, int64_t(a.top_k) * a.in_blocks, kMaxSplit, 2 * sms);
  constexpr auto kernel = down_kernel<BT, kEight>;
  const cudaError_t e = allow_smem<kernel>(dev, kSmem + 1024);
  if (e != cudaSuccess) return set_error(ST_E_CUDA, "st_moe: %s", cudaGetErrorString(e));
  return start("down", kernel, int64_t(a.tiles) * a.splits, kThreads, kSmem + 1024, a.splits, st, maps.down, maps.h, a);
}

template <int BT>
st_status launch_products(const MoeArgs &a, const Maps &maps, int columns, int64_t groups, int dev, int sms, cudaStream_t st) {
  st_status s;
  if (columns == 1) s = launch_up<BT, 1, false>(a, maps, groups, dev, sms, st);
  else if (columns == 2) s = launch_up<BT, 2, true>(a, maps, groups, dev, sms, st);
  else s = launch_up<BT, 3, true>(a, maps, groups, dev, sms, st);
  if (s != ST_OK) return s;
  return columns == 1 ? launch_down<BT, false>(a, maps, dev, sms, st) : launch_down<BT, true>(a, maps, dev, sms, st);
}

}  // namespace

int64_t moe_workspace(const st_moe_args &p) { return lay_out(p, nullptr); }

st_status launch_moe(const st_moe_args &p, void *stream) {
  const char *op = "st_moe";
  MoeArgs a{};
  a.x = p.x; a.router = p.router; a.residual = p.residual; a.bias = p.router_bias; a.y = p.y;
  a.chosen = p.chosen; a.weights = p.weights;
  a.ldx = p.ldx; a.ld_router = p.ld_router; a.ldr = p.ldr; a.ldy = p.ldy;
  a.tokens = static_cast<int>(p.tokens); a.hidden = static_cast<int>(p.hidden); a.inter = static_cast<int>(p.inter);
  a.experts = static_cast<int>(p.experts); a.top_k = static_cast<int>(p.top_k);
  a.sigmoid = p.score == ST_MOE_SIGMOID; a.normalize = p.normalize != 0; a.factor = p.factor;
  a.act = p.act; a.x_dtype = p.x_dtype; a.router_dtype = p.router_dtype; a.y_dtype = p.y_dtype; a.w_dtype = p.w_dtype;
  a.has_up = p.up.w != nullptr;
  const st_moe_weight *const weights[3] = {&p.gate, &p.up, &p.down};
  for (int i = 0; i < 3; ++i) {
    a.scale[i] = weights[i]->scale;
    a.scale_expert[i] = weights[i]->scale_expert;
    a.scale_row[i] = weights[i]->scale_row;
    a.scale_col[i] = weights[i]->scale_col;
  }
  const int item = item_of(p), xc = x_columns_of(p), hc = h_columns_of(p), step = kStageK / item;
  lay_out(p, &a);
  a.h_blocks = (a.hidden + step - 1) / step;
  a.in_blocks = (a.inter + step - 1) / step;
  // Instruction descriptor: binary32 accumulators; formats of A (the weight)
  // and B, both K-major; 128 rows.
  const uint32_t fa = item == 2 ? p.w_dtype == ST_BF16 : p.w_dtype == ST_F8_E5M2, fb = item == 2 ? p.w_dtype == ST_BF16 : 0;
  a.idesc = (1u << 4) | (fa << 7) | (fb << 10) | ((kRows / 16) << 24);
  int dev = 0, sms = 0;
  st_status s = product_device(&dev, &sms, &a.err);
  Maps maps{};
  if (s == ST_OK) s = encode_experts(&maps.gate, p.gate.w, p.hidden, p.inter, p.experts, p.gate.ld, p.gate.expert, item, op);
  if (s == ST_OK && a.has_up) s = encode_experts(&maps.up, p.up.w, p.hidden, p.inter, p.experts, p.up.ld, p.up.expert, item, op);
  if (s == ST_OK) s = encode_experts(&maps.down, p.down.w, p.inter, p.hidden, p.experts, p.down.ld, p.down.expert, item, op);
  const int64_t slots = p.tokens * p.top_k;
  if (s == ST_OK) s = encode(&maps.x, Side{a.xq, a.x_pitch, 0, p.tokens * xc}, p.hidden, item, xc, op);
  if (s == ST_OK) s = encode(&maps.h, Side{a.hq, a.h_pitch, 0, slots * hc}, p.inter, item, 16, op);
  if (s != ST_OK) return s;
  const int64_t groups = groups_of(p);
  if (groups * ((p.inter + kRows - 1) / kRows) * kMaxSplit > 0x7fffffff) return set_error(ST_E_INVAL, "%s: more tiles than one launch has", op);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool scores = p.router_bias && !a.sigmoid;
  auto pick = [&](auto of) {  // kernels by the experts a lane has, and what is compared
    constexpr std::true_type yes;
    constexpr std::false_type no;
    using std::integral_constant;
    if (p.experts <= 64) return scores ? of(integral_constant<int, 2>{}, yes) : of(integral_constant<int, 2>{}, no);
    if (p.experts <= 256) return scores ? of(integral_constant<int, 8>{}, yes) : of(integral_constant<int, 8>{}, no);
    return scores ? of(integral_constant<int, 32>{}, yes) : of(integral_constant<int, 32>{}, no);
  };
  s = start("router", logits_kernel, p.tokens + p.experts * ((p.tokens + kLogitTokens - 1) / kLogitTokens), 32 * kLogitWarps, 0, 1, st, a);
  if (s != ST_OK) return s;
  const unsigned ctas = p.tokens <= 8 ? 1 : p.tokens <= 16 ? 2 : p.tokens <= 32 ? 4 : 8;
  s = start("route", pick([](auto per, auto sc) { return &route_kernel<decltype(per)::value, decltype(sc)::value>; }), ctas, 32 * kRouteWarps, 0, ctas, st, a);
  if (s != ST_OK) return s;
  return p.tokens <= 8    ? launch_products<8>(a, maps, xc, groups, dev, sms, st)
         : p.tokens <= 16 ? launch_products<16>(a, maps, xc, groups, dev, sms, st)
                          : launch_products<32>(a, maps, xc, groups, dev, sms, st);
}

}  // namespace stmat
