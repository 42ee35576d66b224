// select_blocks.cu -- the cache blocks that matter most to a query: per sequence
// and KV head, the blocks whose keys can score highest.
//
// A block's score for a group of query heads is the largest bound of q_i . k over
// the block's keys,
//     s_t = max_{i in group} sum_d max(q_id lo_td, q_id hi_td)
//         = max_i (q_i^+ . hi_t + q_i^- . lo_t),   q^+ = max(q, 0), q^- = min(q, 0),
// two products with the bounds as they lie in memory.  The first and the last
// blocks are taken always, the others by score, in the order of the scores in 64
// bits (ties: the earlier block; NaN as +inf), so that the list does not depend on
// how a kernel sums.
//
// Bound by the bounds' bytes (2 x 256 B a block and KV head, 16-bit), so the
// scores run on mma.sync in 32 bits: a warp takes 8 blocks (n) against up to 16
// query heads a tile (m); a lane's 16-byte pieces of a bounds row are the B
// fragments as they are (the k index is permuted, the same for q).  Such a score
// is off by at most
//     E = 2^-16 max_i sum_d |q_id| max_td |bound_td|:
// four chains of four products of 16 terms, each term off by at most 2^-23 of the
// chain's sum of magnitudes (4 x 17 x 2^-23), and their sum.  The second kernel, a
// CTA to each sequence and KV head, finds the cut v (cut.cuh); blocks
// within 2 E of it, usually none but the cut itself, are scored again in 64 bits.
// Doing all in 64 bits would take 40 times the floor here: 0.6 T products a second.
#include <algorithm>

#include "cut.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr int kScoreWarps = 4;
constexpr int kQStride = 320;  // bytes of a 128-value row in shared memory: rows two banks' groups apart
constexpr float kInf = __builtin_huge_valf();
constexpr float kError = 1.52587890625e-05f;  // 2^-16

// q^+ and q^- of a pair: the halves whose sign bit is clear / set, else 0.
DECATTN_DEV void by_sign(uint32_t w, uint32_t& plus, uint32_t& minus) {
  const uint32_t negative = byte_perm(w, 0u, 0xbb99u);  // (each half's sign, 16 times)
  plus = w & ~negative;
  minus = w & negative;
}

template <bool kF8, bool kBF16, int kTiles>
__global__ void __launch_bounds__(kScoreWarps * 32, kTiles == 1 ? 8 : 1) block_scores_kernel(const SelectParams p) {
  constexpr bool kMmaBF16 = kBF16 && !kF8;
  __shared__ __align__(16) uint8_t qs[kTiles * 16 * kQStride];
  __shared__ float mag[kTiles * 16], part[kScoreWarps];
  launch_dependents();
  const int j = blockIdx.y, b = blockIdx.z, G = p.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int64_t bj = static_cast<int64_t>(b) * p.h_kv + j;
  const int n = p.seq_lens[b];
  const int blocks = n > 0 && n <= p.max_seq_len ? ((n - 1) >> p.log2_block_size) + 1 : 0;
  // Nothing to choose (or a bad length, which the second kernel reports).
  if (blocks <= p.count) return;

  // q of the group (rows past it zero); over 8 bits as fp16, a bf16 query times the
  // power of two that brings the group's largest value to 2^14 .. 2^15 (the
  // scores of the pair (b, j) then all carry that factor; what falls below fp16's
  // smallest step is 2^-38 of that value).
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + bj * G * kHeadDim;
  for (int r = warp; r < kTiles * 16; r += kScoreWarps) {
    uint2 w = make_uint2(0u, 0u);
    if (r < G) w = *reinterpret_cast<const uint2*>(q + r * kHeadDim + lane * 4);
    const float2 x = unpack2<kBF16>(w.x), y = unpack2<kBF16>(w.y);
    float sum = fabsf(x.x) + fabsf(x.y) + fabsf(y.x) + fabsf(y.y);
    float most = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    *reinterpret_cast<uint2*>(qs + r * kQStride + lane * 8) = w;
    if (lane == 0) mag[r] = kF8 && kBF16 ? most : sum;
  }
  __syncthreads();
  float alpha = 1.f, q1 = 0.f;
  if constexpr (kF8 && kBF16) {
    float most = 0.f;
    for (int r = 0; r < G; ++r) most = fmaxf(most, mag[r]);
    const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;  // 128: infinite
    const int k = e >= 128 ? 0 : min(14 - e, 126);
    alpha = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    __syncthreads();
    for (int r = warp; r < G; r += kScoreWarps) {
      uint2* at = reinterpret_cast<uint2*>(qs + r * kQStride + lane * 8);
      const float2 x = unpack2<true>(at->x), y = unpack2<true>(at->y);
      *at = make_uint2(pack2<false>(x.x * alpha, x.y * alpha), pack2<false>(y.x * alpha, y.y * alpha));
      float sum = alpha * (fabsf(x.x) + fabsf(x.y) + fabsf(y.x) + fabsf(y.y));
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) mag[r] = sum;
    }
    __syncthreads();
  }
  for (int r = 0; r < G; ++r) q1 = fmaxf(q1, mag[r]);

  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  constexpr int kRowBytes = kF8 ? kHeadDim : 2 * kHeadDim;
  constexpr int kPieces = kRowBytes / 64;  // 16-byte pieces a lane has of a row
  const int64_t half = static_cast<int64_t>(p.h_kv) * kRowBytes;  // from a block's lo to its hi
  const uint8_t* bounds = static_cast<const uint8_t*>(p.bounds) + j * kRowBytes + t4 * 16;
  const uint8_t* qrow = qs + g * kQStride;
  float* scores = p.scores + bj * p.score_stride;
  const int tiles = (blocks + 7) / 8, step = gridDim.x * kScoreWarps;
  uint32_t widest = 0;  // the largest magnitude seen, packed
  int tile = blockIdx.x * kScoreWarps + warp;
  // (-1 for blocks that are taken always: their bounds are not looked at.)
  auto block_of = [&](int tl) {
    const int t = tl * 8 + g;
    return t >= p.first && t < blocks - p.last ? bt[t] : -1;
  };
  int id = tile < tiles ? block_of(tile) : -1;
  for (; tile < tiles; tile += step) {
    uint4 lo[kPieces], hi[kPieces];
    const bool there = id >= 0 && id < p.num_blocks;  // (a bad id: the second kernel reports it)
    const uint8_t* at = bounds + static_cast<int64_t>(id) * 2 * half;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
      if (there) {
        lo[i] = *reinterpret_cast<const uint4*>(at + i * 64);
        hi[i] = *reinterpret_cast<const uint4*>(at + half + i * 64);
      }
    }
    id = tile + step < tiles ? block_of(tile + step) : -1;
    float best[2] = {-kInf, -kInf};  // columns 2 t4 and 2 t4 + 1: blocks of the tile
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t x[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        widest = kF8 ? __vmaxu4(widest, x[k] & 0x7f7f7f7fu) : __vmaxu2(widest, x[k] & 0x7fff7fffu);
    }
#pragma unroll
    for (int mt = 0; mt < kTiles; ++mt) {
      if (mt * 16 >= G) break;
      float acc[4][4] = {};  // chains: {plus, minus} x {first half, second half of the dims}
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        // The lane's piece i holds dims 8 (t4 + 4 i) .. + 7, or 16 (t4 + 4 i) .. + 15.
#pragma unroll
        for (int hf = 0; hf < (kF8 ? 2 : 1); ++hf) {
          const uint8_t* a = qrow + mt * 16 * kQStride +
                             (kF8 ? (t4 + 4 * i) * 32 + hf * 16 : (t4 + 4 * i) * 16);
          const uint4 u = *reinterpret_cast<const uint4*>(a);
          const uint4 v = *reinterpret_cast<const uint4*>(a + 8 * kQStride);
          const uint32_t ua[4] = {u.x, u.y, u.z, u.w}, va[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // two k-steps: words (0, 1) and (2, 3)
            uint32_t plus[4], minus[4], l0, l1, h0, h1;
            by_sign(ua[2 * k], plus[0], minus[0]);
            by_sign(va[2 * k], plus[1], minus[1]);
            by_sign(ua[2 * k + 1], plus[2], minus[2]);
            by_sign(va[2 * k + 1], plus[3], minus[3]);
            if constexpr (kF8) {
              const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
              const uint32_t hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
              e4m3x4_to_f16x2(lw[2 * hf + k], l0, l1);
              e4m3x4_to_f16x2(hw[2 * hf + k], h0, h1);
            } else {
              l0 = k ? lo[i].z : lo[i].x;
              l1 = k ? lo[i].w : lo[i].y;
              h0 = k ? hi[i].z : hi[i].x;
              h1 = k ? hi[i].w : hi[i].y;
            }
            const int c = kF8 ? 2 * i : 2 * (i >> 1);
            mma_16816<kMmaBF16>(acc[c], plus, h0, h1);
            mma_16816<kMmaBF16>(acc[c + 1], minus, l0, l1);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float s = (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]);
        if (!(fabsf(s) < kInf)) s = kInf;  // not finite: to be scored in 64 bits
        if (mt * 16 + g + (e >> 1) * 8 < G) best[e & 1] = fmaxf(best[e & 1], s);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      best[0] = fmaxf(best[0], __shfl_xor_sync(0xffffffffu, best[0], o));
      best[1] = fmaxf(best[1], __shfl_xor_sync(0xffffffffu, best[1], o));
    }
    if (g == 0)
      *reinterpret_cast<float2*>(scores + tile * 8 + 2 * t4) = make_float2(best[0], best[1]);
  }
  // This CTA's largest bound: E for its blocks (not finite if one of them is not).
  float wide;
  if constexpr (kF8) {
    uint32_t h0, h1;
    e4m3x4_to_f16x2(widest, h0, h1);
    const float2 x = unpack2<false>(h0), y = unpack2<false>(h1);
    wide = fmaxf(fmaxf(x.x, x.y), fmaxf(y.x, y.y));
    if (x.x != x.x || x.y != x.y || y.x != y.x || y.y != y.y) wide = kInf;
  } else {
    const float2 x = unpack2<kBF16>(widest);
    wide = x.x != x.x || x.y != x.y ? kInf : fmaxf(x.x, x.y);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, o));
  if (lane == 0) part[warp] = wide;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < kScoreWarps; ++w) wide = fmaxf(wide, part[w]);
    // (Beyond 1e37 a sum could overflow; NaN is a product of 0 and an infinity.)
    const float m = q1 * wide;
    p.error[bj * gridDim.x + blockIdx.x] = m < 1e37f ? kError * m : kInf;
  }
}

// ------------------------------------------------------------------ the choice

constexpr int kFew = 32;  // blocks near the cut that one warp can order
constexpr int kCachedBlocks = 40960;  // scores that are kept in shared memory

// A block's score from its definition, in 64 bits throughout: what values that are
// not finite take.  lo, hi: the lane's dims 4 l .. 4 l + 3.
template <bool kBF16>
__device__ __noinline__ double score_of_strange_values(const uint16_t* q, int group,
                                                       const float4 lo4, const float4 hi4) {
  const float lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
  const double inf = __longlong_as_double(0x7ff0000000000000ll);
  double best = -inf;
  for (int r = 0; r < group; ++r) {
    const uint2 w = *reinterpret_cast<const uint2*>(q + r * kHeadDim);
    const float2 a = unpack2<kBF16>(w.x), c = unpack2<kBF16>(w.y);
    const float x[4] = {a.x, a.y, c.x, c.y};
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double u = static_cast<double>(x[k]) * lo[k], v = static_cast<double>(x[k]) * hi[k];
      sum += u != u ? u : v != v ? v : u > v ? u : v;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (sum != sum) sum = inf;
    best = sum > best ? sum : best;
  }
  return best;
}

// s_t in 64 bits, by a warp; the same value in every lane, NaN counts as +inf.  A
// product in 64 bits takes a warp 16 cycles here, so only the heads that may hold
// the maximum are taken so: those within the 32-bit sums' error (a lane's four
// products and sums, five more, each 2^-24 of the sum of magnitudes) of the
// largest.  (All heads, and the definition's comparisons in 64 bits, took 18 us
// for three blocks of 8 heads.)
template <bool kF8, bool kBF16>
DECATTN_DEV double exact_score(const SelectParams& p, int64_t bj, int j, int id, int lane) {
  const int64_t row = (static_cast<int64_t>(id) * 2 * p.h_kv + j) * kHeadDim + lane * 4;
  float lo[4], hi[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t at = row + k * static_cast<int64_t>(p.h_kv) * kHeadDim;
    uint32_t w0, w1;
    if constexpr (kF8) {
      e4m3x4_to_f16x2(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.bounds) + at), w0, w1);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.bounds) + at);
      w0 = w.x;
      w1 = w.y;
    }
    const float2 a = unpack2<kBF16 && !kF8>(w0), c = unpack2<kBF16 && !kF8>(w1);
    float* to = k ? hi : lo;
    to[0] = a.x; to[1] = a.y; to[2] = c.x; to[3] = c.y;
  }
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + bj * p.group * kHeadDim + lane * 4;
  float up[4], down[4], sum_all = 0.f;  // what a positive, a negative value of q meets
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    up[k] = fmaxf(lo[k], hi[k]);
    down[k] = fminf(lo[k], hi[k]);
    sum_all += fabsf(lo[k]) + fabsf(hi[k]);
  }
  // Head r's 32-bit sum and its error stay with lane r % 32; eight heads at a time, so
  // that their loads and exchanges overlap.
  float sums[2] = {-kInf, -kInf}, errors[2] = {0.f, 0.f}, floor_ = -kInf;
  bool finite = sum_all < kInf;
  for (int r0 = 0; r0 < p.group; r0 += 8) {
    uint2 w[8];
    float s[8], mag[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      w[r] = *reinterpret_cast<const uint2*>(q + min(r0 + r, p.group - 1) * kHeadDim);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float2 a = unpack2<kBF16>(w[r].x), c = unpack2<kBF16>(w[r].y);
      const float x[4] = {a.x, a.y, c.x, c.y};
      s[r] = mag[r] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float b = x[k] >= 0.f ? up[k] : down[k];
        s[r] = fmaf(x[k], b, s[r]);
        mag[r] = fmaf(fabsf(x[k]), fabsf(b), mag[r]);
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
        mag[r] += __shfl_xor_sync(0xffffffffu, mag[r], o);
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      finite &= mag[r] < 1e37f;
      const float err = fmaf(mag[r], 0x1p-20f, 1e-36f);  // (products below 2^-126 lose their lower bits)
      floor_ = fmaxf(floor_, s[r] - err);
      if (lane == ((r0 + r) & 31) && r0 + r < p.group) {
        if (r0 < 32) {
          sums[0] = s[r];
          errors[0] = err;
        } else {
          sums[1] = s[r];
          errors[1] = err;
        }
      }
    }
  }
  if (!__all_sync(0xffffffffu, finite))
    return score_of_strange_values<kBF16>(q, p.group, make_float4(lo[0], lo[1], lo[2], lo[3]),
                                          make_float4(hi[0], hi[1], hi[2], hi[3]));
  double best = -__longlong_as_double(0x7ff0000000000000ll);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    unsigned may = __ballot_sync(0xffffffffu, sums[h] + errors[h] >= floor_);
    while (may) {
      const int r = 32 * h + __ffs(may) - 1;
      may &= may - 1;
      const uint2 w = *reinterpret_cast<const uint2*>(q + r * kHeadDim);
      const float2 a = unpack2<kBF16>(w.x), c = unpack2<kBF16>(w.y);
      const float x[4] = {a.x, a.y, c.x, c.y};
      double sum = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        sum = fma(static_cast<double>(x[k]), static_cast<double>(x[k] >= 0.f ? up[k] : down[k]), sum);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      best = sum > best ? sum : best;
    }
  }
  return best;
}

template <bool kF8, bool kBF16, int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads) choose_blocks_kernel(const SelectParams p) {
  using T = Team<kCluster>;
  extern __shared__ float cached[];
  __shared__ CutScratch cut;
  __shared__ ListScratch list;
  __shared__ int few[kFew], own_few[kFew], count_few, count_sure;
  __shared__ double few_score[kFew];
  __shared__ unsigned few_taken, widest;
  const int j = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t bj = static_cast<int64_t>(b) * p.h_kv + j;
  int32_t* out = p.selected + bj * p.count;
  // (What the first kernel does not write is read before it has ended.)
  const int n = p.seq_lens[b];
  const bool bad_len = n < 0 || n > p.max_seq_len;
  if (bad_len && tid == 0 && j == 0 && T::rank() == 0) flag_error(p.err_flag, kFlagBadSeqLen);
  const int blocks = n > 0 && !bad_len ? ((n - 1) >> p.log2_block_size) + 1 : 0;
  if (blocks <= p.count) {  // all of them
    wait_for_dependence();
    if (T::rank() == 0)
      for (int k = tid; k < p.count; k += kThreads) out[k] = k < blocks ? k : -1;
    return;
  }
  // This CTA's blocks: [begin, begin + own).
  const int slice = (blocks + T::size() - 1) / T::size();
  const int begin = min(blocks, T::rank() * slice), own = min(slice, blocks - begin);
  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  const float* scores = p.scores + bj * p.score_stride + begin;
  // [first, last) of them are chosen by score, `want` of the team's.
  const int first = p.first - begin, last = blocks - p.last - begin;
  const int want = p.count - p.first - p.last;
  const bool cache = own <= p.cached_blocks;
  cut_prepare(cut);
  if (tid == 0) {
    count_few = count_sure = 0;
    widest = 0;
  }
  // (Every CTA of a team checks the whole table: they go on together.)
  int bad = 0;
#pragma unroll 4
  for (int t = tid; t < blocks; t += kThreads) {
    const int id = bt[t];
    bad |= id < 0 || id >= p.num_blocks;
  }
  wait_for_dependence();  // the scores are there
  // The widest error of the scores (not negative: ordered as its bits), by a warp.
  float e = tid < p.score_ctas ? p.error[bj * p.score_ctas + tid] : 0.f;
  uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll 4
  for (int t = tid; t < own; t += kThreads) {
    const float x = scores[t];
    if (cache) cached[t] = x;
    if (t >= first && t < last) {
      lo = min(lo, order_key(x));
      hi = max(hi, order_key(x));
    }
  }
  if (cache) scores = cached;
  for (int x = tid + kThreads; x < p.score_ctas; x += kThreads)
    e = fmaxf(e, p.error[bj * p.score_ctas + x]);
  if (__syncthreads_or(bad)) {
    if (tid == 0) flag_error(p.err_flag, kFlagBadBlock);
    if (T::rank() == 0)
      for (int k = tid; k < p.count; k += kThreads) out[k] = -1;
    return;
  }
  const unsigned wide = __reduce_max_sync(0xffffffffu, __float_as_uint(e));
  if (lane == 0 && wide) atomicMax(&widest, wide);
  __syncthreads();
  e = __uint_as_float(widest);

  // Blocks surely in score above `above`, surely out below `below`.
  float above = kInf, below = -kInf;
  if (want > 0) {
    const Cut c = cut_largest<kThreads, kCluster>(cut, lo, hi, own, want, [&](int t, uint32_t& k) {
      k = order_key(scores[t]);
      return t >= first && t < last;
    });
    const float v = key_value(c.key);
    // (Not finite anywhere: the scores order nothing.  Rounded outwards.)
    if (e < kInf && v < kInf) {
      above = __fadd_ru(v, 2.f * e);
      below = __fadd_rd(v, -2.f * e);
    }
  }
  const bool by_score = want > 0;
  // 0: out, 1: in, 2: near the cut
  auto near_cut = [&](int t) {
    if (t < first || t >= last) return 1;
    if (!by_score) return 0;
    const float s = scores[t];
    return s > above ? 1 : s < below ? 0 : 2;
  };
  int sure = 0;
#pragma unroll 2
  for (int t0 = 0; t0 < own; t0 += kThreads) {
    const int t = t0 + tid;
    const int k = t < own ? near_cut(t) : 0;
    sure += __popc(__ballot_sync(0xffffffffu, k == 1));
    if (k == 2) T::push(few, &count_few, kFew, begin + t);
  }
  if (lane == 0 && sure) atomicAdd(&count_sure, sure);
  T::sync();
  const int close = T::get(count_few, 0);  // near the cut, and how many of these are in:
  const int left =
      p.count - __reduce_add_sync(0xffffffffu, lane < T::size() ? T::get(count_sure, lane) : 0);

  auto emit = [&](int t, int rank) { out[rank] = begin + t; };
  if (left >= close || left <= 0) {
    list_in_order<kThreads, kCluster>(list, own, 0, [&](int t) {
      const int k = near_cut(t);
      return k == 2 ? (left > 0 ? 1 : 0) : k;
    }, emit);
    return;
  }
  if (close <= kFew) {
    // (Each CTA for itself.)
    for (int c = warp; c < close; c += kThreads / 32) {
      const int t = T::get(few[c], 0);
      const double s = exact_score<kF8, kBF16>(p, bj, j, bt[t], lane);
      if (lane == 0) {
        own_few[c] = t;
        few_score[c] = s;
      }
    }
    __syncthreads();
    if (warp == 0) {
      int better = 0;
      if (lane < close)
        for (int c = 0; c < close; ++c)
          better += few_score[c] > few_score[lane] ||
                    (few_score[c] == few_score[lane] && own_few[c] < own_few[lane]);
      const unsigned taken = __ballot_sync(0xffffffffu, lane < close && better < left);
      if (lane == 0) few_taken = taken;
    }
    __syncthreads();
    list_in_order<kThreads, kCluster>(list, own, 0, [&](int t) {
      int k = near_cut(t);
      if (k == 2) {
        k = 0;
        for (int c = 0; c < close; ++c)
          if (own_few[c] == begin + t) k = few_taken >> c & 1;
      }
      return k;
    }, emit);
    return;
  }
  // Many blocks alike (equal keys, values that are not finite): all of them in 64
  // bits, cut by the upper word of their order, then by the lower.
  uint64_t* exact = p.exact + bj * p.score_stride + begin;
  for (int t = warp; t < own; t += kThreads / 32) {
    if (near_cut(t) != 2) continue;
    const double s = exact_score<kF8, kBF16>(p, bj, j, bt[begin + t], lane);
    if (lane == 0) exact[t] = order_key(s);
  }
  __syncthreads();
  const Cut up = cut_largest<kThreads, kCluster>(cut, 0u, 0xffffffffu, own, left, [&](int t, uint32_t& k) {
    if (near_cut(t) != 2) return false;
    k = static_cast<uint32_t>(exact[t] >> 32);
    return true;
  });
  const Cut lower = cut_largest<kThreads, kCluster>(cut, 0u, 0xffffffffu, own, up.ties, [&](int t, uint32_t& k) {
    if (near_cut(t) != 2 || exact[t] >> 32 != up.key) return false;
    k = static_cast<uint32_t>(exact[t]);
    return true;
  });
  const uint64_t at = static_cast<uint64_t>(up.key) << 32 | lower.key;
  list_in_order<kThreads, kCluster>(list, own, lower.ties, [&](int t) {
    const int k = near_cut(t);
    return k != 2 ? k : exact[t] > at ? 1 : exact[t] == at ? 2 : 0;
  }, emit);
}

template <bool kF8, bool kBF16, int kThreads, bool kCluster>
cudaError_t launch_choice(const SelectParams& p, cudaStream_t stream) {
  auto kern = choose_blocks_kernel<kF8, kBF16, kThreads, kCluster>;
  const size_t smem = static_cast<size_t>(p.cached_blocks) * sizeof(float);
  if (smem > 36 * 1024) {  // (beside static shared memory, of 48 KB)
    // (The largest that is ever asked for, so that no call lowers another's limit.)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kCachedBlocks * static_cast<int>(sizeof(float)));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.team), static_cast<unsigned>(p.h_kv),
                     static_cast<unsigned>(p.batch));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.team);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.score_ctas > 0 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kF8, bool kBF16>
cudaError_t launch_t(const SelectParams& p, cudaStream_t stream) {
  if (p.score_ctas > 0) {
    const dim3 grid(static_cast<unsigned>(p.score_ctas), static_cast<unsigned>(p.h_kv),
                    static_cast<unsigned>(p.batch));
    if (p.group <= 16)
      block_scores_kernel<kF8, kBF16, 1><<<grid, kScoreWarps * 32, 0, stream>>>(p);
    else
      block_scores_kernel<kF8, kBF16, 4><<<grid, kScoreWarps * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return p.team > 1 ? launch_choice<kF8, kBF16, 512, true>(p, stream)
                    : launch_choice<kF8, kBF16, 512, false>(p, stream);
}

}  // namespace

int select_score_ctas(int batch, int h_kv, int blocks, int count, int num_sms) {
  if (blocks <= count) return 0;
  // A warp's tile is 8 blocks; about two waves of eight CTAs an SM.
  const int64_t most = (blocks + 8 * kScoreWarps - 1) / (8 * kScoreWarps);
  const int64_t share = std::max<int64_t>(1, static_cast<int64_t>(num_sms) * 16 /
                                                 (static_cast<int64_t>(batch) * h_kv));
  return static_cast<int>(std::min(most, share));
}

// The second kernel's CTAs to a sequence and KV head: a cluster of up to eight, while
// there are SMs for them and 1024 blocks for each.
void plan_choice(SelectParams& p, int blocks, int num_sms) {
  p.team = 1;
  p.cached_blocks = 0;
  if (blocks <= p.count) return;
  while (p.team < 8 && static_cast<int64_t>(p.batch) * p.h_kv * p.team * 2 <= num_sms &&
         blocks >= 2 * p.team * 1024)
    p.team *= 2;
  while (p.team < 8 && blocks > p.team * kCachedBlocks) p.team *= 2;
  const int own = (blocks + p.team - 1) / p.team;
  p.cached_blocks = own <= kCachedBlocks ? own : 0;
}

cudaError_t launch_select_blocks(const SelectParams& p, bool e4m3, bool bf16, cudaStream_t stream) {
  if (e4m3) return bf16 ? launch_t<true, true>(p, stream) : launch_t<true, false>(p, stream);
  return bf16 ? launch_t<false, true>(p, stream) : launch_t<false, false>(p, stream);
}

}  // namespace decattn
