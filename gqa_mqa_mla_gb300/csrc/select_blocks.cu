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
// scores run on mma.sync in 32 bits: a warp takes 16 blocks (m) against 8 query heads
// at a time (n); a lane's 16-byte pieces of the bounds' rows are the A fragments as
// they are (the k index is permuted, the same for q), and up to 8 heads' q^+ and q^-
// stay in registers as B fragments.  (With the heads as m, 8 blocks as n, the kernel
// spent its issue slots on splitting q by sign for each tile: 37 us for 196 MB.)  Such
// a score is off by at most
//     E = 2^-16 max_i sum_d |q_id| max_td |bound_td|:
// four chains of four products of 16 terms, each term off by at most 2^-23 of the
// chain's sum of magnitudes (4 x 17 x 2^-23), and their sum.  The second kernel, a
// CTA to each sequence and KV head, finds the cut v (cut.cuh); blocks
// within 2 E of it, usually none but the cut itself, are scored again, in 32 bits with
// tighter bounds on the error and, where these leave something open, in 64.
// Doing all in 64 bits would take 40 times the floor here: 0.6 T products a second.
#include <algorithm>

#include "cut.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr int kScoreWarps = 4;
constexpr int kScoreBlocks = 16;  // blocks of a warp's tile
constexpr int kQStride = 320;     // bytes of a 128-value row in shared memory: rows two banks' groups apart
constexpr float kInf = __builtin_huge_valf();
constexpr float kError = 1.52587890625e-05f;  // 2^-16

// q^+ and q^- of a pair: the halves whose sign bit is clear / set, else 0.
DECATTN_DEV uint4 by_sign(uint4 w, bool negative) {
  auto part = [&](uint32_t x) {
    const uint32_t sign = byte_perm(x, 0u, 0xbb99u);  // (each half's sign, 16 times)
    return negative ? x & sign : x & ~sign;
  };
  return make_uint4(part(w.x), part(w.y), part(w.z), part(w.w));
}

// Over 8 bits q is multiplied as fp16, a bf16 query times a power of two for its group
// (the scores of the pair (b, j) then all carry that factor).
template <bool kF8, bool kBF16>
DECATTN_DEV float query_scale(float most) {
  return kF8 && kBF16 ? fp16_scale(most) : 1.f;
}
template <bool kBF16>
DECATTN_DEV float largest(uint4 w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  float most = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2<kBF16>(x[k]);
    most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  return most;
}
// w times alpha, as it is multiplied, and the sum of its magnitudes added to `sum`.
template <bool kF8, bool kBF16>
DECATTN_DEV uint4 scaled(uint4 w, float alpha, float& sum) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2<kBF16>(x[k]);
    sum += alpha * (fabsf(f.x) + fabsf(f.y));
    if constexpr (kF8 && kBF16) x[k] = pack2<false>(f.x * alpha, f.y * alpha);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// kHeads: 8 (their fragments in registers), 16 or 64 heads a KV head at most.  kSpread
// (8): a CTA's warps take p.score_heads neighbouring KV heads of the same blocks, whose
// bounds are neighbours in memory, and load the queries themselves (32 sequences of
// 16-32k tokens, 196 MB: 34.5 us, 36.5 with a KV head to a CTA); else a CTA's warps share
// one KV head's, which lie in shared memory.
template <bool kF8, bool kBF16, int kHeads, bool kSpread>
__global__ void __launch_bounds__(kScoreWarps * 32, 4) block_scores_kernel(const SelectParams p) {
  constexpr bool kMmaBF16 = kBF16 && !kF8;
  constexpr int kRows = kSpread ? 1 : kHeads;
  static_assert(!kSpread || kHeads == 8, "fragments in registers");
  __shared__ __align__(16) uint8_t qs[2][kRows * kQStride];  // q^+, q^-
  __shared__ float mag[kRows], part[kScoreWarps];
  __shared__ uint32_t part_lo[kScoreWarps], part_hi[kScoreWarps];
  launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int heads = kSpread ? p.score_heads : 1;  // (a power of two that divides h_kv)
  const int j = blockIdx.y * heads + (warp & (heads - 1)), b = blockIdx.z, G = p.group;
  const int sub = kSpread ? warp / heads : warp, subs = kScoreWarps / heads;
  const int64_t bj = static_cast<int64_t>(b) * p.h_kv + j;
  const int n = p.seq_lens[b];
  const int blocks = n > 0 && n <= p.max_seq_len ? ((n - 1) >> p.log2_block_size) + 1 : 0;
  // Nothing to choose (or a bad length, which the second kernel reports).
  if (blocks <= p.count) return;

  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  const int tiles = (blocks + kScoreBlocks - 1) / kScoreBlocks, step = gridDim.x * subs;
  int tile = blockIdx.x * subs + sub;
  // (-1 for blocks that are taken always: their bounds are not looked at.)
  auto block_of = [&](int tl, int row) {
    const int t = tl * kScoreBlocks + row;
    return tl < tiles && t >= p.first && t < blocks - p.last ? bt[t] : -1;
  };
  int id[2] = {block_of(tile, g), block_of(tile, g + 8)};
  constexpr int kRowBytes = kF8 ? kHeadDim : 2 * kHeadDim;
  constexpr int kPieces = kRowBytes / 64;         // 16-byte pieces a lane has of a row
  constexpr int kParts = kF8 ? 2 * kPieces : kPieces;  // of a row of q (16 bytes: two k-steps)
  const int64_t half = static_cast<int64_t>(p.h_kv) * kRowBytes;  // from a block's lo to its hi
  const uint8_t* bounds = static_cast<const uint8_t*>(p.bounds) + j * kRowBytes + t4 * 16;
  // A head's part i: dims 8 (t4 + 4 i) .. + 7, or (8-bit: the lane's piece i / 2 of a
  // bounds row has dims 16 (t4 + 4 (i / 2)) .. + 15) the half i % 2 of them.  In bytes:
  auto part_at = [&](int i) {
    return kF8 ? (t4 + 4 * (i >> 1)) * 32 + (i & 1) * 16 : (t4 + 4 * i) * 16;
  };
  const uint8_t* q = static_cast<const uint8_t*>(p.q) + bj * G * (2 * kHeadDim);
  float q1 = 0.f;
  uint4 held[2][kHeads == 8 ? kParts : 1];
  auto q_part = [&](int sign, int nt, int i) {
    return *reinterpret_cast<const uint4*>(qs[sign] + (nt * 8 + g) * kQStride + part_at(i));
  };
  if constexpr (kSpread) {
    uint4 w[kParts];
    float most = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      w[i] = make_uint4(0, 0, 0, 0);
      if (g < G) w[i] = *reinterpret_cast<const uint4*>(q + g * (2 * kHeadDim) + part_at(i));
      most = fmaxf(most, largest<kBF16>(w[i]));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float alpha = query_scale<kF8, kBF16>(most);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      w[i] = scaled<kF8, kBF16>(w[i], alpha, sum);
      held[0][i] = by_sign(w[i], false);
      held[1][i] = by_sign(w[i], true);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    q1 = fmaxf(0.f, sum);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) q1 = fmaxf(q1, __shfl_xor_sync(0xffffffffu, q1, o));
  } else {
    // 16 lanes have a row, 8 values each (rows past the group: zeros).
    const int piece = lane & 15;
    auto q_row = [&](int r) {
      return r < G ? *reinterpret_cast<const uint4*>(q + r * (2 * kHeadDim) + piece * 16)
                   : make_uint4(0, 0, 0, 0);
    };
    float alpha = 1.f;
    if constexpr (kF8 && kBF16) {
      for (int r = 2 * warp + (lane >> 4); r < kHeads; r += 2 * kScoreWarps) {
        float most = largest<kBF16>(q_row(r));
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (piece == 0) mag[r] = most;
      }
      __syncthreads();
      float most = 0.f;
      for (int r = 0; r < G; ++r) most = fmaxf(most, mag[r]);
      alpha = query_scale<kF8, kBF16>(most);
      __syncthreads();
    }
    for (int r = 2 * warp + (lane >> 4); r < kHeads; r += 2 * kScoreWarps) {
      float sum = 0.f;
      const uint4 w = scaled<kF8, kBF16>(q_row(r), alpha, sum);
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (piece == 0) mag[r] = sum;
      *reinterpret_cast<uint4*>(qs[0] + r * kQStride + piece * 16) = by_sign(w, false);
      *reinterpret_cast<uint4*>(qs[1] + r * kQStride + piece * 16) = by_sign(w, true);
    }
    __syncthreads();
    for (int r = 0; r < G; ++r) q1 = fmaxf(q1, mag[r]);
    if constexpr (kHeads == 8) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        held[0][i] = q_part(0, 0, i);
        held[1][i] = q_part(1, 0, i);
      }
    }
  }
  float* scores = p.scores + bj * p.score_stride;
  uint32_t key_lo = 0xffffffffu, key_hi = 0u;  // the range of the scores, as cut.cuh orders them
  // The largest bound and the largest of minus the bounds, packed (8-bit: the codes'
  // magnitudes in the first).
  uint32_t most_hi = kF8 ? 0u : (kBF16 ? 0xff80ff80u : 0xfc00fc00u), most_lo = most_hi;
  for (; tile < tiles; tile += step) {
    uint4 x[2][2][kPieces];  // blocks g and g + 8; lo and hi
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool there = id[r] >= 0 && id[r] < p.num_blocks;  // (a bad id: the second kernel reports it)
      const uint8_t* at = bounds + static_cast<int64_t>(id[r]) * 2 * half;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          x[r][e][i] = make_uint4(0u, 0u, 0u, 0u);
          if (there) x[r][e][i] = *reinterpret_cast<const uint4*>(at + e * half + i * 64);
        }
    }
    id[0] = block_of(tile + step, g);
    id[1] = block_of(tile + step, g + 8);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint4 l = x[r][0][i], h = x[r][1][i];
        if constexpr (kF8) {
          constexpr uint32_t kMag = 0x7f7f7f7fu;
          most_hi = __vmaxu4(most_hi, __vmaxu4(__vmaxu4(l.x & kMag, l.y & kMag), __vmaxu4(l.z & kMag, l.w & kMag)));
          most_hi = __vmaxu4(most_hi, __vmaxu4(__vmaxu4(h.x & kMag, h.y & kMag), __vmaxu4(h.z & kMag, h.w & kMag)));
        } else {  // (lo <= hi: the largest magnitude is hi's largest or minus lo's smallest)
          most_hi = max2<kBF16>(most_hi, max2<kBF16>(max2<kBF16>(h.x, h.y), max2<kBF16>(h.z, h.w)));
          most_lo = max2<kBF16>(most_lo, max2<kBF16>(max2<kBF16>(l.x ^ 0x80008000u, l.y ^ 0x80008000u),
                                                     max2<kBF16>(l.z ^ 0x80008000u, l.w ^ 0x80008000u)));
        }
      }
    float best[2] = {-kInf, -kInf};  // of blocks g and g + 8
#pragma unroll
    for (int nt = 0; nt < kHeads / 8; ++nt) {
      if (nt * 8 >= G) break;
      float acc[4][4] = {};  // chains: {lo, hi} x {first half, second half of the dims}
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
#pragma unroll
        for (int hf = 0; hf < kParts / kPieces; ++hf) {
          const int part_i = kF8 ? 2 * i + hf : i, c = kF8 ? 2 * i : 2 * (i >> 1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // lo meets q^-, hi q^+
            uint4 w;
            if constexpr (kHeads == 8)
              w = held[e ? 0 : 1][part_i];
            else
              w = q_part(e ? 0 : 1, nt, part_i);
            const uint4 u = x[0][e][i], v = x[1][e][i];
            if constexpr (kF8) {
              const uint32_t u2[2] = {hf ? u.z : u.x, hf ? u.w : u.y};
              const uint32_t v2[2] = {hf ? v.z : v.x, hf ? v.w : v.y};
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t a[4];
                e4m3x4_to_f16x2(u2[k], a[0], a[2]);
                e4m3x4_to_f16x2(v2[k], a[1], a[3]);
                mma_16816<false>(acc[c + e], a, k ? w.z : w.x, k ? w.w : w.y);
              }
            } else {
              const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
              mma_16816<kMmaBF16>(acc[c + e], a0, w.x, w.y);
              mma_16816<kMmaBF16>(acc[c + e], a1, w.z, w.w);
            }
          }
        }
      }
      // Element e of the lane: block g + 8 (e / 2), head 8 nt + 2 t4 + e % 2.
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float s = (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]);
        if (!(fabsf(s) < kInf)) s = kInf;  // not finite: to be scored in 64 bits
        if (nt * 8 + 2 * t4 + (e & 1) < G) best[e >> 1] = fmaxf(best[e >> 1], s);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
      const int t = tile * kScoreBlocks + g + 8 * r;
      if (t4 == 0) scores[t] = best[r];
      if (t >= p.first && t < blocks - p.last) {
        key_lo = min(key_lo, order_key(best[r]));
        key_hi = max(key_hi, order_key(best[r]));
      }
    }
  }
  // This CTA's largest bound, E for its blocks (not finite if one of them is not), and
  // the range of its scores.
  float wide = 0.f;
  if constexpr (kF8) {
    uint32_t h0, h1;
    e4m3x4_to_f16x2(most_hi, h0, h1);
    const float2 u = unpack2<false>(h0), v = unpack2<false>(h1);
    wide = fmaxf(fmaxf(u.x, u.y), fmaxf(v.x, v.y));
    if (u.x != u.x || u.y != u.y || v.x != v.x || v.y != v.y) wide = kInf;
  } else {
    const float2 u = unpack2<kBF16>(max2<kBF16>(most_hi, most_lo));
    wide = u.x != u.x || u.y != u.y ? kInf : fmaxf(0.f, fmaxf(u.x, u.y));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, o));
  key_lo = __reduce_min_sync(0xffffffffu, key_lo);
  key_hi = __reduce_max_sync(0xffffffffu, key_hi);
  if (lane == 0) {
    part[warp] = wide;
    part_lo[warp] = key_lo;
    part_hi[warp] = key_hi;
  }
  __syncthreads();
  if (lane == 0 && sub == 0) {
    for (int w = 1; w < subs; ++w) {
      wide = fmaxf(wide, part[warp + w * heads]);
      key_lo = min(key_lo, part_lo[warp + w * heads]);
      key_hi = max(key_hi, part_hi[warp + w * heads]);
    }
    // (Beyond 1e37 a sum could overflow, NaN is a product of 0 and an infinity; factors
    // and products below 2^-126 may count as 0, 128 of them.)
    const float m = q1 * wide, lost = 0x1p-118f * (1.f + wide + q1);
    const float e = m < 1e37f ? fmaf(kError, m, lost) : kInf;
    p.parts[bj * gridDim.x + blockIdx.x] = make_uint4(__float_as_uint(e), key_lo, key_hi, 0u);
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

// A block's lo and hi for the lane's dims 4 l .. 4 l + 3.
template <bool kF8, bool kBF16>
DECATTN_DEV void load_bounds(const SelectParams& p, int j, int id, int lane, float (&lo)[4], float (&hi)[4]) {
  const int64_t row = (static_cast<int64_t>(id) * 2 * p.h_kv + j) * kHeadDim + lane * 4;
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
}

// s_t in 32 bits, by a warp, with bounds on its error: a lane's four products and sums,
// five more, and the bound itself, each off by 2^-24 of the sum of magnitudes at most: 11 of these.  (Tighter than E,
// which takes one magnitude for all dims, and adds as the tensor cores do.)
struct Rough {
  float lo, hi;               // the maximum over the heads lies within
  float sums[2], errors[2];   // heads lane and lane + 32
  bool finite;                // else nothing is known
};
template <bool kBF16>
DECATTN_DEV Rough rough_score(const uint16_t* q, int group, int lane, const float (&lo)[4],
                              const float (&hi)[4], const float (&up)[4], const float (&down)[4]) {
  Rough r = {-kInf, -kInf, {-kInf, -kInf}, {0.f, 0.f}, true};
  float sum_all = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) sum_all += fabsf(lo[k]) + fabsf(hi[k]);
  r.finite = sum_all < kInf;
  // Eight heads at a time, so that their loads and exchanges overlap.
  for (int h0 = 0; h0 < group; h0 += 8) {
    uint2 w[8];
    float s[8], mag[8];
#pragma unroll
    for (int h = 0; h < 8; ++h)
      w[h] = *reinterpret_cast<const uint2*>(q + min(h0 + h, group - 1) * kHeadDim);
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const float2 a = unpack2<kBF16>(w[h].x), c = unpack2<kBF16>(w[h].y);
      const float x[4] = {a.x, a.y, c.x, c.y};
      s[h] = mag[h] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float b = x[k] >= 0.f ? up[k] : down[k];
        s[h] = fmaf(x[k], b, s[h]);
        mag[h] = fmaf(fabsf(x[k]), fabsf(b), mag[h]);
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        s[h] += __shfl_xor_sync(0xffffffffu, s[h], o);
        mag[h] += __shfl_xor_sync(0xffffffffu, mag[h], o);
      }
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      r.finite &= mag[h] < 1e37f;
      const float err = fmaf(mag[h], 0x1.6p-21f, 1e-36f);  // (products below 2^-126 lose their lower bits)
      r.lo = fmaxf(r.lo, s[h] - err);
      r.hi = fmaxf(r.hi, s[h] + err);
      if (lane == ((h0 + h) & 31) && h0 + h < group) {
        if (h0 < 32) {
          r.sums[0] = s[h];
          r.errors[0] = err;
        } else {
          r.sums[1] = s[h];
          r.errors[1] = err;
        }
      }
    }
  }
  r.finite = __all_sync(0xffffffffu, r.finite);
  return r;
}

template <bool kF8, bool kBF16>
DECATTN_DEV Rough look_score(const SelectParams& p, int64_t bj, int j, int id, int lane,
                             float (&lo)[4], float (&hi)[4], float (&up)[4], float (&down)[4]) {
  load_bounds<kF8, kBF16>(p, j, id, lane, lo, hi);
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // what a positive, a negative value of q meets
    up[k] = fmaxf(lo[k], hi[k]);
    down[k] = fminf(lo[k], hi[k]);
  }
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + bj * p.group * kHeadDim + lane * 4;
  return rough_score<kBF16>(q, p.group, lane, lo, hi, up, down);
}

// s_t in 64 bits, by a warp; the same value in every lane, NaN counts as +inf.  A
// product in 64 bits takes a warp 16 cycles here, so only the heads that may hold
// the maximum are taken so.  (All heads, and the definition's comparisons in 64 bits,
// took 18 us for three blocks of 8 heads.)
template <bool kF8, bool kBF16>
__device__ __noinline__ double exact_score(const SelectParams& p, int64_t bj, int j, int id, int lane) {
  float lo[4], hi[4], up[4], down[4];
  const Rough rough = look_score<kF8, kBF16>(p, bj, j, id, lane, lo, hi, up, down);
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + bj * p.group * kHeadDim + lane * 4;
  if (!rough.finite)
    return score_of_strange_values<kBF16>(q, p.group, make_float4(lo[0], lo[1], lo[2], lo[3]),
                                          make_float4(hi[0], hi[1], hi[2], hi[3]));
  double best = -__longlong_as_double(0x7ff0000000000000ll);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    unsigned may = __ballot_sync(0xffffffffu, rough.sums[h] + rough.errors[h] >= rough.lo);
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

// (Without a cluster there are more CTAs than SMs, and two have to fit: at 72 registers
// the choice took 21 us for 256 of them, 14 at 64.)
template <bool kF8, bool kBF16, int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads, kCluster ? 1 : 1024 / kThreads) choose_blocks_kernel(const SelectParams p) {
  using T = Team<kCluster>;
  extern __shared__ float cached[];
  __shared__ CutScratch cut;
  __shared__ ListScratch list;
  __shared__ int few[kFew], own_few[kFew], count_few;
  __shared__ double few_score[kFew];
  __shared__ float few_lo[kFew], few_hi[kFew];
  __shared__ unsigned few_taken, few_open, widest, key_lo, key_hi;
  const int j = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t bj = static_cast<int64_t>(b) * p.h_kv + j;
  int32_t* out = p.selected + bj * p.count;
  // (What the first kernel does not write is read before it has ended.)
  const int n = p.seq_lens[b];
  const bool bad_len = n < 0 || n > p.max_seq_len;
  if (bad_len && tid == 0 && j == 0 && T::rank() == 0) flag_error(p.err_flag, kFlagBadSeqLen);
  const int blocks = n > 0 && !bad_len ? ((n - 1) >> p.log2_block_size) + 1 : 0;
  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  // (Every CTA of a team checks the whole table: they go on together.)
  int bad = 0;
#pragma unroll 4
  for (int t = tid; t < blocks; t += kThreads) {
    const int id = bt[t];
    bad |= id < 0 || id >= p.num_blocks;
  }
  if (blocks <= p.count) {  // all of them
    wait_for_dependence();
    const bool wrong = __syncthreads_or(bad);
    if (wrong && tid == 0) flag_error(p.err_flag, kFlagBadBlock);
    if (T::rank() == 0)
      for (int k = tid; k < p.count; k += kThreads) out[k] = k < blocks && !wrong ? k : -1;
    return;
  }
  // This CTA's blocks: [begin, begin + own).
  const int slice = (blocks + T::size() - 1) / T::size();
  const int begin = min(blocks, T::rank() * slice), own = min(slice, blocks - begin);
  const float* scores = p.scores + bj * p.score_stride + begin;
  // [first, last) of them are chosen by score, `want` of the team's.
  const int first = p.first - begin, last = blocks - p.last - begin;
  const int want = p.count - p.first - p.last;
  const bool cache = own <= p.cached_blocks;
  cut_prepare(cut);
  if (tid == 0) {
    count_few = 0;
    widest = key_hi = 0u;
    key_lo = 0xffffffffu;
  }
  wait_for_dependence();  // the scores are there
  // The widest error of the scores (not negative: ordered as its bits) and their range,
  // from what the first kernel's CTAs left.
  const uint4* parts = p.parts + bj * p.score_ctas;
  uint4 mine = tid < p.score_ctas ? parts[tid] : make_uint4(0u, 0xffffffffu, 0u, 0u);
  if (cache) {
#pragma unroll 4
    for (int t = tid; t < own; t += kThreads) cached[t] = scores[t];
    scores = cached;
  }
  for (int x = tid + kThreads; x < p.score_ctas; x += kThreads) {
    const uint4 w = parts[x];
    mine = make_uint4(max(mine.x, w.x), min(mine.y, w.y), max(mine.z, w.z), 0u);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) flag_error(p.err_flag, kFlagBadBlock);
    if (T::rank() == 0)
      for (int k = tid; k < p.count; k += kThreads) out[k] = -1;
    return;
  }
  if (warp * 32 < p.score_ctas) {
    const unsigned e = __reduce_max_sync(0xffffffffu, mine.x);
    const unsigned lo = __reduce_min_sync(0xffffffffu, mine.y), hi = __reduce_max_sync(0xffffffffu, mine.z);
    if (lane == 0) {
      atomicMax(&widest, e);
      atomicMin(&key_lo, lo);
      atomicMax(&key_hi, hi);
    }
  }
  __syncthreads();
  const float e = __uint_as_float(widest);

  // Blocks surely in score above `above`, surely out below `below`.
  float above = kInf, below = -kInf;
  if (want > 0) {
    const Cut c = cut_largest<kThreads, kCluster, true>(cut, key_lo, key_hi, own, want, [&](int t, uint32_t& k) {
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
  auto emit = [&](int t, int rank) { out[rank] = begin + t; };
  // The list in one go: what is in and what is near the cut are counted, the close ones
  // collected; then, `left` of these being in, it is settled which.
  bool settled = true, all = false;
  int close = 0, left = 0;
  list_in_order<kThreads, kCluster>(
      list, own,
      [&](int t, bool again) {
        const int k = near_cut(t);
        if (k == 2 && !again) T::push(few, &count_few, kFew, begin + t);
        return k;
      },
      [&](int in, int tied) {
        close = tied;
        left = p.count - in;
        all = left >= close;
        settled = all || left <= 0 || close <= kFew;
        if (!settled || all || left <= 0) return;
        // (Each CTA for itself; a warp to a block.)  First with the 32-bit sums' own
        // errors, which mostly tell the blocks apart (one sequence of 131072 tokens 22.9
        // us, 24.1 with 64 bits at once).
        for (int c = warp; c < close; c += kThreads / 32) {
          const int t = T::get(few[c], 0);
          float lo[4], hi[4], up[4], down[4];
          const Rough r = look_score<kF8, kBF16>(p, bj, j, bt[t], lane, lo, hi, up, down);
          if (lane == 0) {
            own_few[c] = t;
            few_lo[c] = r.finite ? r.lo : -kInf;
            few_hi[c] = r.finite ? r.hi : kInf;
          }
        }
        __syncthreads();
        if (warp == 0) {
          int surely = 0, perhaps = 0;  // better than the lane's block
          if (lane < close)
            for (int c = 0; c < close; ++c) {
              surely += c != lane && few_lo[c] > few_hi[lane];
              perhaps += c != lane && few_hi[c] >= few_lo[lane];
            }
          const unsigned taken = __ballot_sync(0xffffffffu, lane < close && perhaps < left);
          const unsigned open = __ballot_sync(0xffffffffu, lane < close && perhaps >= left && surely < left);
          if (lane == 0) {
            few_taken = taken;
            few_open = open;
          }
        }
        __syncthreads();
        if (few_open == 0) return;
        for (int c = warp; c < close; c += kThreads / 32) {
          const double s = exact_score<kF8, kBF16>(p, bj, j, bt[own_few[c]], lane);
          if (lane == 0) few_score[c] = s;
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
      },
      [&](int t, bool tied, int in_before, int tied_before) {
        if (!settled) return;
        bool is_in = !tied || all;
        int before = in_before + (all ? tied_before : 0);
        if (!all && left > 0)
          for (int c = 0; c < close; ++c) {
            if (!(few_taken >> c & 1)) continue;
            before += own_few[c] < begin + t;
            is_in |= tied && own_few[c] == begin + t;
          }
        if (is_in) emit(t, before);
      });
  if (settled) return;
  // Many blocks alike (equal keys, values that are not finite): all of them in 64
  // bits, cut by the upper word of their order, then by the lower.
  uint64_t* exact = p.exact + bj * p.score_stride + begin;
  for (int t = warp; t < own; t += kThreads / 32) {
    if (near_cut(t) != 2) continue;
    const double s = exact_score<kF8, kBF16>(p, bj, j, bt[begin + t], lane);
    if (lane == 0) exact[t] = order_key(s);
  }
  __syncthreads();
  const Cut up = cut_largest<kThreads, kCluster, true>(cut, 0u, 0xffffffffu, own, left, [&](int t, uint32_t& k) {
    if (near_cut(t) != 2) return false;
    k = static_cast<uint32_t>(exact[t] >> 32);
    return true;
  });
  const Cut lower = cut_largest<kThreads, kCluster, true>(cut, 0u, 0xffffffffu, own, up.ties, [&](int t, uint32_t& k) {
    if (near_cut(t) != 2 || exact[t] >> 32 != up.key) return false;
    k = static_cast<uint32_t>(exact[t]);
    return true;
  });
  const uint64_t at = static_cast<uint64_t>(up.key) << 32 | lower.key;
  list_largest<kThreads, kCluster>(list, own, lower.ties, [&](int t, bool) {
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
    const dim3 grid(static_cast<unsigned>(p.score_ctas),
                    static_cast<unsigned>(p.h_kv / p.score_heads), static_cast<unsigned>(p.batch));
    if (p.score_heads > 1)
      block_scores_kernel<kF8, kBF16, 8, true><<<grid, kScoreWarps * 32, 0, stream>>>(p);
    else if (p.group <= 8)
      block_scores_kernel<kF8, kBF16, 8, false><<<grid, kScoreWarps * 32, 0, stream>>>(p);
    else if (p.group <= 16)
      block_scores_kernel<kF8, kBF16, 16, false><<<grid, kScoreWarps * 32, 0, stream>>>(p);
    else
      block_scores_kernel<kF8, kBF16, 64, false><<<grid, kScoreWarps * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return p.team > 1 ? launch_choice<kF8, kBF16, 512, true>(p, stream)
                    : launch_choice<kF8, kBF16, 512, false>(p, stream);
}

}  // namespace

// The first kernel's CTAs to a sequence and its KV heads (p.score_heads to a CTA).
void plan_scores(SelectParams& p, int blocks, int num_sms) {
  p.score_heads = 1;
  p.score_ctas = 0;
  if (blocks <= p.count || p.first + p.last == p.count) return;  // no choice to make
  // (Up to two tiles a warp of the GPU there is no stream to keep together: one sequence
  // of 131072 tokens 23.1 us with a head to a CTA, 24.6 with four; 32 of 16-32k 49.2, 47.3.)
  const int64_t tiles = static_cast<int64_t>(p.batch) * p.h_kv * ((blocks + kScoreBlocks - 1) / kScoreBlocks);
  if (p.group <= 8 && tiles > static_cast<int64_t>(num_sms) * 16 * 2)
    while (p.score_heads < kScoreWarps && p.h_kv % (2 * p.score_heads) == 0) p.score_heads *= 2;
  // About two waves of four CTAs an SM.
  const int cta = kScoreBlocks * kScoreWarps / p.score_heads;
  const int64_t most = (blocks + cta - 1) / cta;
  const int64_t share = std::max<int64_t>(
      1, static_cast<int64_t>(num_sms) * 8 / (static_cast<int64_t>(p.batch) * (p.h_kv / p.score_heads)));
  p.score_ctas = static_cast<int>(std::min(most, share));
}

// The second kernel's CTAs to a sequence and KV head: a cluster of up to eight, while
// there are SMs for them and 1024 blocks for each.
void plan_choice(SelectParams& p, int blocks, int num_sms) {
  p.team = 1;
  p.cached_blocks = 0;
  if (blocks <= p.count || p.first + p.last == p.count) return;
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
