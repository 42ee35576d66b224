// weigh.cuh -- attention weights of cached tokens, from the scores that a partial
// kernel kept and its splits' log-sum-exps:
//     w_t = (t was weighed before ? decay w_t : 0) + sum_i 2^(s_it - lse_i)
// over the query heads i of a KV head.  Bound by the scores' bytes, 4 a head and token
// beside K's and V's 512 a KV head and token (16-bit), which are read again soon
// after they were written (L2).
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace decattn {

// The group's log-sum-exps (log2 domain) over all splits into lse[0 .. group), a warp
// to four rows at a time: +inf where a split met bad data, -inf for an empty softmax,
// NaN for a row of NaN.  Partials may come from other CTAs: they are read from L2.
template <int kWarps>
DECATTN_DEV void weigh_lse(const GqaParams& p, size_t row0, float* lse) {
  constexpr float kInf = __builtin_huge_valf();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.group, ns = p.n_split;
  const float* part = p.part_lse + row0 * ns;
  if (ns == 1) {
    for (int r = threadIdx.x; r < G; r += kWarps * 32) lse[r] = __ldcg(part + r);
    return;
  }
  for (int r0 = warp; r0 < G; r0 += 4 * kWarps) {
    // Splits lane, lane + 32, ... of rows r0, r0 + kWarps, ...: up to 256.
    float v[4][2], mx[4], sum[4];
    bool bad[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      mx[q] = -kInf;
      sum[q] = 0.f;
      bad[q] = false;
    }
    for (int s0 = 0; s0 < ns; s0 += 64) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = r0 + q * kWarps, s = s0 + 32 * h + lane;
          v[q][h] = r < G && s < ns ? __ldcg(part + static_cast<size_t>(r) * ns + s) : -kInf;
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // (A lane's own maximum and sum; NaN is not a maximum but makes the sum NaN.)
        bad[q] |= v[q][0] == kInf || v[q][1] == kInf;
        const float m = fmaxf(mx[q], fmaxf(v[q][0], v[q][1]));
        const float base = m == -kInf ? 0.f : m;
        sum[q] = sum[q] * ex2(mx[q] - base) + ex2(v[q][0] - base) + ex2(v[q][1] - base);
        mx[q] = m;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float m = mx[q];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -kInf ? 0.f : m;
      float l = sum[q] * ex2(mx[q] - base);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const bool poison = __any_sync(0xffffffffu, bad[q]);
      if (lane == 0 && r0 + q * kWarps < G)
        lse[r0 + q * kWarps] = poison ? kInf : l == 0.f ? -kInf : m + lg2(l);
    }
  }
}

// kVec tokens from t on of sequence b and KV head j (1 or 4; blocks hold a multiple of
// 8): load() before the log-sum-exps are known, the slots' weights and the scores of
// the first kAhead heads; store() adds up.  A token's heads are added one after the
// other, always in the same order.
template <int kVec>
struct Weighed {
  static constexpr int kAhead = 8;
  float old[kVec], x[kAhead][kVec];
  float* at;
  const float* scores;

  DECATTN_DEV void head(int r, const GqaParams& p, float (&y)[kVec]) const {
    if constexpr (kVec == 4) {
      const float4 s = __ldcg(reinterpret_cast<const float4*>(scores + r * p.score_stride));
      y[0] = s.x; y[1] = s.y; y[2] = s.z; y[3] = s.w;
    } else {
      y[0] = __ldcg(scores + r * p.score_stride);
    }
  }
  DECATTN_DEV void load(const GqaParams& p, int j, int b, int t) {
    const int id = p.block_table[static_cast<size_t>(b) * p.max_blocks_per_seq + (t >> p.log2_block_size)];
    scores = p.scores + (static_cast<size_t>(b) * p.h_q + static_cast<size_t>(j) * p.group) * p.score_stride + t;
#pragma unroll
    for (int r = 0; r < kAhead; ++r)
      if (r < p.group) head(r, p, x[r]);
    // (A bad id, of a sequence whose log-sum-exps will say so, is not followed.)
    at = id < 0 || id >= p.num_blocks
             ? nullptr
             : p.weights + (static_cast<int64_t>(id) * p.h_kv + j) * p.block_size + (t & (p.block_size - 1));
    if (at) {
      if constexpr (kVec == 4) {
        const float4 w = *reinterpret_cast<const float4*>(at);
        old[0] = w.x; old[1] = w.y; old[2] = w.z; old[3] = w.w;
      } else {
        old[0] = *at;
      }
    }
  }
  DECATTN_DEV void store(const GqaParams& p, int t, int n, int weighed, const float* lse) {
    constexpr float kInf = __builtin_huge_valf();
    float sum[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum[k] = 0.f;
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      if (r >= p.group) break;
      const float l = lse[r];
#pragma unroll
      for (int k = 0; k < kVec; ++k) sum[k] += l != -kInf ? ex2(x[r][k] - l) : 0.f;
    }
#pragma unroll 8
    for (int r = kAhead; r < p.group; ++r) {
      float y[kVec];
      head(r, p, y);
      const float l = lse[r];
#pragma unroll
      for (int k = 0; k < kVec; ++k) sum[k] += l != -kInf ? ex2(y[k] - l) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      if (t + k < weighed) sum[k] = fmaf(p.decay, old[k], sum[k]);
    if (kVec == 4 && t + 3 < n) {
      *reinterpret_cast<float4*>(at) = make_float4(sum[0], sum[kVec > 1 ? 1 : 0], sum[kVec > 2 ? 2 : 0],
                                                   sum[kVec > 3 ? 3 : 0]);
    } else {  // (slots past the sequence stay as they are)
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (t + k < n) at[k] = sum[k];
    }
  }
};

}  // namespace decattn
