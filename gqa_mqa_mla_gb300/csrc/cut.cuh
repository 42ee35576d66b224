// cut.cuh -- the m largest of n keys by one CTA, and a list of some of n entries
// in order: shared by the block selection and the eviction.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace decattn {

// A float's bits as an unsigned key of the same order: -0 is 0, every NaN the
// largest key.
DECATTN_DEV uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 + 0 = 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
DECATTN_DEV uint64_t order_key(double x) {
  if (x != x) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u >> 63 ? ~u : u | 1ull << 63;
}

// What separates the m largest keys from the others: the keys above `key` are
// among them, and `ties` of those equal to it.
struct Cut {
  uint32_t key;
  int ties;
};

constexpr int kCutBins = 2048;
struct CutScratch {
  int bins[kCutBins];
  int sums[32];
  int digit, left;
};

// Radix selection from the top, 11, 11 and 10 bits a pass.  key(i, k) gives entry
// i's key and whether it takes part; 1 <= m <= the entries that do.  Keys share
// their upper bits, so a warp adds its equal digits up before it counts them
// in shared memory.  Called by all kThreads threads; ends behind a barrier.
template <int kThreads, class Key>
DECATTN_DEV Cut cut_largest(CutScratch& s, int n, int m, Key key) {
  constexpr int kOwn = kCutBins / kThreads;
  static_assert(kCutBins % kThreads == 0 && kThreads % 32 == 0, "bins per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0, mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) s.bins[tid + k * kThreads] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + tid;
      uint32_t k = 0;
      const bool on = i < n && key(i, k) && (k & mask) == prefix;
      const int digit = on ? static_cast<int>((k >> shift) & ((1u << bits) - 1)) : -1;
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      if (on && lane == __ffs(same) - 1) atomicAdd(&s.bins[digit], __popc(same));
    }
    __syncthreads();
    // Thread t owns the bins from kCutBins - 1 - t kOwn down; sums from the top.
    const int top = kCutBins - 1 - tid * kOwn;
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) mine += s.bins[top - k];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s.sums[warp] = upto;
    __syncthreads();
    int above = upto - mine;
    for (int w = 0; w < warp; ++w) above += s.sums[w];
    if (above < m && m <= above + mine) {
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const int c = s.bins[top - k];
        if (above < m && m <= above + c) {
          s.digit = top - k;
          s.left = m - above;
        }
        above += c;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s.digit) << shift;
    mask |= ((1u << bits) - 1) << shift;
    m = s.left;
  }
  return {prefix, m};
}

// Go through n entries in order: kind(i) is 0 (not listed), 1 (listed) or 2 (the
// first `ties` of these are listed); emit(i, rank) for each listed entry with its
// place in the list.  kind is asked twice.  counts: shared memory.
template <int kThreads>
struct ListScratch {
  int in[kThreads / 32], tied[kThreads / 32];
};
template <int kThreads, class Kind, class Emit>
DECATTN_DEV void list_in_order(ListScratch<kThreads>& s, int n, int ties, Kind kind, Emit emit) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int own = ((n + kThreads - 1) / kThreads) * 32;  // entries of a warp, in order
  const int begin = min(n, warp * own), end = min(n, begin + own);
  int in = 0, tied = 0;
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const int k = i < end ? kind(i) : 0;
    in += __popc(__ballot_sync(0xffffffffu, k == 1));
    tied += __popc(__ballot_sync(0xffffffffu, k == 2));
  }
  if (lane == 0) {
    s.in[warp] = in;
    s.tied[warp] = tied;
  }
  __syncthreads();
  in = tied = 0;
  for (int w = 0; w < warp; ++w) {
    in += s.in[w];
    tied += s.tied[w];
  }
  static_assert(kWarps <= 32, "warps of a CTA");
  const unsigned below = (1u << lane) - 1;
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const int k = i < end ? kind(i) : 0;
    const unsigned is_in = __ballot_sync(0xffffffffu, k == 1);
    const unsigned is_tied = __ballot_sync(0xffffffffu, k == 2);
    const int my_in = in + __popc(is_in & below), my_tied = tied + __popc(is_tied & below);
    if (k == 1 || (k == 2 && my_tied < ties)) emit(i, my_in + min(my_tied, ties));
    in += __popc(is_in);
    tied += __popc(is_tied);
  }
}

}  // namespace decattn
