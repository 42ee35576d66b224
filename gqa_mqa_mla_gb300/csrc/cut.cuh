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
constexpr int kCutFew = 64;  // keys that are ranked against one another
struct CutScratch {
  int bins[kCutBins];
  int sums[32];
  uint32_t few[kCutFew];
  uint32_t lo, hi;
  int bin, left, count, gathered;
};

// The keys' range is divided into 2048 bins of equal width (keys of floats: equal
// ratios, or equal steps where they are alike), counted, and the bin of the m-th
// largest found; the bin's keys are then ranked directly if they are few, else
// their range is divided again (each time by 1024 at least, so at most four
// times).  One counting and one collecting pass where the keys are spread: with
// 32768 weights a third of the time of three radix passes, whose upper digits few
// values share.  A value that many lanes of a warp hold is counted once for all.
// key(i, k) gives entry i's key and whether it takes part; 1 <= m <= the entries
// that do.  Called by all kThreads threads; ends behind a barrier.
template <int kThreads, class Key>
DECATTN_DEV Cut cut_largest(CutScratch& s, int n, int m, Key key) {
  constexpr int kOwn = kCutBins / kThreads;
  static_assert(kCutBins % kThreads == 0 && kThreads % 32 == 0 && kThreads >= kCutFew, "bins");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s.lo = 0xffffffffu;
    s.hi = 0u;
  }
  __syncthreads();
  uint32_t lo = 0xffffffffu, hi = 0u;
  for (int i = tid; i < n; i += kThreads) {
    uint32_t k = 0;
    if (key(i, k)) {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    atomicMin(&s.lo, lo);
    atomicMax(&s.hi, hi);
  }
  __syncthreads();
  lo = s.lo;
  hi = s.hi;
  __syncthreads();  // (all have read before a next call writes)
  while (lo < hi) {
    const uint32_t range = hi - lo;
    // Key k falls into bin floor((k - lo) scale / 2^32), or k - lo.
    const bool direct = range < kCutBins;
    const uint32_t scale =
        direct ? 0u : static_cast<uint32_t>((static_cast<uint64_t>(kCutBins) << 32) / (range + 1ull));
#pragma unroll
    for (int k = 0; k < kOwn; ++k) s.bins[tid + k * kThreads] = 0;
    if (tid == 0) s.gathered = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + tid;
      uint32_t k = 0;
      const bool on = i < n && key(i, k) && k >= lo && k <= hi;
      const unsigned some = __ballot_sync(0xffffffffu, on);
      if (some == 0) continue;
      const int bin = static_cast<int>(direct ? k - lo : __umulhi(k - lo, scale));
      const int lead = __ffs(some) - 1;
      const int common = __shfl_sync(0xffffffffu, bin, lead);
      const unsigned same = __ballot_sync(0xffffffffu, on && bin == common);
      if (lane == lead) atomicAdd(&s.bins[common], __popc(same));
      if (on && bin != common) atomicAdd(&s.bins[bin], 1);
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
    int above = upto - mine + __reduce_add_sync(0xffffffffu, lane < warp ? s.sums[lane] : 0);
    if (above < m && m <= above + mine) {
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const int c = s.bins[top - k];
        if (above < m && m <= above + c) {
          s.bin = top - k;
          s.left = m - above;
          s.count = c;
        }
        above += c;
      }
    }
    __syncthreads();
    const uint32_t bin = static_cast<uint32_t>(s.bin);
    const int count = s.count;
    m = s.left;
    if (direct) {
      lo = hi = lo + bin;
      break;
    }
    // The bin's keys: from the first that falls into it to the last.
    auto from = [&](uint32_t b) {
      return ((static_cast<uint64_t>(b) << 32) + scale - 1) / scale;
    };
    const uint64_t next = lo + from(bin + 1) - 1;
    lo += static_cast<uint32_t>(from(bin));
    hi = next < hi ? static_cast<uint32_t>(next) : hi;
    if (count <= kCutFew) {
      for (int i = tid; i < n; i += kThreads) {
        uint32_t k = 0;
        if (key(i, k) && k >= lo && k <= hi) s.few[atomicAdd(&s.gathered, 1)] = k;
      }
      __syncthreads();
      if (tid < count) {
        const uint32_t k = s.few[tid];
        int more = 0, equal = 0;
        for (int c = 0; c < count; ++c) {
          more += s.few[c] > k;
          equal += s.few[c] == k;
        }
        if (more < m && m <= more + equal) {  // (the same for all of these)
          s.lo = k;
          s.left = m - more;
        }
      }
      __syncthreads();
      const Cut c = {s.lo, s.left};
      __syncthreads();
      return c;
    }
    __syncthreads();  // (s.bin, s.left and s.count are read before they are written again)
  }
  return {lo, m};
}

// Go through n entries in order: kind(i) is 0 (not listed), 1 (listed) or 2 (the
// first `ties` of these are listed); emit(i, rank) for each listed entry with its
// place in the list.  A warp takes a run of entries: it counts them, and when all
// have, gives out their places; lane s keeps what it saw in step s (of the first 32,
// then kind is asked again).
template <int kThreads>
struct ListScratch {
  int in[32], tied[32];
};
template <int kThreads, class Kind, class Emit>
DECATTN_DEV void list_in_order(ListScratch<kThreads>& s, int n, int ties, Kind kind, Emit emit) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 32, "warps of a CTA");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int steps = (n + kThreads - 1) / kThreads;  // of a warp's run
  const int begin = warp * steps * 32;
  auto look = [&](int st, unsigned& in, unsigned& tied) {
    const int i = begin + st * 32 + lane;
    const int k = i < n ? kind(i) : 0;
    in = __ballot_sync(0xffffffffu, k == 1);
    tied = __ballot_sync(0xffffffffu, k == 2);
  };
  int in = 0, tied = 0;
  unsigned kept_in = 0, kept_tied = 0;
  for (int st = 0; st < steps; ++st) {
    unsigned a, b;
    look(st, a, b);
    if (lane == st) {
      kept_in = a;
      kept_tied = b;
    }
    in += __popc(a);
    tied += __popc(b);
  }
  if (lane == 0) {
    s.in[warp] = in;
    s.tied[warp] = tied;
  }
  __syncthreads();
  in = __reduce_add_sync(0xffffffffu, lane < warp ? s.in[lane] : 0);
  tied = __reduce_add_sync(0xffffffffu, lane < warp ? s.tied[lane] : 0);
  const unsigned me = 1u << lane, below = me - 1;
  for (int st = 0; st < steps; ++st) {
    unsigned a = __shfl_sync(0xffffffffu, kept_in, st & 31);
    unsigned b = __shfl_sync(0xffffffffu, kept_tied, st & 31);
    if (st >= 32) look(st, a, b);
    const int my_in = in + __popc(a & below), my_tied = tied + __popc(b & below);
    if ((a & me) || ((b & me) && my_tied < ties))
      emit(begin + st * 32 + lane, my_in + min(my_tied, ties));
    in += __popc(a);
    tied += __popc(b);
  }
}

}  // namespace decattn
