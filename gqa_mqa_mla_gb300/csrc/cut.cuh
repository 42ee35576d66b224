// cut.cuh -- the m largest of n keys by a CTA, or by the CTAs of a cluster, and a list
// of some of n entries in order: shared by the block selection and the eviction.
//
// With few sequences and KV heads a long row would leave most SMs idle: the CTAs of a
// cluster then take a slice of its entries each, and read one another's counts
// through distributed shared memory (128 of one sequence's 8192 blocks for 8 KV heads:
// 33 us with clusters of four and a flushed L2, 36 with a CTA each).
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace decattn {

// A float's bits as an unsigned key of the same order: -0 is 0, every NaN the
// largest key.
DECATTN_DEV uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 + 0 = 0)
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return x != x ? 0xffffffffu : k;
}
DECATTN_DEV uint64_t order_key(double x) {
  if (x != x) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u >> 63 ? ~u : u | 1ull << 63;
}
// The float of a key.
DECATTN_DEV float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The CTAs that share the entries: one, or a cluster (along x).
template <bool kCluster>
struct Team {
  DECATTN_DEV static void sync() {
    if constexpr (kCluster) {
      __syncwarp();  // (the cluster's barrier is for whole warps)
      cluster_sync();
    } else {
      __syncthreads();
    }
  }
  DECATTN_DEV static int size() { return kCluster ? static_cast<int>(gridDim.x) : 1; }
  DECATTN_DEV static int rank() { return kCluster ? static_cast<int>(blockIdx.x) : 0; }
  // Variable x of the team's CTA r (a word of shared memory).
  template <class T>
  DECATTN_DEV static T get(const T& x, int r) {
    static_assert(sizeof(T) == 4, "a word");
    if constexpr (kCluster) {
      uint32_t v;
      asm volatile("ld.shared::cluster.u32 %0, [%1];"
                   : "=r"(v)
                   : "r"(mapa_shared(smem_u32(&x), static_cast<uint32_t>(r)))
                   : "memory");
      return static_cast<T>(v);
    } else {
      return x;
    }
  }
  // The words x[0 .. kN) of all CTAs added up, this one's first (so that the CTAs do
  // not all read the same one at a time), 16 or 8 bytes a load, all in flight.
  template <int kN>
  DECATTN_DEV static void add_up(const int* x, int (&sum)[kN]) {
    static_assert(kN == 2 || kN == 4, "one load");
    if constexpr (kCluster) {
#pragma unroll
      for (int k = 0; k < kN; ++k) sum[k] = 0;
      const uint32_t at = smem_u32(x);
      int v[8][kN];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r >= size()) break;
        const uint32_t from = mapa_shared(at, static_cast<uint32_t>((rank() + r) % size()));
        if constexpr (kN == 4)
          asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[r][0]), "=r"(v[r][1]), "=r"(v[r][2]), "=r"(v[r][3])
                       : "r"(from)
                       : "memory");
        else
          asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                       : "=r"(v[r][0]), "=r"(v[r][1])
                       : "r"(from)
                       : "memory");
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r >= size()) break;
#pragma unroll
        for (int k = 0; k < kN; ++k) sum[k] += v[r][k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k) sum[k] = x[k];
    }
  }
  // The first CTA's x[i] = v, with i counted up in its `n`; places from `most` on are
  // counted but not written.
  template <class T>
  DECATTN_DEV static void push(T* x, int* n, int most, T v) {
    if constexpr (kCluster) {
      const uint32_t count = mapa_shared(smem_u32(n), 0), to = mapa_shared(smem_u32(x), 0);
      uint32_t i;
      asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(i) : "r"(count) : "memory");
      if (i < static_cast<uint32_t>(most))
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 4 * i),
                     "r"(static_cast<uint32_t>(v))
                     : "memory");
    } else {
      const int i = atomicAdd(n, 1);
      if (i < most) x[i] = v;
    }
  }
};

// What separates the m largest keys from the others: the keys above `key` are
// among them, and `ties` of those equal to it.
struct Cut {
  uint32_t key;
  int ties;
};

constexpr int kCutBins = 2048;
constexpr int kCutFew = 64;  // keys that are ranked against one another
struct CutScratch {
  __align__(16) int bins[kCutBins];
  int sums[32];
  uint32_t few[kCutFew], own[kCutFew];
  uint32_t lo, hi;  // between calls: an empty range
  int gathered;
  int bin, left, count;
};

// Before the first call (a barrier of the CTA has to follow).
DECATTN_DEV void cut_prepare(CutScratch& s) {
  if (threadIdx.x == 0) {
    s.lo = 0xffffffffu;
    s.hi = 0u;
    s.gathered = 0;
  }
}

// The keys' range is divided into up to 2048 bins of equal width, a power of two (keys
// of floats: equal ratios, or equal steps where they are alike), counted, and the bin
// of the m-th largest found; the bin's keys are then ranked directly if they are few,
// else their range is divided again (each time by 1024 at least, so at most four
// times).  One counting and one collecting pass where the keys are spread, against
// three counting ones by digits, whose upper digits few values share.  A value that
// many lanes of a warp hold is counted once for all.
// key(i, k) gives entry i's key (of this CTA's n) and whether it takes part; lo, hi:
// the range of the keys that this thread has looked at (all are by the team's
// threads; empty: lo > hi), or kKnown: that of the team's keys; 1 <= m <= the team's
// entries that take part.  Called by all kThreads threads of each CTA; ends behind a
// barrier.
template <int kThreads, bool kCluster, bool kKnown, class Key>
DECATTN_DEV Cut cut_largest(CutScratch& s, uint32_t lo, uint32_t hi, int n, int m, Key key) {
  using T = Team<kCluster>;
  constexpr int kOwn = kCutBins / kThreads;
  static_assert(kCutBins % kThreads == 0 && kThreads % 32 == 0 && kThreads >= kCutFew, "bins");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) s.bins[tid + k * kThreads] = 0;
  if constexpr (kKnown) {
    __syncthreads();
  } else {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&s.lo, lo);
      atomicMax(&s.hi, hi);
    }
    T::sync();
    if constexpr (kCluster) {
      if (warp == 0) {
        lo = lane < T::size() ? T::get(s.lo, lane) : 0xffffffffu;
        hi = lane < T::size() ? T::get(s.hi, lane) : 0u;
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
          s.own[0] = lo;
          s.own[1] = hi;
        }
      }
      __syncthreads();
      lo = s.own[0];
      hi = s.own[1];
    } else {
      lo = s.lo;
      hi = s.hi;
    }
  }
  while (lo < hi) {
    // Key k falls into bin (k - lo) >> shift.
    const int shift = max(0, 21 - __clz(hi - lo));
#pragma unroll 2
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + tid;
      uint32_t k = 0;
      const bool on = i < n && key(i, k) && k >= lo && k <= hi;
      const unsigned some = __ballot_sync(0xffffffffu, on);
      if (some == 0) continue;
      const int bin = static_cast<int>((k - lo) >> shift);
      const int lead = __ffs(some) - 1;
      const int common = __shfl_sync(0xffffffffu, bin, lead);
      const unsigned same = __ballot_sync(0xffffffffu, on && bin == common);
      if (lane == lead) atomicAdd(&s.bins[common], __popc(same));
      if (on && bin != common) atomicAdd(&s.bins[bin], 1);
    }
    T::sync();
    // Thread t owns the bins from kCutBins - kOwn - t kOwn up; sums from the top.
    const int first = kCutBins - kOwn - tid * kOwn;
    int each[kOwn], mine = 0;
    T::add_up(s.bins + first, each);
#pragma unroll
    for (int k = 0; k < kOwn; ++k) mine += each[k];
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
      for (int k = kOwn - 1; k >= 0; --k) {
        if (above < m && m <= above + each[k]) {
          s.bin = first + k;
          s.left = m - above;
          s.count = each[k];
        }
        above += each[k];
      }
    }
    __syncthreads();
    const int count = s.count;
    m = s.left;
    lo += static_cast<uint32_t>(s.bin) << shift;
    if (hi - lo >= 1u << shift) hi = lo + ((1u << shift) - 1);
    if (lo == hi) break;
    if (count <= kCutFew) {
      for (int i = tid; i < n; i += kThreads) {
        uint32_t k = 0;
        if (key(i, k) && k >= lo && k <= hi) T::push(s.few, &s.gathered, kCutFew, k);
      }
      T::sync();
      if (tid < count) s.own[tid] = T::get(s.few[tid], 0);
      __syncthreads();
      if (tid < count) {
        const uint32_t k = s.own[tid];
        int more = 0, equal = 0;
#pragma unroll 8
        for (int c = 0; c < count; ++c) {
          more += s.own[c] > k;
          equal += s.own[c] == k;
        }
        if (more < m && m <= more + equal) {  // (the same for all of these)
          s.bin = static_cast<int>(k);
          s.left = m - more;
        }
      }
      __syncthreads();
      lo = static_cast<uint32_t>(s.bin);
      m = s.left;
      break;
    }
    T::sync();  // (the bins have been read everywhere)
#pragma unroll
    for (int k = 0; k < kOwn; ++k) s.bins[tid + k * kThreads] = 0;
    __syncthreads();
  }
  T::sync();  // (nothing of this call is read any more)
  cut_prepare(s);
  __syncthreads();
  return {lo, m};
}

// Go through the team's entries in order, this CTA's n behind those of the CTAs before
// it: kind(i, again) is 0 (out), 1 (in) or 2 (tied); settle(in, tied) is told the team's totals
// (by all threads, behind a barrier); emit(i, tied?, in before, tied before) sees each
// entry that is not out, with the numbers of the team's entries before it.  Returns the
// entries in and tied of the CTAs before this one, and this one's.  A warp takes a run
// of entries: it counts them, and when all have, goes through them again; lane s
// keeps what it saw in step s (of the first 32, then kind is asked again).
struct ListScratch {
  int in[32], tied[32];
  int all_in, all_tied;
};
template <int kThreads, bool kCluster, class Kind, class Settle, class Emit>
DECATTN_DEV int4 list_in_order(ListScratch& s, int n, Kind kind, Settle settle, Emit emit) {
  using T = Team<kCluster>;
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 32, "warps of a CTA");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int steps = (n + kThreads - 1) / kThreads;  // of a warp's run
  const int begin = warp * steps * 32;
  unsigned kept_in = 0, kept_tied = 0;
  int in = 0, tied = 0;
#pragma unroll 2
  for (int st = 0; st < steps; ++st) {
    const int i = begin + st * 32 + lane;
    const int k = i < n ? kind(i, false) : 0;
    const unsigned a = __ballot_sync(0xffffffffu, k == 1), b = __ballot_sync(0xffffffffu, k == 2);
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
  int in_here = lane < kWarps ? s.in[lane] : 0, tied_here = lane < kWarps ? s.tied[lane] : 0;
  in = __reduce_add_sync(0xffffffffu, lane < warp ? in_here : 0);
  tied = __reduce_add_sync(0xffffffffu, lane < warp ? tied_here : 0);
  in_here = __reduce_add_sync(0xffffffffu, in_here);
  tied_here = __reduce_add_sync(0xffffffffu, tied_here);
  int in_before = 0, tied_before = 0, in_all = in_here, tied_all = tied_here;
  if constexpr (kCluster) {
    if (threadIdx.x == 0) {
      s.all_in = in_here;
      s.all_tied = tied_here;
    }
    T::sync();
    const int a = lane < T::size() ? T::get(s.all_in, lane) : 0;
    const int b = lane < T::size() ? T::get(s.all_tied, lane) : 0;
    in_all = __reduce_add_sync(0xffffffffu, a);
    tied_all = __reduce_add_sync(0xffffffffu, b);
    in_before = __reduce_add_sync(0xffffffffu, lane < T::rank() ? a : 0);
    tied_before = __reduce_add_sync(0xffffffffu, lane < T::rank() ? b : 0);
    in += in_before;
    tied += tied_before;
  }
  settle(in_all, tied_all);
  const unsigned me = 1u << lane, below = me - 1;
  for (int st = 0; st < steps; ++st) {
    unsigned a = __shfl_sync(0xffffffffu, kept_in, st & 31);
    unsigned b = __shfl_sync(0xffffffffu, kept_tied, st & 31);
    const int i = begin + st * 32 + lane;
    if (st >= 32) {
      const int k = i < n ? kind(i, true) : 0;
      a = __ballot_sync(0xffffffffu, k == 1);
      b = __ballot_sync(0xffffffffu, k == 2);
    }
    if ((a | b) & me) emit(i, (b & me) != 0, in + __popc(a & below), tied + __popc(b & below));
    in += __popc(a);
    tied += __popc(b);
  }
  if constexpr (kCluster) T::sync();  // (a CTA that others read stays until they have)
  return make_int4(in_before, tied_before, in_here, tied_here);
}

// The list of the entries in and of the first `ties` of those tied: emit(i, its place).
// Returns the first place of this CTA's entries and the one behind its last.
template <int kThreads, bool kCluster, class Kind, class Emit>
DECATTN_DEV int2 list_largest(ListScratch& s, int n, int ties, Kind kind, Emit emit) {
  const int4 c = list_in_order<kThreads, kCluster>(
      s, n, kind, [](int, int) {},
      [&](int i, bool tied, int in_before, int tied_before) {
        if (!tied || tied_before < ties) emit(i, in_before + min(tied_before, ties));
      });
  return make_int2(c.x + min(c.y, ties), c.x + c.z + min(c.y + c.w, ties));
}

}  // namespace decattn
