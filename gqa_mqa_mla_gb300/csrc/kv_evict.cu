// kv_evict.cu -- a cache keeps its heaviest and its latest tokens: per sequence
// and KV head, the choice by accumulated attention weight, and the move of what
// stays to the front of the sequence, in order.
//
// A sequence of n > limit tokens keeps, of its first n - recent, the keep -
// recent with the largest weights (ties: the earlier token; NaN is largest), and
// its last `recent`.  Entry r of the list of kept positions is the token that
// moves to position r.
//
// Two launches.  The first, a CTA or a cluster to each sequence and KV head, brings the
// weights into shared memory (the cut and the list go over them several times), cuts,
// lists, and moves the weights themselves.  The second moves K and V: a kept position
// is never before its place (the list ascends), so a CTA that loads a run of rows,
// meets, stores it and goes on to the next run overwrites no row that is still to be
// read, and CTAs that take different columns of the rows need not know of one another.
// Bound by the moved rows' bytes, read and written once.
#include <algorithm>

#include "cut.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr int kThreads = 1024;
constexpr int kCachedTokens = 53248;  // weights that shared memory holds (208 KB)

template <bool kCluster>
__global__ void __launch_bounds__(kThreads) evict_rank_kernel(const EvictParams p) {
  using T = Team<kCluster>;
  extern __shared__ __align__(16) float cached[];
  __shared__ CutScratch cut;
  __shared__ ListScratch list;
  launch_dependents();
  const int j = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int lg = p.log2_block_size, in_block = p.block_size - 1;
  int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.h_kv + j) * p.keep;
  const int n = p.seq_lens[b];
  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  bool stays = n <= p.limit;
  if (n < 0 || n > p.max_seq_len) {
    if (tid == 0 && j == 0 && T::rank() == 0) flag_error(p.err_flag, kFlagBadSeqLen);
    stays = true;
  }
  float* weights = p.weights + static_cast<int64_t>(j) * p.block_size;
  const int64_t block_stride = static_cast<int64_t>(p.h_kv) * p.block_size;
  auto slot = [&](int t) { return weights + bt[t >> lg] * block_stride + (t & in_block); };
  // This CTA's tokens: [begin, begin + own), of which the first `old` may go.
  const int slice = stays ? 0 : ((n + T::size() - 1) / T::size() + 3) & ~3;
  const int begin = min(n, T::rank() * slice), own = min(slice, n - begin);
  const int all_old = n - p.recent, old = max(0, min(own, all_old - begin)), heavy = p.keep - p.recent;
  const bool cache = kCluster || own <= p.cached_tokens;
  uint32_t lo = 0xffffffffu, hi = 0u;
  if (!stays) {
    cut_prepare(cut);
    int bad = 0;
    // Four tokens (of one block) at a time, all of a thread's loads in flight.
#pragma unroll 4
    for (int i = tid * 4; i < own; i += kThreads * 4) {
      const int t = begin + i, id = bt[t >> lg];
      const bool wrong = id < 0 || id >= p.num_blocks;
      bad |= wrong;
      if (wrong) continue;
      const float4 w = *reinterpret_cast<const float4*>(weights + id * block_stride + (t & in_block));
      if (cache) *reinterpret_cast<float4*>(cached + i) = w;
      const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i + k < old) {
          lo = min(lo, order_key(x[k]));
          hi = max(hi, order_key(x[k]));
        }
      }
    }
    // (Every CTA of a team sees the whole table's verdict: they go on together.)
    if constexpr (kCluster) {
      for (int k = tid; k <= (n - 1) >> lg; k += kThreads) bad |= bt[k] < 0 || bt[k] >= p.num_blocks;
    }
    if (__syncthreads_or(bad)) {
      if (tid == 0) flag_error(p.err_flag, kFlagBadBlock);
      stays = true;
    }
  }
  if (stays) {
    for (int r = T::rank() * kThreads + tid; r < p.keep; r += T::size() * kThreads) kept[r] = -1;
    if (tid == 0 && j == 0 && T::rank() == 0) p.new_lens[b] = 0;
    return;
  }
  auto weight = [&](int i) { return cache ? cached[i] : *slot(begin + i); };
  int2 places = make_int2(0, 0);  // of this CTA's heavy tokens in the list
  if (heavy > 0) {
    const Cut c = cut_largest<kThreads, kCluster, false>(cut, lo, hi, old, heavy, [&](int i, uint32_t& k) {
      k = order_key(weight(i));
      return true;
    });
    places = list_largest<kThreads, kCluster>(list, old, c.ties, [&](int i, bool) {
      const uint32_t k = order_key(weight(i));
      return k > c.key ? 1 : k == c.key ? 2 : 0;
    }, [&](int i, int r) { kept[r] = begin + i; });
  } else {
    T::sync();  // (every weight has been read before the first is written)
  }
  if (tid == 0 && j == 0 && T::rank() == 0) p.new_lens[b] = p.keep - n;
  const int latest = max(0, all_old - begin);  // the first of this CTA's that is among the last
  for (int i = latest + tid; i < own; i += kThreads) {
    const int r = heavy + begin + i - all_old;
    kept[r] = begin + i;
    if (cache) *slot(r) = cached[i];
  }
  __syncthreads();
  if (cache) {
#pragma unroll 4
    for (int r = places.x + tid; r < places.y; r += kThreads) *slot(r) = cached[kept[r] - begin];
  } else {  // (one CTA) in runs, as the rows are moved
    for (int r0 = 0; r0 < p.keep; r0 += kThreads) {
      const int r = r0 + tid;
      const float w = r < p.keep ? *slot(kept[r]) : 0.f;
      __syncthreads();
      if (r < p.keep) *slot(r) = w;
    }
  }
}

constexpr int kMoveThreads = 256;
constexpr int kAhead = 8;  // 16-byte pieces a thread holds

// A CTA moves some columns (2^lg_pieces 16-byte pieces of a head's row) of K or V, in runs
// of as many rows as its threads hold; a run's places are looked up (through the list
// and the table) while the rows of the run before are on their way.
__global__ void __launch_bounds__(kMoveThreads, 3) evict_move_kernel(const EvictParams p, int lg_pieces) {
  wait_for_dependence();  // the list is there
  const int j = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.h_kv + j) * p.keep;
  if (kept[0] < 0) return;  // nothing is evicted
  const int parts = gridDim.x / 2;
  const bool is_v = static_cast<int>(blockIdx.x) >= parts;
  const int part = blockIdx.x - (is_v ? parts : 0);
  const int lg = p.log2_block_size, in_block = p.block_size - 1;
  const int64_t row_bytes = static_cast<int64_t>(p.h_kv) * p.head_bytes;
  const int piece = tid & ((1 << lg_pieces) - 1), row = tid >> lg_pieces;
  uint8_t* cache = (is_v ? p.v_cache : p.k_cache) + j * p.head_bytes + ((part << lg_pieces) + piece) * 16;
  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  auto place = [&](int t) { return (bt[t >> lg] << lg) + (t & in_block); };  // the row, < 2^31
  const int step = kMoveThreads >> lg_pieces;  // rows of one load
  int from[kAhead], to[kAhead];  // (-1: the row stays where it is, or there is none)
  auto look_up = [&](int r0) {
    int t[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int r = r0 + a * step + row;
      t[a] = r < p.keep ? kept[r] : r;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int r = r0 + a * step + row;
      from[a] = t[a] != r ? place(t[a]) : -1;
      to[a] = t[a] != r ? place(r) : -1;
    }
  };
  look_up(0);
  for (int r0 = 0; r0 < p.keep; r0 += step * kAhead) {
    uint4 x[kAhead];
    int at[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      at[a] = to[a];
      if (at[a] >= 0) x[a] = *reinterpret_cast<const uint4*>(cache + from[a] * row_bytes);
    }
    if (r0 + step * kAhead < p.keep) look_up(r0 + step * kAhead);
    __syncthreads();
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (at[a] >= 0) *reinterpret_cast<uint4*>(cache + at[a] * row_bytes) = x[a];
  }
}

}  // namespace

template <bool kCluster>
static cudaError_t launch_rank(const EvictParams& p, cudaStream_t stream) {
  const size_t smem = (static_cast<size_t>(p.cached_tokens) + 3) / 4 * 4 * sizeof(float);
  if (smem > 36 * 1024) {  // (beside static shared memory, of 48 KB)
    const cudaError_t e = cudaFuncSetAttribute(evict_rank_kernel<kCluster>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kCachedTokens * static_cast<int>(sizeof(float)));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.team), static_cast<unsigned>(p.h_kv),
                     static_cast<unsigned>(p.batch));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.team);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_rank_kernel<kCluster>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_evict(EvictParams p, int num_sms, cudaStream_t stream) {
  // A cluster of up to eight CTAs to a sequence and KV head, while there are SMs for
  // them and 4096 tokens for each (2 x 30-32k tokens, 8 KV heads: 28 us, 39 with 2048),
  // or their shared memory is needed; past that one CTA reads the weights from global
  // memory.
  const int64_t units = static_cast<int64_t>(p.batch) * p.h_kv;
  p.team = 1;
  while (p.team < 8 && ((units * p.team * 2 <= num_sms && p.max_seq_len >= 2 * p.team * 4096) ||
                        p.max_seq_len > p.team * kCachedTokens))
    p.team *= 2;
  if (p.max_seq_len > p.team * (kCachedTokens - 4)) p.team = 1;
  p.cached_tokens = std::min((p.max_seq_len + p.team - 1) / p.team + 3, kCachedTokens);
  cudaError_t e = p.team > 1 ? launch_rank<true>(p, stream) : launch_rank<false>(p, stream);
  if (e != cudaSuccess) return e;
  // 128 bytes of a row to a CTA (64 sequences, a fifth of them cut to 4096 tokens of 8
  // heads: 93 us, 101 with 64 bytes), or 32 where that fills no wave.
  const int64_t rows = static_cast<int64_t>(p.batch) * p.h_kv * 2;
  const int lg_pieces = rows * (p.head_bytes / 64) < num_sms * 4 ? 1 : 3;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (p.head_bytes >> (4 + lg_pieces))),
                     static_cast<unsigned>(p.h_kv), static_cast<unsigned>(p.batch));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_move_kernel, p, lg_pieces);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
