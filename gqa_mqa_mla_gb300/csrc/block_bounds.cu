// block_bounds.cu -- smallest and largest key of a cache block, per KV head and
// dimension: what a query's scores over the block are bounded by.
//
// For the block of tokens T (those before the sequence's end) and KV head j
//     lo_d = min_{t in T} k_td,   hi_d = max_{t in T} k_td,
// NaN in both where one of the keys is NaN.  Whole blocks are taken anew, so
// that a block whose tokens were given back or replaced needs no other care.
//
// Bound by the keys' bytes: one pass, a warp to a (block, head), whose lanes
// read 16-byte pieces of two (16-bit) or four (8-bit) token rows at once, eight
// loads in flight each; the warps of a CTA take neighbouring heads of a block,
// whose rows are neighbours in memory.  What the loads in flight can cover bounds
// it: 5.5 TB/s, 0.83 of the measured copy, at 171k tokens of 8 heads.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kAhead = 8;  // loads in flight per lane

// Two fp16 values that are e4m3 values (or NaN) to their codes, exactly.
DECATTN_DEV uint32_t f16x2_to_e4m3x2(uint32_t x) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(x));
  return c;
}

// kF8: e4m3 codes, compared as the fp16 values they stand for.
template <bool kF8, bool kBF16>
__global__ void __launch_bounds__(kThreads, 5) block_bounds_kernel(const BoundsParams p) {
  constexpr int kLanes = kF8 ? 8 : 16;         // lanes to a token row of 128 or 256 bytes
  constexpr int kRows = 32 / kLanes;           // token rows a load
  constexpr int kWords = kF8 ? 8 : 4;          // 16-bit pairs in 16 bytes
  constexpr uint32_t kInf = kBF16 && !kF8 ? 0x7f807f80u : 0x7c007c00u;
  __shared__ int64_t before[kThreads + 1];  // units of the sequences before each of a batch
  __shared__ int lens[kThreads], firsts[kThreads];
  __shared__ int64_t sums[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = lane & (kLanes - 1), row0 = lane / kLanes;
  const int lg = p.log2_block_size;
  const int64_t row_bytes = static_cast<int64_t>(p.h_kv) * kLanes * 16;
  const uint8_t* keys = static_cast<const uint8_t*>(p.k_cache);
  // The (block, head) units of 256 sequences at a time, numbered through and dealt
  // out to the grid's warps, so that sequences of any lengths load them alike.
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int mine = b0 + threadIdx.x;
    int64_t units = 0;
    if (mine < p.batch) {
      const int n = p.seq_lens[mine], first = p.first_lens ? p.first_lens[mine] : 0;
      const int from = min(first, n - 1) >> lg;
      if (n < 0 || n > p.max_seq_len || first < 0) {
        if (blockIdx.x == 0) flag_error(p.err_flag, kFlagBadSeqLen);
      } else if (n > 0) {
        units = static_cast<int64_t>(((n - 1) >> lg) + 1 - from) * p.h_kv;
      }
      lens[threadIdx.x] = n;
      firsts[threadIdx.x] = from;
    }
    int64_t upto = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += sums[w];
    before[threadIdx.x + 1] = upto;
    if (threadIdx.x == 0) before[0] = 0;
    __syncthreads();
    const int64_t all = before[kThreads], stride = static_cast<int64_t>(gridDim.x) * kWarps;
    // Unit u: its KV head, its block's id (-1: none, or a bad one) and that block's rows.
    auto look_up = [&](int64_t u, int& j, int& id, int& rows) {
      id = -1;
      if (u >= all) return;
      int lo_b = 0, hi_b = kThreads;  // the last sequence with before <= u
      while (hi_b - lo_b > 1) {
        const int mid = (lo_b + hi_b) >> 1;
        if (before[mid] <= u) lo_b = mid; else hi_b = mid;
      }
      const int k = static_cast<int>((u - before[lo_b]) / p.h_kv), lb = firsts[lo_b] + k;
      j = static_cast<int>(u - before[lo_b] - static_cast<int64_t>(k) * p.h_kv);
      rows = min(p.block_size, lens[lo_b] - (lb << lg));
      id = p.block_table[static_cast<int64_t>(b0 + lo_b) * p.max_blocks_per_seq + lb];
    };
    int j, id, rows, next_j = 0, next_id = -1, next_rows = 0;
    int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    look_up(u, next_j, next_id, next_rows);
    for (; u < all; u += stride) {
      j = next_j;
      id = next_id;
      rows = next_rows;
      look_up(u + stride, next_j, next_id, next_rows);  // (behind this unit's loads)
      if (id < 0 || id >= p.num_blocks) {
        if (lane == 0) flag_error(p.err_flag, kFlagBadBlock);
        continue;
      }
      const uint8_t* src = keys + static_cast<int64_t>(id) * p.block_size * row_bytes +
                           j * (kLanes * 16) + piece * 16;
      uint32_t lo[kWords], hi[kWords];
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        lo[k] = kInf;
        hi[k] = kInf | 0x80008000u;
      }
      for (int r0 = row0; r0 < rows; r0 += kRows * kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int r = min(r0 + a * kRows, rows - 1);  // (the last row again, for none)
          x[a] = *reinterpret_cast<const uint4*>(src + r * row_bytes);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const uint32_t w[4] = {x[a].x, x[a].y, x[a].z, x[a].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kF8) {
              uint32_t h0, h1;
              e4m3x4_to_f16x2(w[k], h0, h1);
              lo[2 * k] = min2<false>(lo[2 * k], h0);
              hi[2 * k] = max2<false>(hi[2 * k], h0);
              lo[2 * k + 1] = min2<false>(lo[2 * k + 1], h1);
              hi[2 * k + 1] = max2<false>(hi[2 * k + 1], h1);
            } else {
              lo[k] = min2<kBF16>(lo[k], w[k]);
              hi[k] = max2<kBF16>(hi[k], w[k]);
            }
          }
        }
      }
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          lo[k] = min2<kBF16 && !kF8>(lo[k], __shfl_xor_sync(0xffffffffu, lo[k], o));
          hi[k] = max2<kBF16 && !kF8>(hi[k], __shfl_xor_sync(0xffffffffu, hi[k], o));
        }
      }
      if (row0 < 2) {  // the first row's lanes write lo, the second's hi
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (kF8)
            out[k] = row0 ? f16x2_to_e4m3x2(hi[2 * k]) | f16x2_to_e4m3x2(hi[2 * k + 1]) << 16
                          : f16x2_to_e4m3x2(lo[2 * k]) | f16x2_to_e4m3x2(lo[2 * k + 1]) << 16;
          else
            out[k] = row0 ? hi[k] : lo[k];
        }
        uint8_t* dst = static_cast<uint8_t*>(p.bounds) +
                       ((static_cast<int64_t>(id) * 2 + row0) * p.h_kv + j) * (kLanes * 16) + piece * 16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
    __syncthreads();  // (the next sequences' numbers)
  }
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsParams& p, bool e4m3, bool bf16, int num_sms,
                                cudaStream_t stream) {
  // A warp to each (block, head) that there can be, up to two waves of five CTAs an SM
  // (4 prompts of 20-65k tokens: 45 us, one wave 46.5, with 8 CTAs of half the loads each 50).
  const int64_t blocks = (static_cast<int64_t>(p.max_seq_len) + p.block_size - 1) / p.block_size;
  const int64_t units = std::max<int64_t>(1, (blocks * p.h_kv * p.batch + kWarps - 1) / kWarps);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(units, static_cast<int64_t>(num_sms) * 10)));
  if (e4m3)
    block_bounds_kernel<true, false><<<grid, kThreads, 0, stream>>>(p);
  else if (bf16)
    block_bounds_kernel<false, true><<<grid, kThreads, 0, stream>>>(p);
  else
    block_bounds_kernel<false, false><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace decattn
