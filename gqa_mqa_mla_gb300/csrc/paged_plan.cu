// paged_plan.cu -- a serving step's paged state, built on the GPU from the
// requests' lengths: block tables, slot map, positions and row offsets.
//
// Request b holds c_b cached tokens in ceil(c_b / S) blocks (S = block size)
// and moves by n_b: n_b > 0 new tokens, n_b < 0 tokens taken back.  With
//   held_b = ceil(c_b / S), now_b = ceil((c_b + n_b) / S)
// it returns lost_b = max(0, held_b - now_b) blocks and needs need_b =
// max(0, now_b - held_b).  Three prefix sums over the requests (new tokens,
// needed and returned blocks) give every token its row, every returned block
// its place on the free stack and every needed block the entry it takes.
//
// Bound by latency: a step moves a few KB to a few hundred KB, so the cost
// is the launch and the chain load lengths -> scan -> load ids -> store.  One
// launch does it all, with no workspace: every CTA repeats the scan over all
// requests (a few KB, read from L2) and the rest is shared out by thread.
// A block that is given back and taken again in the same step is looked up in
// the row that gives it back, not on the stack, so no write is read again and
// the CTAs need not wait for one another -- except where the lengths or the
// free count are updated in place: then one CTA does a small step, and a
// cluster of eight, behind a barrier, a larger one.  Measured (replayed): 64
// requests with a token each 2.9 us, in place 3.4; 1024 mixed ones with 64k rows
// 6.3 us, in place 18.9.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMost = 0x7fffffff;

// Sums of non-negative counts stay at 2^31 - 1 once they reach it (a total
// beyond it is refused, so its exact value is not needed).
__device__ __forceinline__ int sat_add(int a, int b) {
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b),
                              static_cast<unsigned>(kMost)));
}

// Largest b in [0, n) with pre[b] <= i, for i < pre[n] (pre is an exclusive
// prefix sum): the request that owns the i-th token or block.
__device__ __forceinline__ int owner(const int* pre, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PlanParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ int sm[];
  const int B = p.batch, S = p.block_size, lg = p.log2_block_size;
  int* cached = sm;             // [B] c_b (0 for a request with bad lengths)
  int* moved = cached + B;      // [B] n_b (0 for a request with bad lengths)
  int* tok = moved + B;         // [B + 1] exclusive prefix of the new tokens
  int* need = tok + B + 1;      // [B + 1] of the needed blocks
  int* lost = need + B + 1;     // [B + 1] of the returned blocks
  __shared__ int tot[3][kWarps], upto[3][kWarps + 1];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  const int64_t room = static_cast<int64_t>(p.max_blocks_per_seq) * S;
  const int F = *p.free_count;

  int carry[3] = {0, 0, 0};
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    int c = 0, n = 0, v[3] = {0, 0, 0};
    if (b < B) {
      c = p.cached_lens[b];
      n = p.new_lens[b];
      const int64_t after = static_cast<int64_t>(c) + n;
      if (c < 0 || c > room || after < 0 || after > room) {
        if (blockIdx.x == 0) flag_error(p.err_flag, kFlagBadSeqLen);
        if (c < 0 || c > room) c = 0;
        n = 0;
      }
      const int held = static_cast<int>((static_cast<int64_t>(c) + S - 1) >> lg);
      const int now = static_cast<int>((static_cast<int64_t>(c) + n + S - 1) >> lg);
      v[0] = max(0, n);
      v[1] = max(0, now - held);
      v[2] = max(0, held - now);
      cached[b] = c;
      moved[b] = n;
    }
    int inc[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int up = __shfl_up_sync(kFull, inc[k], o);
        if (lane >= o) inc[k] = sat_add(inc[k], up);
      }
    }
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < 3; ++k) tot[k][warp] = inc[k];
    }
    __syncthreads();
    if (warp < 3) {  // a warp scans the warps' totals of one count: sums before each
      const int mine = lane < kWarps ? tot[warp][lane] : 0;
      int w = mine;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) {
        const int up = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w = sat_add(w, up);
      }
      if (lane < kWarps) upto[warp][lane + 1] = w;
      if (lane == 0) upto[warp][0] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      // Exclusive: the warps before this one, then the lanes before this one.
      int ex = __shfl_up_sync(kFull, inc[k], 1);
      if (lane == 0) ex = 0;
      ex = sat_add(carry[k], sat_add(upto[k][warp], ex));
      if (b < B) (k == 0 ? tok : k == 1 ? need : lost)[b] = ex;
      carry[k] = sat_add(carry[k], upto[k][kWarps]);
    }
    // (The next chunk of requests writes tot behind its own reads of upto, which
    // lie before the barrier that lets upto be written again.)
  }
  if (tid == 0) {
    tok[B] = carry[0];
    need[B] = carry[1];
    lost[B] = carry[2];
  }
  __syncthreads();

  // A free count outside the pool, or more returned blocks than the pool can
  // hold, is a broken pool: nothing moves.  A step that does not fit (blocks
  // or token rows) makes its trims, and no request grows.
  const int T = carry[0], A = carry[1], R = carry[2];
  const bool broken = F < 0 || F > p.num_blocks || R > p.num_blocks - F;
  const bool no_room = !broken && (A > F + R || T > p.max_tokens);
  const bool grows = !broken && !no_room;
  const bool trims = !broken;
  const int top = broken ? 0 : F + R;
  if (gtid == 0 && broken) flag_error(p.err_flag, kFlagBadBlock);
  if (gtid == 0 && no_room) flag_error(p.err_flag, kFlagNoRoom);

  // Returned blocks go onto the stack in request order, each request's in
  // ascending order: the i-th of them.
  auto row_of = [&](int b) { return p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq; };
  auto returned = [&](int i) {
    const int b = owner(lost, B, i);
    const int now = (cached[b] + moved[b] + S - 1) >> lg;
    return row_of(b)[now + i - lost[b]];
  };
  // Trims, growth and rows begin at different CTAs: each is a chain of a search and
  // dependent loads (1024 mixed requests 6.5 us, 7.3 with all at the first).
  const int half = gsize / 2, from_half = gtid >= half ? gtid - half : gtid + gsize - half;
  if (trims) {
    for (int i = from_half; i < R; i += gsize) {
      const int id = returned(i);
      if (id < 0 || id >= p.num_blocks) flag_error(p.err_flag, kFlagBadBlock);
      p.free_blocks[F + i] = id;
    }
  }
  // In place: every CTA has read the lengths and the free count behind this.
  if (p.in_place) cluster_sync();

  // The k-th needed block is the k-th from the top of the stack.
  auto fresh = [&](int k) {
    const int at = top - 1 - k;
    return at >= F ? returned(at - F) : p.free_blocks[at];
  };
  if (grows) {
    for (int k = gsize - 1 - gtid; k < A; k += gsize) {
      const int b = owner(need, B, k);
      const int held = static_cast<int>((static_cast<int64_t>(cached[b]) + S - 1) >> lg);
      const int id = fresh(k);
      if (id < 0 || id >= p.num_blocks) flag_error(p.err_flag, kFlagBadBlock);
      row_of(b)[held + k - need[b]] = id;
    }
  }
  const int live = grows ? T : 0;
  // (Unsigned: i may pass 2^31 behind the last row.)
  for (unsigned row = gtid; row < static_cast<unsigned>(p.max_tokens); row += gsize) {
    const int i = static_cast<int>(row);
    int slot = -1, pos = -1;
    if (i < live) {
      const int b = owner(tok, B, i);
      pos = cached[b] + i - tok[b];
      const int held = static_cast<int>((static_cast<int64_t>(cached[b]) + S - 1) >> lg);
      const int lb = pos >> lg;
      const int id = lb >= held ? fresh(need[b] + lb - held) : row_of(b)[lb];
      if (id >= 0 && id < p.num_blocks)
        slot = id * S + (pos & (S - 1));
      else
        flag_error(p.err_flag, kFlagBadBlock);
    }
    p.slots[i] = slot;
    p.positions[i] = pos;
  }
  for (int b = gtid; b <= B; b += gsize) {
    if (b < B) {
      const int n = moved[b];
      p.seq_lens[b] = cached[b] + ((n > 0 && grows) || (n < 0 && trims) ? n : 0);
    }
    p.q_start[b] = grows ? tok[b] : 0;
  }
  if (gtid == 0) *p.free_count_out = broken ? F : top - (grows ? A : 0);
}

template <int kThreads>
cudaError_t launch_t(const PlanParams& p, cudaStream_t stream) {
  auto kern = paged_plan_kernel<kThreads>;
  auto bytes = [](int batch) { return (5 * batch + 3) * static_cast<int>(sizeof(int)); };
  const int smem = bytes(p.batch);
  cudaError_t e = cudaSuccess;
  // The default limit of 48 KB is for static (under 1 KB) and dynamic shared memory
  // together.  What is asked for is always the largest batch's, so that a call of one
  // thread never lowers the limit that another has set for its launch.
  if (smem > 47 * 1024)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes(kPlanMaxBatch));
  if (e != cudaSuccess) return e;
  // A token a thread, up to a CTA on every other SM (more only repeat the
  // scan); a cluster's CTAs where the step is updated in place.
  const int by_rows = p.max_tokens / kThreads + 1;
  const int ctas = p.in_place ? (p.max_tokens <= 2048 ? 1 : 8) : std::max(1, std::min(by_rows, 64));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.in_place ? static_cast<unsigned>(ctas) : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t stream) {
  // Few requests and rows: a small CTA starts and meets sooner (64 requests with a
  // token each 3.0 us, 3.5 with 1024 threads; 256 with four 3.1 and 3.9).
  return p.batch <= 256 && p.max_tokens <= 1024 ? launch_t<256>(p, stream)
                                                : launch_t<1024>(p, stream);
}

}  // namespace decattn
