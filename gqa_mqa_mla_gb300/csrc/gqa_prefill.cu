// gqa_prefill.cu -- attention of a chunk of new tokens per sequence over a
// paged KV cache (MHA / GQA / MQA), on tcgen05 / TMEM, sm_103a.
//
// Row (i, h) of sequence b, position p = L - n + i, sees cache positions
// t <= p (with a window W and S kept first tokens: t > p - W or t < S):
//     out = sum_t e^{s_t} v_t / sum_t e^{s_t},   s_t = scale q . k_t.
// The G = h_q / h_kv query heads of a KV head read the same cache rows, so a
// Q tile packs floor(128 / G) tokens x G heads into the 128 rows of an MMA,
// and a CTA works on two such tiles (A: the first tokens, B: the next ones)
// of one KV head, against the same 128-token K and V tiles:
//     S_X = Q_X K^T   128 x 128 x 128        X = A, B
//     O_X += P_X V    128 x 128 x 128
// Bound by the tensor cores and their operands' path once a chunk has a few
// hundred rows per KV head: each 64 KB pair of K and V tiles serves 2 x 2 groups
// of eight MMAs (2^21 products), each 512 cycles at the nominal rate, 629 at
// cuBLAS's best, and moves 256 KB through shared memory (S takes both operands
// from there); measured 3100 cycles a pair, a group being issued in 650 to 700, with
// the softmax warps waiting half of the time (an 8192-token prompt of 64 heads on 8:
// 720 us, 1.53 PFLOP/s, 0.78 of cuBLAS's burst).  S in halves of 64 tokens ahead of
// the softmax moves 320 KB and takes a fifth longer: the bytes are the bound.
// Bound by HBM below that: 32 chunks of 8 tokens over 8k caches take 169 us, 6.4
// TB/s.  Few rows over a long cache are cut along the cache (n_split) and joined by
// a log-sum-exp combine: one chunk of 8 tokens over 131k tokens 94 us, 5.7 TB/s.
//
// Operand placement:
//   Q_A, Q_B   shared memory [2 halves][128 rows][128 B], 128-byte swizzle,
//              by TMA (a 3-D box: 64 columns x G heads x tokens)   A of S
//   K, V       one TMA ring of four 32 KB slots, K(0) V(0) K(1) V(1) ...,
//              [2 halves][128 tokens][128 B], 128-byte swizzle, one box per
//              half and cache block         K: B of S;  V: B of P V (MN-major)
//   out        32 KB in which a warp turns its rows' lanes into whole lines
//   S_X, P_X   TMEM, 128 fp32 columns; P_X (16-bit, 64 columns) over S_X  A of P V
//   O_X        TMEM, 128 fp32 columns
// (2 x (128 + 128) columns: all of TMEM, one CTA per SM.)
//
// Warps (384 threads):
//   0-3, 4-7  softmax of tile A, of tile B: a thread owns a row (TMEM lane),
//             so no value of a row is ever exchanged: running maximum, lazy
//             rescale of O, P, running sum; epilogue;
//   8, 10     TMA producers of Q and K, of V (they walk the block table and
//             check the block ids); 8 is the scheduler too (below);
//   9         MMA issuer: P_A V, S_A of the next tile, P_B V, S_B of the next
//             tile: while one tile's softmax runs, the tensor cores work on
//             the other's products.  MMAs of one thread run in order, so
//             S_A(j + 1) may overwrite P_A(j) right behind its last reader;
//   11        TMEM allocation.
//
// A CTA stays on its SM and goes from piece to piece (two Q tiles of one
// sequence and KV head): the scheduler takes over CTAs of the grid that have
// not started (cluster launch control) while the present piece is worked on,
// so the next one's Q, K and V are on their way, and its first S is computed,
// during the softmax warps' epilogue.  Pieces come longest first.
//
// A piece with one Q tile (few rows: drafted tokens, single tokens, a chunk's
// rest) would leave the second set of softmax warps idle and every tile's chain
// of product, softmax and product uncovered.  There (`solo`) both sets work on
// the same rows, A on the even K / V tiles, B on the odd ones, with S, P and O
// of their own, joined at the end (32 chunks of 8 tokens
// over 8k caches, 64 heads on 8, when this was added: 187 us instead of 203).
//
// An 8-bit (e4m3) cache takes the same pipeline with four changes: the K tile's
// codes, as they land, are the B operand of S on kind::f8f6f4, whose A operand is
// Q as two (bf16) or three (fp16) e4m3 terms that the softmax warps make of their
// rows; warps 10 and 11 convert each V tile to fp16; P is fp16; K's scale and
// Q's row exponents join the score scale, V's scale the final division.  (With K
// converted too, a tile took 4800 cycles, bound by the conversion; shared memory
// is what a converter waits for: the MMAs' operands take most of its bandwidth.)
#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr int kM = 128;                        // rows of a Q tile
constexpr int kKv = 128;                       // tokens of a K / V tile
constexpr int kHalf = 128 * 128;               // 64 columns x 128 rows, 16 KB
constexpr int kTileBytes = 2 * kHalf;          // 32 KB
constexpr int kRing = 4;
constexpr int kOffRing = 2 * kTileBytes;       // behind Q_A, Q_B
constexpr int kOffStage = kOffRing + kRing * kTileBytes;
constexpr int kCodeBytes = kTileBytes / 2;     // a tile, or a term of Q, in e4m3 codes
constexpr int kStageBytes = 32 * 128;          // one softmax warp's: 32 rows x 128 B
constexpr int kOffBars = kOffStage + 8 * kStageBytes;
constexpr int kOffMerge = kOffBars + 1024;     // 128 rows' (maximum, sum), see `solo`
constexpr int kSmemBytes = 1024 + kOffMerge + 128 * 8;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

constexpr int kThreads = 384;
// (8-bit cache: warp 8 loads K and V, 10 and 11 convert them.)
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpV = 10, kWarpTmem = 11;
constexpr int kTmemS = 0;                      // S_X: 128 X
constexpr int kTmemO = 256;                    // O_X: 256 + 128 X
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kRescaleThreshold = 8.0f;      // log2 units: P stays <= 2^8

enum : int {
  kBarQ = 0,                    // Q tiles landed
  kBarQFree = 1,                // every S of the piece computed
  kBarFull = 2,                 // ring slot landed
  kBarEmpty = kBarFull + kRing, // ring slot free
  kBarS = kBarEmpty + kRing,    // 2: S_X computed
  kBarP = kBarS + 2,            // 2 x 2: P_X, tokens 0-63 and 64-127, written (128 arrivals)
  kBarO = kBarP + 4,            // 2: O_X complete
  kBarItem = kBarO + 2,         // 2: piece published
  kBarItemFree = kBarItem + 2,  // 2: piece done by every other role
  kBarNext = kBarItemFree + 2,  // the launch control's answer
  kBarFull16 = kBarNext + 1,    // 8-bit cache, 2: fp16 V tile converted (64 arrivals)
  kBarEmpty16 = kBarFull16 + 2, // 8-bit cache, 2: fp16 V tile free
  kBarPair = kBarEmpty16 + 2,   // 4: the two softmax warps of the same rows (solo)
  kBarDrain = kBarPair + 4,
  kNumBars = kBarDrain + 1
};

// Behind the barriers, in the same kilobyte.
constexpr int kOffWords = kOffBars + 288;   // abort, bad, copies made by the producers, TMEM
constexpr int kOffAnswer = kOffBars + 352;  // the launch control's answer, 16 bytes
constexpr int kOffItems = kOffBars + 416;   // two pieces
constexpr int kOffQExp = kOffBars + 640;    // 8-bit cache: Q's row exponents, 2 x 128 bytes
static_assert(kNumBars * 8 <= 288, "barriers");

// A piece of work: rows of one sequence and KV head against a range of tiles.
struct Item {
  int valid;        // 0: no more pieces
  int j, split;
  int n, len;       // chunk length, cache length
  int b, q0;        // sequence, its first packed row
  int i0;           // first token of the chunk in tile A
  int tok_a, tok_b; // tokens in tile A, B
  int lo, s_end, base, sink_tiles;
  int hi;           // one past the last position any row sees
  int tile0;        // first tile of this split
  int n_a, n_b;     // tiles that tile A, B need, from tile0 on
  int gap0, gap1;   // tiles [gap0, gap1) lie before tile B's window (A's only)
  int solo;         // one Q tile: the warps of tile B take every other K / V tile
  int bad;
};
static_assert(2 * sizeof(Item) <= 640 - 416, "items");

struct Tile {
  int t0, skip, nval;  // rows [skip, nval) hold tokens that may be seen
};

__device__ __forceinline__ Tile tile_of(const Item& w, int it) {
  const int vt = w.tile0 + it;
  const bool sink = vt < w.sink_tiles;
  Tile r;
  r.t0 = sink ? vt * kKv : w.base + (vt - w.sink_tiles) * kKv;
  r.skip = sink ? 0 : max(0, w.lo - r.t0);
  r.nval = min(kKv, (sink ? w.s_end : w.hi) - r.t0);
  return r;
}

// Offsets (in tokens, from this split's first tile) of the window's first
// token and of the sequence's end as tile_of counts them: the tiles at
// [full_lo, full_hi) have no row outside [skip, nval) (sinks' tiles left out).
__device__ __forceinline__ int win0_of(const Item& w) {
  return w.base + (w.tile0 - w.sink_tiles) * kKv;
}
__device__ __forceinline__ int full_lo(const Item& w) {
  return max(w.lo - win0_of(w), w.s_end - w.tile0 * kKv);
}
__device__ __forceinline__ int full_hi(const Item& w) { return w.hi - win0_of(w); }

template <bool kValue>
struct Const {
  __device__ constexpr operator bool() const { return kValue; }
};

// Number of tiles up to and including the one that holds position `last`.
__device__ __forceinline__ int tiles_to(const Item& w, int last) {
  return last < w.base ? 0 : w.sink_tiles + (last - w.base) / kKv + 1;
}

// By how many tokens a chunk's first piece is shorter than the others (which
// follow it without a gap).  A piece's tiles start at the block boundary before its
// first row's window, and rounded down so 128 rows of a window of 1024 need ten
// tiles instead of nine; pieces whose windows start at a boundary do not.  Not
// where a tile is no whole number of blocks, or where it would take one more piece.
// (4 chunks of 1500 to 2048 tokens, window 1024, 32 heads: 136 us, 144 with equal
// pieces.)
__device__ __forceinline__ int shorter_by(const PrefillParams& p, int n, int len) {
  const int tpi = 2 * p.tokens_per_tile, step = min(p.block_size, kKv);
  if (p.window <= 0 || p.tokens_per_tile % step != 0) return 0;
  const int s = static_cast<int>((static_cast<uint32_t>(len) - n + 1u - p.window) & (step - 1));
  return (n + s + tpi - 1) / tpi > (n + tpi - 1) / tpi ? 0 : s;
}

// Are sequence b's row offsets a, e = q_start[b], q_start[b + 1] those of a chunk?
__device__ __forceinline__ bool rows_fit(const PrefillParams& p, int a, int e) {
  return a >= 0 && e >= a && e <= p.tokens && e - a <= p.max_q_len;
}

// Walks the pieces, 32 sequences at a time (one per lane), from the last sequences
// back.  Among the 32 the longest come first (a piece of two Q tiles counts
// double), and within a chunk the last rows, which see most: what is left for the
// end is short.  (32 chunks of 1 to 8 tokens over 4 to 8k, 64 heads on 8: 131 us,
// 142 in the batch's order.)
struct Cursor {
  int b0;      // the lanes hold sequences b0 .. b0 + 31
  int before;  // pieces behind those sequences
  int start, n, len, cnt, pre;  // this lane's sequence; pre: pieces of those before it
  int all;                      // pieces of the 32
};

__device__ __forceinline__ void load_cursor(const PrefillParams& p, Cursor& c, int lane) {
  const int b = c.b0 + lane, tpi = 2 * p.tokens_per_tile;
  c.cnt = c.n = c.start = c.len = 0;
  if (b >= 0 && b < p.batch) {
    const int a = p.q_start[b], e = p.q_start[b + 1];
    c.len = p.seq_lens[b];
    if (rows_fit(p, a, e)) {
      c.start = a;
      c.n = e - a;
      c.cnt = (e - a + tpi - 1) / tpi;
    }
  }
  c.all = __reduce_add_sync(0xffffffffu, c.cnt);
  c.pre = 0;
  // (A grid of one wave starts all of its pieces at once: any order will do.)
  const uint32_t key = p.steal ? static_cast<uint32_t>(c.len) << (c.n > p.tokens_per_tile) : 0u;
  for (int j = max(0, -c.b0); j < 32; ++j) {
    const uint32_t other = __shfl_sync(0xffffffffu, key, j);
    const int pieces = __shfl_sync(0xffffffffu, c.cnt, j);
    if (other > key || (other == key && j > lane)) c.pre += pieces;
  }
}

// The index-th piece (all lanes; index counts from the end); false if there
// are not that many.
__device__ __forceinline__ bool find_item(const PrefillParams& p, Cursor& c, int index, Item& w) {
  const int lane = threadIdx.x & 31;
  if (index < c.before) {  // (launch control hands out later pieces; be safe)
    c.b0 = p.batch - 32;
    c.before = 0;
    load_cursor(p, c, lane);
  }
  for (;;) {
    if (index < c.before + c.all) break;
    if (c.b0 <= 0) return false;
    c.before += c.all;
    c.b0 -= 32;
    load_cursor(p, c, lane);
  }
  const int at = index - c.before;
  const bool mine = at >= c.pre && at < c.pre + c.cnt;
  const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  const int tpi = 2 * p.tokens_per_tile;
  w.valid = 1;
  w.b = c.b0 + src;
  w.q0 = __shfl_sync(0xffffffffu, c.start, src);
  w.n = __shfl_sync(0xffffffffu, c.n, src);
  w.len = __shfl_sync(0xffffffffu, c.len, src);
  const int cnt = __shfl_sync(0xffffffffu, c.cnt, src), pre = __shfl_sync(0xffffffffu, c.pre, src);
  const int end = (cnt - (at - pre)) * tpi - shorter_by(p, w.n, w.len);
  w.i0 = max(0, end - tpi);
  const int tok = min(w.n, end) - w.i0;
  w.tok_a = min(p.tokens_per_tile, tok);
  w.tok_b = tok - w.tok_a;
  w.bad = w.len < 0 || w.len > p.max_seq_len;
  if (w.bad) {
    if (lane == 0) flag_error(p.err_flag, kFlagBadSeqLen);
    w.len = 0;
  }
  // Positions of the first and last rows, and the tiles that they see: with
  // a window those of [0, s_end) (kept first tokens before the window of the
  // first row), then those from the window's block boundary on.  Kept tokens
  // that reach the window join it.
  const int p_first = w.len - w.n + w.i0;
  const int p_last = p_first + w.tok_a + w.tok_b - 1;
  w.hi = max(0, min(w.len, p_last + 1));
  w.lo = p.window > 0 && p_first >= p.window ? p_first + 1 - p.window : 0;
  if (p.sinks >= w.lo) w.lo = 0;
  w.lo = min(w.lo, w.hi);
  w.s_end = min(p.sinks, w.lo);
  w.base = w.lo & ~(min(p.block_size, kKv) - 1);
  w.sink_tiles = (w.s_end + kKv - 1) / kKv;
  const int total = w.bad ? 0 : tiles_to(w, w.hi - 1);
  const int total_a = w.bad ? 0 : max(0, min(total, tiles_to(w, p_first + w.tok_a - 1)));
  const int per = (total + p.n_split - 1) / p.n_split;
  w.tile0 = min(total, w.split * per);
  w.n_a = max(0, min(per, total_a - w.tile0));
  w.n_b = w.tok_b > 0 ? min(per, total - w.tile0) : 0;
  w.solo = w.tok_b == 0 && w.n_a >= 2;
  // With a window, the first window tiles may lie before every row of tile B.
  const int before_b = w.lo > 0 ? (p_first + w.tok_a + 1 - p.window - w.base) / kKv : 0;
  w.gap0 = max(0, min(w.n_b, w.sink_tiles - w.tile0));
  w.gap1 = max(w.gap0, min(w.n_b, w.sink_tiles + before_b - w.tile0));
  if (w.gap1 == w.n_b) {  // nothing behind the gap (in this split)
    w.n_b = w.gap0;
    w.gap0 = w.gap1 = 0;
  }
  return true;
}

// The lowest n bits set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(0xffffffffu), "r"(max(n, 0)));  // clamps at 32
  return ~r;
}

// A warp's 32 rows of 128 bytes (eight 16-byte pieces, one row per thread)
// go through its own 4 KB of shared memory, so that eight lanes store a row's
// whole line: piece c of row r lies at place c ^ (r % 8) of its row.
__device__ __forceinline__ uint4* staged(uint8_t* stage, int row, int c) {
  return reinterpret_cast<uint4*>(stage + row * 128 + ((c ^ (row & 7)) << 4));
}

// 32 rows of a Q tile as sums of kTerms e4m3 values of row r times alpha_r = 2^k
// (the largest power of two with max |q_r| alpha_r <= 448): t1 = e4m3(x), t2 =
// e4m3(x - t1), ...  Each remainder is a multiple of the query's own last bit
// no larger than half of the term's step, so two terms hold a bf16 query and
// three an fp16 one exactly, but for parts up to 2^-10 (half of e4m3's smallest
// step) of the scaled row, whose largest value is above 224.  Term t of the tile:
// [128 rows][128 codes], 128-byte swizzle; k goes to qexp[r].  16 lanes take a row,
// 8 values each; of the 32 rows the pairs [b0, b1) are this warp's, as far as they
// are real (the others may hold anything).
template <bool kBF16, int kTerms>
__device__ __forceinline__ void split_q(const PrefillParams& p, const Item& w, int x, int part,
                                        int b0, int b1, uint32_t inv_g, uint8_t* dst, int8_t* qexp) {
  const int lane = threadIdx.x & 31, c = lane & 15;
  const int rows = (x ? w.tok_b : w.tok_a) * p.group;
  const uint16_t* src =
      static_cast<const uint16_t*>(p.q) +
      (static_cast<int64_t>(w.q0 + w.i0 + x * p.tokens_per_tile) * p.h_q + w.j * p.group) * kHeadDim +
      8 * c;
  // The group's next four rows are on their way while four are split.
  auto load = [&](int b, uint4 (&y)[4]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = 32 * part + 2 * (b + u) + (lane >> 4);
      const int tk = static_cast<int>((static_cast<uint32_t>(r) * inv_g) >> 16);
      y[u] = b < b1 && r < rows
                 ? *reinterpret_cast<const uint4*>(
                       src + static_cast<int64_t>(tk * (p.h_q - p.group) + r) * kHeadDim)
                 : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 y[4], ahead[4];
  b1 = min(b1, (rows - 32 * part + 1) >> 1);
  load(b0, y);
#pragma unroll 1
  for (int b = b0; b < b1; b += 4) {
    load(b + 4, ahead);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = 32 * part + 2 * (b + u) + (lane >> 4);
      float v[8];
      const uint32_t in[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<kBF16>(in[k]);
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      }
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[k]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t bits = __float_as_uint(m);
      const int ex = static_cast<int>((bits >> 23) & 0xffu) - 127;
      const int k2 = min(max(((bits & 0x7fffffu) <= 0x600000u ? 8 : 7) - ex, -126), 126);
      // (An infinite value has no such terms: all of its row's become NaN.)
      const float alpha =
          __uint_as_float(bits == 0x7f800000u ? 0x7fc00000u : static_cast<uint32_t>(k2 + 127) << 23);
      if (c == 0) qexp[r] = static_cast<int8_t>(k2);
      uint32_t code[kTerms][2] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a0 = v[2 * k] * alpha, a1 = v[2 * k + 1] * alpha;
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
          float r0, r1;
          code[t][k >> 1] |= e4m3_round2(a0, a1, r0, r1) << (16 * (k & 1));
          a0 -= r0;
          a1 -= r1;
        }
      }
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
        *reinterpret_cast<uint2*>(dst + t * kCodeBytes + r * 128 + (((c >> 1) ^ (r & 7)) << 4) +
                                  (c & 1) * 8) = make_uint2(code[t][0], code[t][1]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = ahead[u];
  }
}

// kF8: the cache holds e4m3 codes with per-KV-head scales.
template <bool kBF16, bool kF8>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  constexpr bool kMmaBF16 = kBF16 && !kF8;  // operand type of the 16-bit products
  // 8-bit cache: a bf16 query is two e4m3 terms, an fp16 one three; behind Q
  // the ring of codes, then what is left below the staging for fp16 V tiles.
  constexpr int kTerms = kBF16 ? 2 : 3;
  constexpr int kRingAt = kF8 ? 2 * kTerms * kCodeBytes : kOffRing;
  constexpr int kV16At = kRingAt + kRing * kCodeBytes;
  constexpr int kV16 = (kOffStage - kV16At) / kTileBytes;
  static_assert(!kF8 || (kV16 >= 1 && kV16 <= 2), "fp16 V tiles");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + kOffBars;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  volatile int* abort_word = reinterpret_cast<volatile int*>(smem + kOffWords);
  volatile int* bad_word = abort_word + 1;  // 2: a piece met a bad block id
  volatile int* made_by = abort_word + 3;   // copies made by the K and V producers, Q loads
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffWords + 32);
  Item* items = reinterpret_cast<Item*>(smem + kOffItems);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;

  if (threadIdx.x == 0) {
    mbar_init(bar(kBarQ), kF8 ? 256 : 1);  // the copies, or every softmax thread
    mbar_init(bar(kBarQFree), 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), kF8 && (s & 1) ? 2 : 1);  // (V codes: two converters)
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(kBarS + x), 1);
      mbar_init(bar(kBarP + x), kM);
      mbar_init(bar(kBarP + 2 + x), kM);
      mbar_init(bar(kBarO + x), 1);
      mbar_init(bar(kBarItem + x), 1);
      // V producer or the two converters, MMA, softmax
      mbar_init(bar(kBarItemFree + x), kF8 ? 11 : 10);
      mbar_init(bar(kBarFull16 + x), 64);
      mbar_init(bar(kBarEmpty16 + x), 1);
    }
    mbar_init(bar(kBarNext), 1);
    for (int x = 0; x < 4; ++x) mbar_init(bar(kBarPair + x), 64);
    mbar_init(bar(kBarDrain), 1);
    for (int k = 0; k < 6; ++k) abort_word[k] = 0;
    fence_barrier_init();
  }
  if (warp == kWarpTmem) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // The scheduler looks for its first piece meanwhile.
  Cursor cursor;
  Item first;
  // Grid index: KV heads of a piece, then its splits, then pieces.
  auto find = [&](int x, Item& w) -> bool {
    const int rest = x / p.h_kv, item = rest / p.n_split;
    w.j = x - rest * p.h_kv;
    w.split = rest - item * p.n_split;
    return find_item(p, cursor, item, w);
  };
  if (warp == kWarpLoad) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    cursor.b0 = p.batch - 32;
    cursor.before = 0;
    load_cursor(p, cursor, lane);
    first.valid = find(static_cast<int>(blockIdx.x), first);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The k-th piece, as every role sees it (all lanes of its warp); released
  // once the role is done with it.
  auto get_item = [&](int k, Item& w) -> bool {
    if (!mbar_wait_or_abort_warp(bar(kBarItem + (k & 1)), (k >> 1) & 1, p.err_flag, abort_word))
      return false;
    w = items[k & 1];
    return w.valid != 0;
  };
  auto release_item = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarItemFree + (k & 1)));
  };

  if (warp >= 8) {
    if (warp == kWarpLoad || (!kF8 && warp == kWarpV)) {
      // ---------------- TMA producers: one warp for Q and K, one for V (two
      // streams of boxes; a warp gets a small box accepted about every 100
      // cycles); over an 8-bit cache, with half the boxes, one warp for all.
      // Warp 8 also is the scheduler: it publishes each piece when it begins
      // to load it.
      const bool lead = warp == kWarpLoad;
      // A cache that only one piece of each sequence and KV head reads (few rows)
      // streams through L2; otherwise its tiles are kept for the next piece.
      // (32 chunks of 8 tokens over 8k caches, when this was added: 180 us, 187 with
      // tiles kept.)
      const uint64_t keep = p.once ? policy_evict_first() : policy_evict_last();
      const int bs = p.block_size, lg = p.log2_block_size;
      constexpr int kBytes = kF8 ? kCodeBytes : kTileBytes;  // of a tile
      // K(it) is the ring's copy 2 it, V(it) the copy 2 it + 1, counted over
      // all pieces: slot and phase parity of this warp's next one, and the
      // numbers it made.
      int slot = lead ? 0 : 1, made_k = 0, made_v = 0, q_loads = 0;
      uint32_t phase = 0;
      int x = blockIdx.x, asks = 0;
      // Takes over a CTA that has not started: its index in x, or -1.  Asked
      // for once the last copies of a piece are on their way, about two tiles
      // ahead (at the piece's start it would be kept from CTAs that run out
      // sooner: 256 pieces of 1 to 64 tiles took 146 us that way, 112 so).  A
      // grid of one wave has none to hand over.
      auto claim = [&]() -> bool {
        x = -1;
        if (!p.steal) return true;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kBarNext), 16);
          clc_try_cancel(sbase + kOffAnswer, bar(kBarNext));
        }
        __syncwarp();
        if (!mbar_wait_or_abort_warp(bar(kBarNext), asks++ & 1, p.err_flag, abort_word))
          return false;
        x = clc_answer(sbase + kOffAnswer);
        fence_proxy_async_smem();  // the answer is read before the next one is asked for
        return true;
      };
      bool ok = true;
      Item w;
      for (int k = 0; ok; ++k) {
        if (lead) {
          bool some = k == 0 && first.valid;
          if (some) {
            w = first;
          } else {
            if (k == 0) ok = claim();
            while (ok && x >= 0 && !some) {
              some = find(x, w);
              if (!some) ok = claim();
            }
          }
          w.valid = some;
          if (lane == 0 && ok) {
            ok = mbar_wait_or_abort(bar(kBarItemFree + (k & 1)), ((k >> 1) & 1) ^ 1, p.err_flag,
                                    abort_word);
            if (ok) {
              bad_word[k & 1] = 0;
              items[k & 1] = w;
              mbar_arrive(bar(kBarItem + (k & 1)));
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok || !some) break;
        } else if (!get_item(k, w)) {
          break;
        }
        const int n = max(w.n_a, w.n_b);
        if (!kF8 && n > 0 && lead) {
          if (lane == 0) {
            ok = mbar_wait_or_abort(bar(kBarQFree), (q_loads & 1) ^ 1, p.err_flag, abort_word);
            if (ok) {
              const int tiles = w.tok_b > 0 ? 2 : 1;
              mbar_arrive_expect_tx(
                  bar(kBarQ), static_cast<uint32_t>(tiles * 2 * p.tokens_per_tile * G * 128));
              for (int q = 0; q < tiles; ++q)
                for (int h = 0; h < 2; ++h)
                  tma_load_3d(sbase + q * kTileBytes + h * kHalf, &tm_q, 64 * h, w.j * G,
                              w.q0 + w.i0 + q * p.tokens_per_tile, bar(kBarQ));
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          if (ok) made_by[2] = ++q_loads;
        }
        const int32_t* bt = p.block_table + static_cast<size_t>(w.b) * p.max_blocks_per_seq;
        const int x0 = w.j * kHeadDim;  // element (= byte, of an 8-bit cache) column of head j
        const int kb_end = ((w.hi - 1) >> lg) + 1;
        int cache0 = -(1 << 30), my_id = 0;
        for (int it = 0; ok && it < n; ++it) {
          const Tile t = tile_of(w, it);
          const int kb0 = t.t0 >> lg;
          const int nblk = bs >= kKv ? 1 : (t.nval + bs - 1) >> lg;
          // The lanes hold the ids of the next 32 blocks (read ahead of use).
          if (kb0 + nblk > cache0 + 32) {
            cache0 = kb0;
            my_id = kb0 + lane < kb_end ? bt[kb0 + lane] : 0;
          }
          int id = __shfl_sync(0xffffffffu, my_id, kb0 - cache0 + min(lane, nblk - 1));
          if (id < 0 || id >= p.num_blocks) {
            // Copy block 0 instead; the rows become zeros.
            id = 0;
            bad_word[k & 1] = 1;
            flag_error(p.err_flag, kFlagBadBlock);
          }
          const int row = id * bs + (bs >= kKv ? (t.t0 & (bs - 1)) : 0);
          const uint32_t bytes =
              static_cast<uint32_t>(bs >= kKv ? kBytes : nblk * bs * (kF8 ? 128 : 256));
#pragma unroll 1
          for (int kv = lead ? 0 : 1; ok && kv < (kF8 || !lead ? 2 : 1); ++kv) {
            if (lane == 0) {
              ok = mbar_wait_or_abort(bar(kBarEmpty + slot), phase ^ 1u, p.err_flag, abort_word);
              if (ok) mbar_arrive_expect_tx(bar(kBarFull + slot), bytes);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane < nblk) {
              const CUtensorMap* tm = kv ? &tm_v : &tm_k;
              const uint32_t dst =
                  sbase + kRingAt + slot * kBytes + static_cast<uint32_t>(lane * bs * 128);
              tma_load_2d_hint(dst, tm, x0, row, bar(kBarFull + slot), keep);
              if (!kF8) tma_load_2d_hint(dst + kHalf, tm, x0 + 64, row, bar(kBarFull + slot), keep);
            }
            if (kv)
              ++made_v;
            else
              ++made_k;
            slot += kF8 ? 1 : 2;
            if (slot >= kRing) {
              slot -= kRing;
              phase ^= 1u;
            }
          }
        }
        if (ok && lead) ok = claim();
        if (ok && !lead) release_item(k);
      }
      if (lane == 0) {
        if (kF8 || lead) made_by[0] = made_k;
        if (kF8 || !lead) made_by[1] = made_v;
      }
      __syncwarp();
    } else if (kF8 && (warp == kWarpV || warp == kWarpTmem)) {
      // ---------------- converters (8-bit cache): each V tile's [128 tokens][128
      // codes] to fp16 [2 halves][128 tokens][128 B], both with 128-byte swizzle,
      // warp 10 the first 64 tokens, 11 the others; e4m3 -> fp16 is exact.  Rows
      // outside [skip, nval) become zeros (their slots may hold NaN codes).
      const int part = warp == kWarpV ? 0 : 1;
      int c = 0;  // tiles, over all pieces
      bool ok = true;
      Item w;
      for (int k = 0; ok && get_item(k, w); ++k) {
        const int n = max(w.n_a, w.n_b), full_from = full_lo(w), full_to = full_hi(w);
        for (int it = 0; it < n; ++it, ++c) {
          const int from = (2 * c + 1) % kRing, to = c % kV16;
          ok = mbar_wait_or_abort(bar(kBarFull + from), (2 * c / kRing) & 1, p.err_flag,
                                  abort_word) &&
               mbar_wait_or_abort(bar(kBarEmpty16 + to), (c / kV16 & 1) ^ 1, p.err_flag, abort_word);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          int lo = 0, hi = kKv;
          if (it * kKv < full_from || it * kKv + kKv > full_to) {
            const Tile t = tile_of(w, it);
            lo = t.skip;
            hi = t.nval;
          }
          const uint8_t* src = smem + kRingAt + from * kCodeBytes;
          // Lane: 16 codes e = lane % 8 of rows lane / 8, + 4, ...; its two
          // output pieces are 2 (e % 4) and the next one of half e / 4, the
          // odd one first for e >= 4 (no bank is hit twice).
          const int e = lane & 7, odd = e >> 2, e0 = 2 * (e & 3);
          uint8_t* dst = smem + kV16At + to * kTileBytes + odd * kHalf;
          // (Eight rows are read before any is written: a load does not pass a
          // store to shared memory by itself.)
#pragma unroll 1
          for (int r0 = 64 * part + (lane >> 3); r0 < 64 * part + 64; r0 += 32) {
            uint4 y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int r = r0 + 4 * u;
              y[u] = *reinterpret_cast<const uint4*>(src + r * 128 + ((e ^ (r & 7)) << 4));
            }
            if (lo > 0 || hi < kKv) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                if (r0 + 4 * u < lo || r0 + 4 * u >= hi) y[u] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int r = r0 + 4 * u;
              uint4 a, b;
              e4m3x4_to_f16x2(y[u].x, a.x, a.y);
              e4m3x4_to_f16x2(y[u].y, a.z, a.w);
              e4m3x4_to_f16x2(y[u].z, b.x, b.y);
              e4m3x4_to_f16x2(y[u].w, b.z, b.w);
              uint8_t* o = dst + r * 128;
              *reinterpret_cast<uint4*>(o + (((e0 + odd) ^ (r & 7)) << 4)) = odd ? b : a;
              *reinterpret_cast<uint4*>(o + (((e0 + 1 - odd) ^ (r & 7)) << 4)) = odd ? a : b;
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(kBarFull16 + to));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarEmpty + from));
        }
        if (ok) release_item(k);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ---------------- MMA issuer: the whole warp runs the loop, lane 0
      // waits, one elected lane issues.
      const uint64_t dq = smem_desc_sw128(sbase, 16, 1024);
      const uint64_t dk = smem_desc_sw128(sbase + kRingAt, 16, 1024);
      const uint64_t dv = smem_desc_sw128(sbase + (kF8 ? kV16At : kOffRing), kHalf, 1024);
      constexpr uint32_t idesc_s =
          kF8 ? idesc_e4m3(kM, kKv) : idesc_f16(kMmaBF16, kM, kKv, false, false);
      constexpr uint32_t idesc_o = idesc_f16(kMmaBF16, kM, kHeadDim, false, true);
      // All lanes probe; lane 0 waits where that does not succeed at once.
      auto wait = [&](int bi, uint32_t parity) -> bool {
        bool g = mbar_try_wait(bar(bi), parity);
        if (!__all_sync(0xffffffffu, g)) {
          if (lane == 0) g = mbar_wait_or_abort(bar(bi), parity, p.err_flag, abort_word);
          g = __shfl_sync(0xffffffffu, g ? 1 : 0, 0) != 0;
        }
        tc_fence_after();
        return g;
      };
      // S_X = Q_X K^T (Q tile q): eight k-steps of 16 dims, four per 64-column
      // half; 8-bit: for each term of Q four k-steps of 32 dims on the codes.
      // `last`: no other tile reads this K slot after this one; `end`: this is
      // the piece's last S.
      auto issue_s = [&](int x, int q, int s, bool last, bool end) {
        constexpr int kQTile = kF8 ? kTerms * kCodeBytes : kTileBytes;
        const uint64_t a = dq + static_cast<uint64_t>((q * kQTile) >> 4);
        const uint64_t b = dk + static_cast<uint64_t>((s * (kF8 ? kCodeBytes : kTileBytes)) >> 4);
        const uint32_t done = bar(kBarS + x), empty = bar(kBarEmpty + s), q_free = bar(kBarQFree);
        const uint32_t d = tmem + kTmemS + kKv * x;
        if (elect_one()) {
          if constexpr (kF8) {
#pragma unroll
            for (int t = 0; t < kTerms; ++t)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc_mma_f8(d, a + static_cast<uint64_t>((t * kCodeBytes + ks * 32) >> 4),
                          b + static_cast<uint64_t>((ks * 32) >> 4), idesc_s,
                          (t | ks) > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint64_t off = static_cast<uint64_t>(((ks >> 2) * kHalf + (ks & 3) * 32) >> 4);
              tc_mma_f16(d, a + off, b + off, idesc_s, ks > 0 ? 1u : 0u);
            }
          }
          tc_commit(done);
          if (last) tc_commit(empty);
          if (end) tc_commit(q_free);
        }
        __syncwarp();
      };
      // O_X += P_X V: k-steps of 16 tokens, P from TMEM.  `done`: O_X is complete
      // behind this one; `last` as above, for the V slot.
      // In two halves, so that the first starts while the softmax is at the second
      // (8192-token prompt, 64 / 8 heads: 719 us, 724 in one).
      auto issue_pv_half = [&](int h, int x, int s, bool first, bool done, bool last) {
        const uint64_t b = dv + static_cast<uint64_t>((s * kTileBytes) >> 4);
        const uint32_t acc0 = first ? 0u : 1u;
        const uint32_t d = tmem + kTmemO + kHeadDim * x, a = tmem + kTmemS + kKv * x;
        const uint32_t full = bar(kBarO + x), empty = bar(kF8 ? kBarEmpty16 + s : kBarEmpty + s);
        if (elect_one()) {
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int ks = 4 * h + k4;
            tc_mma_f16_ts(d, a + ks * 8, b + static_cast<uint64_t>((ks * 2048) >> 4), idesc_o,
                          ks > 0 ? 1u : acc0);
          }
          if (h == 1) {
            if (done) tc_commit(full);
            if (last) tc_commit(empty);
          }
        }
        __syncwarp();
      };
      // The same for a tile of which only the k-steps live & 15 to live >> 4 (not
      // included) hold tokens, after both halves of P.  (4 chunks of 1500 to 2048
      // tokens in a window of 1024 behind 4 kept ones, 32 heads: 160 us, 174 with
      // all eight steps taken.)
      constexpr int kAll = 8 << 4;
      auto issue_pv_some = [&](int live, int x, int s, bool first, bool done, bool last) {
        const uint64_t b = dv + static_cast<uint64_t>((s * kTileBytes) >> 4);
        const uint32_t d = tmem + kTmemO + kHeadDim * x, a = tmem + kTmemS + kKv * x;
        const int from = live & 15, to = live >> 4;
        if (elect_one()) {
#pragma unroll 1
          for (int ks = from; ks < to; ++ks)
            tc_mma_f16_ts(d, a + ks * 8, b + static_cast<uint64_t>((ks * 2048) >> 4), idesc_o,
                          ks > from || !first ? 1u : 0u);
          if (done) tc_commit(bar(kBarO + x));
          if (last) tc_commit(bar(kF8 ? kBarEmpty16 + s : kBarEmpty + s));
        }
        __syncwarp();
      };
      // The c-th tile of all pieces: K and V go round the ring's four slots (an
      // 8-bit cache's V then into one of the fp16 tiles).
      auto k_slot = [](int c) { return (2 * c) % kRing; };
      auto v_slot = [](int c) { return kF8 ? c % kV16 : (2 * c + 1) % kRing; };
      auto phase_of = [](int c) { return static_cast<uint32_t>((2 * c / kRing) & 1); };
      auto wait_k = [&](int c) { return wait(kBarFull + k_slot(c), phase_of(c)); };
      // The k-steps with rows of [skip, nval) go to `live`; rows of theirs outside
      // become zeros (P is 0 there, but the slots may hold NaN), while the softmax
      // works on the tile.  (All 128 bytes of a row: the swizzle does not matter.)
      // An 8-bit cache's converters wrote every row: there all steps are taken.
      // `inner`: the tile is whole.
      auto wait_v = [&](int c, const Item& w, int it, auto inner, int& live) {
        if (!(kF8 ? wait(kBarFull16 + v_slot(c), c / kV16 & 1)
                  : wait(kBarFull + v_slot(c), phase_of(c))))
          return false;
        live = kAll;
        if (!kF8 && !inner) {
          const Tile t = tile_of(w, it);
          live = t.skip >> 4 | (t.nval + 15) >> 4 << 4;
          uint8_t* v = smem + kOffRing + v_slot(c) * kTileBytes;
#pragma unroll 1
          for (int i = lane; i < ((t.skip & 15) + (-t.nval & 15)) * 16; i += 32) {
            const int k = i >> 4, col = i & 15, before = t.skip & 15;
            const int r = k < before ? (t.skip & ~15) + k : t.nval + k - before;
            *reinterpret_cast<uint4*>(v + (col >> 3) * kHalf + r * 128 + ((col & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        return true;
      };
      int c = 0, q_loads = 0;  // over all pieces: tiles, Q loads, P's phases
      uint32_t phase_p[2] = {0, 0};
      auto do_pv = [&](int live, int x, int s, bool first, bool done, bool last) {
        const uint32_t ph = x ? phase_p[1] : phase_p[0];
        if (x)
          phase_p[1] ^= 1u;
        else
          phase_p[0] ^= 1u;
        if (!wait(kBarP + x, ph)) return false;
        if (live != kAll) {
          if (!wait(kBarP + 2 + x, ph)) return false;
          issue_pv_some(live, x, s, first, done, last);
          return true;
        }
        issue_pv_half(0, x, s, first, done, last);
        if (!wait(kBarP + 2 + x, ph)) return false;
        issue_pv_half(1, x, s, first, done, last);
        return true;
      };
      bool ok = true;
      Item w;
      for (int k = 0; ok && get_item(k, w); ++k) {
        const int n = max(w.n_a, w.n_b), lo = full_lo(w), hi = full_hi(w);
        if (n > 0) {
          ok = wait(kBarQ, q_loads++ & 1) && wait_k(c);
          if (!ok) break;
        }
        // The tiles at [lo, hi) are whole and need none of wait_v's care: the issue
        // lies on the path from P to the next S, and a loop with that care in it is
        // 2 to 3 % slower.
        auto tiles = [&](auto step) {
          for (int it = 0; ok && it < n;) {
            if (kF8 || (it * kKv >= lo && it * kKv + kKv <= hi)) {
              const int to = kF8 ? n : min(n, hi / kKv);
              for (; ok && it < to; ++it, ++c) ok = step(it, Const<true>{});
            } else {
              ok = step(it, Const<false>{});
              ++it, ++c;
            }
          }
        };
        if (w.solo) {
          issue_s(0, 0, k_slot(c), true, false);
          ok = wait_k(c + 1);
          if (!ok) break;
          issue_s(1, 0, k_slot(c + 1), true, n == 2);
          tiles([&](int it, auto inner) -> bool {
            const int x = it & 1;
            int live;
            if (!wait_v(c, w, it, inner, live) ||
                !do_pv(live, x, v_slot(c), it < 2, it + 2 >= n, true))
              return false;
            if (it + 2 < n) {
              if (!wait_k(c + 2)) return false;
              issue_s(x, 0, k_slot(c + 2), true, it + 3 == n);
            }
            return true;
          });
        } else {
          // Each tile is needed by A, by B or by both (B leaves out the gap;
          // either may end first).  A K or V slot is free behind its last
          // reader: B's product, or A's where B has none.
          auto has_b = [&](int it) { return it < w.n_b && (it < w.gap0 || it >= w.gap1); };
          const int first_b = w.gap0 > 0 ? 0 : w.gap1;
          if (w.n_a > 0) issue_s(0, 0, k_slot(c), !has_b(0), n == 1 && !has_b(0));
          if (has_b(0)) issue_s(1, 1, k_slot(c), true, n == 1);
          tiles([&](int it, auto inner) -> bool {
            // The next K tile is waited for first, so that O += P V and the
            // next S follow each other without a pause.
            int live;
            if (!wait_v(c, w, it, inner, live) || !(it + 1 == n || wait_k(c + 1))) return false;
            const bool b0 = has_b(it), b1 = has_b(it + 1);
            if (it < w.n_a) {
              if (!do_pv(live, 0, v_slot(c), it == 0, it + 1 == w.n_a, !b0)) return false;
              if (it + 1 < w.n_a) issue_s(0, 0, k_slot(c + 1), !b1, it + 2 == n && !b1);
            }
            if (b0 && !do_pv(live, 1, v_slot(c), it == first_b, it + 1 == w.n_b, true))
              return false;
            if (b1) issue_s(1, 1, k_slot(c + 1), true, it + 2 == n);
            return true;
          });
        }
        if (ok) release_item(k);
      }
      // Wait (bounded) until every MMA this warp issued has completed.
      if (elect_one()) {
        tc_commit(bar(kBarDrain));
        mbar_wait(bar(kBarDrain), 0, p.err_flag);
      }
      __syncwarp();
    }
  } else {
    // ---------------- softmax: thread = row r of tile x
    // (The first CTA, which every grid starts, also looks at every sequence's row
    // offsets while its first copies are on their way: a bad one has no piece, so no
    // scheduler need come by it.)
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b < p.batch; b += 2 * kM)
        if (!rows_fit(p, p.q_start[b], p.q_start[b + 1])) flag_error(p.err_flag, kFlagBadSeqLen);
    const int x = warp >> 2;
    const int r = 32 * (warp & 3) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + kTmemS + kKv * x;
    const uint32_t to = tmem + lanes + kTmemO + kHeadDim * x;
    uint8_t* stage = smem + kOffStage + warp * kStageBytes;
    // Row r is head r % G of token r / G: the division for r < 128, G <= 64.
    const uint32_t inv_g = 65536u / static_cast<uint32_t>(G) + 1u;
    const int r_tok = static_cast<int>((static_cast<uint32_t>(r) * inv_g) >> 16);
    uint32_t phase_s = 0, phase_o = 0, phase_pair = 0;
    int q_made = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      // What the tiles' loop needs of the piece (a row's 128 scores leave few
      // registers: the rest is read again where it is used).
      int nt, step, pos, plain_lo, plain_hi, gap0, gap1;
      bool idle;
      float scale = p.scale_log2;
      bool negate = p.negate != 0;
      {
        Item w;
        if (!get_item(k, w)) break;
        // (Solo: tiles x, x + 2, ... for the rows of tile A.)
        const int half = w.solo ? 0 : x;
        const int tok = half ? w.tok_b : w.tok_a;
        nt = w.solo ? (w.n_a + 1 - x) >> 1 : x ? w.n_b : w.n_a;
        step = w.solo ? 2 * kKv : kKv;
        // (B's tiles leave out the gap; nt counts those in it too.)
        gap0 = x && !w.solo ? w.gap0 * kKv : 0;
        gap1 = x && !w.solo ? w.gap1 * kKv : 0;
        idle = 32 * (warp & 3) >= tok * G;
        // Positions, counted as the tiles: of this row, and of the tile's first
        // and last rows.  Tiles at or before the first (and inside the last
        // one's window) need no mask.
        const int pos0 = w.len - w.n + w.i0 + half * p.tokens_per_tile - win0_of(w);
        pos = pos0 + min(r_tok, max(0, tok - 1));
        plain_lo = full_lo(w);
        if (p.window > 0) plain_lo = max(plain_lo, pos0 + tok - p.window);
        plain_hi = min(full_hi(w), pos0 + 1);
        if constexpr (kF8) {
          if (max(w.n_a, w.n_b) > 0) {
            // Q as e4m3 terms, once the last S of the piece before has read it.
            int8_t* qexp = reinterpret_cast<int8_t*>(smem + kOffQExp);
            ok = mbar_wait_or_abort_warp(bar(kBarQFree), (q_made & 1) ^ 1, p.err_flag, abort_word);
            if (!ok) break;
            // (Solo: tile A's rows, half of them each.)
            if (w.solo || x == 0 || w.tok_b > 0)
              split_q<kBF16, kTerms>(p, w, half, warp & 3, w.solo ? 8 * x : 0,
                                     w.solo ? 8 * x + 8 : 16, inv_g,
                                     smem + half * kTerms * kCodeBytes, qexp + half * kM);
            fence_proxy_async_smem();
            // The row's exponent is read before this thread has arrived: behind it the
            // other tile's warps may, with this piece done (a single K / V tile: its
            // scores need no more of this warp), write the next piece's.
            __syncwarp();
            int ex = w.solo || r >= tok * G ? 0 : qexp[half * kM + r];
            mbar_arrive(bar(kBarQ));
            // (Solo: some of a warp's row exponents come from another warp, which
            // writes no others before the two have met at this piece's end.)
            if (w.solo) {
              ok = mbar_wait_or_abort_warp(bar(kBarQ), q_made & 1, p.err_flag, abort_word);
              if (!ok) break;
              if (r < tok * G) ex = qexp[r];
            }
            ++q_made;
            // K's scale multiplies every score of KV head j, and the row carries
            // 2^(its exponent).
            const float ks = p.k_scale[w.j];
            negate ^= ks < 0.f;
            scale *= fabsf(ks);
            scale = fmaxf(scale * __uint_as_float((127 - ex) << 23), 1e-37f);
          }
        }
        if (negate) plain_hi = plain_lo;  // (every tile changes its scores' sign)
      }
      float m = kNegInf, l = 0.f;
      int o = step > kKv ? x * kKv : 0;  // this tile's first token
      const int end = o + nt * step;
      if (o == gap0) o += gap1 - gap0;
      if (idle) {
        // No row of this warp is real: its P may be anything.
        for (; ok && o < end; o += o + step == gap0 ? step + gap1 - gap0 : step) {
          ok = mbar_wait_or_abort_warp(bar(kBarS + x), phase_s, p.err_flag, abort_word);
          phase_s ^= 1u;
          if (ok) {
            mbar_arrive(bar(kBarP + x));
            mbar_arrive(bar(kBarP + 2 + x));
          }
        }
      }
      for (const int o0 = o; o < end; o += o + step == gap0 ? step + gap1 - gap0 : step) {
        if (!mbar_wait_or_abort_warp(bar(kBarS + x), phase_s, p.err_flag, abort_word)) {
          ok = false;
          break;
        }
        phase_s ^= 1u;
        tc_fence_after();
        // The row's 128 scores, in registers from here on.
        float va[32], vb[32], vc[32], vd[32];
        tmem_ld32(ts, va);
        tmem_ld32(ts + 32, vb);
        tmem_ld32(ts + 64, vc);
        tmem_ld32(ts + 96, vd);
        tc_wait_ld_for(va);
        tc_wait_ld_for(vb);
        tc_wait_ld_for(vc);
        tc_wait_ld_for(vd);
        bool narrow = false;  // no more than 32 tokens (a few kept first ones; a rest)
        if (o < plain_lo || o + kKv > plain_hi) {
          // Seen columns: [skip, hi), of them those from lo on or below sink (at
          // or before the row's position; in its window or kept first tokens).
          const volatile Item& w = items[k & 1];
          const int s_rel = w.s_end - w.tile0 * kKv;
          const int win0 = w.base + (w.tile0 - w.sink_tiles) * kKv;
          const bool sink = o < s_rel;
          const int skip = sink ? 0 : w.lo - win0 - o;
          const int row = sink ? kKv : pos - o;  // (a sink's tile is before every row)
          const int c_hi = min(sink ? s_rel - o : w.hi - win0 - o, row + 1);
          const int c_lo = p.window > 0 && !sink ? row + 1 - p.window : 0;
          const int c_sink = p.sinks - win0 - o;
          narrow = (sink ? s_rel : w.hi - win0) - o <= 32;
          if (negate) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              va[j] = -va[j];
              vb[j] = -vb[j];
              vc[j] = -vc[j];
              vd[j] = -vd[j];
            }
          }
          auto mask = [&](float (&v)[32], int c0) {
            const uint32_t seen = (below(c_hi - c0) & ~below(skip - c0)) &
                                  (~below(c_lo - c0) | below(c_sink - c0));
            if (__all_sync(0xffffffffu, seen == 0xffffffffu)) return;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = (seen >> j) & 1u ? v[j] : kNegInf;
          };
          mask(va, 0);
          mask(vb, 32);
          mask(vc, 64);
          mask(vd, 96);
        }
        float mx0 = kNegInf, mx1 = kNegInf;
        auto peak = [&](float (&v)[32]) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            mx0 = fmaxf(mx0, fmaxf(v[k], v[k + 1]));
            mx1 = fmaxf(mx1, fmaxf(v[k + 2], v[k + 3]));
          }
        };
        peak(va);
        peak(vb);
        peak(vc);
        peak(vd);
        const float mt = fmaxf(mx0, mx1) * scale;
        // Lazy rescale: the maximum used for the exponentials moves only when
        // a score exceeds it by more than 2^8 (P and l stay far from fp32's
        // limits, and the final division uses the same maximum).  S(it) is
        // complete, so O += P(it - 1) V before it is too.
        const bool need = mt > m + kRescaleThreshold;
        if (__builtin_expect(__any_sync(0xffffffffu, need), 0)) {
          const float m_new = need ? mt : m;
          const float f = need ? ex2(m - m_new) : 1.f;  // 0 from -inf
          if (o > o0) {
#pragma unroll 1
            for (int c = 0; c < kHeadDim; c += 8) {
              float o[8];
              tmem_ld8(to + c, o);
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] *= f;
              tmem_st8(to + c, o);
            }
          }
          l *= f;
          m = m_new;
        }
        const float neg_m = m == kNegInf ? 0.f : -m;
        const uint64_t scale2 = pair2(scale, scale), neg2 = pair2(neg_m, neg_m);
        uint64_t sum2 = 0;
        auto probs = [&](float (&v)[32], int c0) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 e = unpair2(fma2(pair2(v[2 * k], v[2 * k + 1]), scale2, neg2));
            const float p0 = ex2(e.x), p1 = ex2(e.y);
            sum2 = add2(sum2, pair2(p0, p1));
            pk[k] = pack2<kMmaBF16>(p0, p1);
          }
          tmem_st16(ts + c0 / 2, pk);
        };
        auto zeros = [&](int c0) {  // (8-bit: every step of P V is taken)
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) pk[k] = 0;
          tmem_st16(ts + c0 / 2, pk);
        };
        probs(va, 0);
        if (!narrow) {
          probs(vb, 32);
        } else if (kF8) {
          zeros(32);
          zeros(64);
          zeros(96);
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarP + x));
        if (!narrow) {
          probs(vc, 64);
          probs(vd, 96);
        }
        {
          const float2 e = unpair2(sum2);
          l += e.x + e.y;
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarP + 2 + x));
      }
      // ---------------- epilogue
      if (ok && nt > 0) {
        ok = mbar_wait_or_abort_warp(bar(kBarO + x), phase_o, p.err_flag, abort_word);
        phase_o ^= 1u;
      }
      const Item w = items[k & 1];
      // (The loop's scale is at least 1e-37 whatever K's: one that is not finite
      // counts here, for every row that sees something.)
      if (kF8 && l != 0.f) l += 0.f * p.k_scale[w.j];
      const int half = w.solo ? 0 : x;
      const int tok = half ? w.tok_b : w.tok_a;
      const int i0 = w.i0 + half * p.tokens_per_tile;
      if (ok && 32 * (warp & 3) < tok * G) {
        tc_fence_after();
        const bool bad = w.bad || bad_word[k & 1] != 0;
        // Weight of this warp's O (and, solo, of the other's): 1 / l, times an
        // 8-bit cache's V scale; 0 for a row that sees nothing (l = 0, exactly) or
        // is bad.  NaN scores make l NaN, and the row with it.
        auto norm = [&]() { return l == 0.f || bad ? 0.f : (kF8 ? p.v_scale[w.j] : 1.f) / l; };
        float wa = norm(), wb = 0.f;
        // This lane stores piece lane % 8 of the warp's rows lane / 8, + 4, ...
        // + 28: their places among the packed rows, from the tile's first one on.
        const int64_t row0 = static_cast<int64_t>(w.q0 + i0) * p.h_q + w.j * G;
        const int rows = tok * G;
        int place[8];
        bool real[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int q = 32 * (warp & 3) + (lane >> 3) + 4 * e;
          const int tk = static_cast<int>((static_cast<uint32_t>(q) * inv_g) >> 16);
          place[e] = tk * (p.h_q - G) + q;
          real[e] = q < rows;
        }
        // 128 staged bytes of each row go to base + row * pitch bytes.
        auto store = [&](uint8_t* base, int pitch) {
          base += row0 * pitch + 16 * (lane & 7);
          __syncwarp();
          uint4 y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = *staged(stage, (lane >> 3) + 4 * e, lane & 7);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (real[e])
              *reinterpret_cast<uint4*>(base + static_cast<int64_t>(place[e]) * pitch) = y[e];
          __syncwarp();
        };
        // Solo: the two halves of a row join.  Both warps of a row reach all of its
        // TMEM lane, so each weighs and stores 64 columns of the sum.  They meet
        // when both O are complete, when the A warp has the weights (from its
        // maxima and sums and the B warp's), and when both O are read.  (Bounded
        // barriers: a warp that gave up elsewhere does not leave the other waiting.
        // 3 chunks of 5 tokens over 300, 8 heads: 10.3 us; through shared memory, by
        // the A warp alone, 11.4.)
        float2* ml = reinterpret_cast<float2*>(smem + kOffMerge) + r;
        auto meet = [&]() {
          const uint32_t at = bar(kBarPair + (warp & 3));
          tc_fence_before();
          mbar_arrive(at);
          ok = mbar_wait_or_abort_warp(at, phase_pair, p.err_flag, abort_word);
          phase_pair ^= 1u;
          tc_fence_after();
        };
        if (w.solo) {
          if (x == 1) *ml = make_float2(m, l);
          meet();
          if (x == 0) {
            const float2 other = *ml;
            const float top = fmaxf(m, other.x);
            wa = m == kNegInf ? 0.f : ex2(m - top);
            wb = other.x == kNegInf ? 0.f : ex2(other.x - top);
            l = wa * l + wb * other.y;
            m = top;
            const float f = norm();
            wa *= f;
            wb *= f;
            *ml = make_float2(wa, wb);
          }
          if (ok) meet();
          if (x == 1) {
            const float2 both = *ml;
            wa = both.x;
            wb = both.y;
          }
        }
        const uint32_t to_a = tmem + lanes + kTmemO, to_b = to_a + kHeadDim;
        const int c0 = w.solo ? 64 * x : 0, c1 = w.solo ? c0 + 64 : kHeadDim;
#pragma unroll 1
        for (int c = c0; ok && c < c1 && (nt > 0 || p.n_split == 1); c += 32) {
          float o[32];
          if (w.solo) {
            float y[32];
            tmem_ld32(to_a + c, o);
            tmem_ld32(to_b + c, y);
            tc_wait_ld_for(o);
            tc_wait_ld_for(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = wa * o[e] + wb * y[e];
          } else {
            tmem_ld32(to + c, o);
            tc_wait_ld_for(o);
            const uint64_t wa2 = pair2(wa, wa);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 f = unpair2(mul2(pair2(o[e], o[e + 1]), wa2));
              o[e] = f.x;
              o[e + 1] = f.y;
            }
          }
          if (__any_sync(0xffffffffu, wa == 0.f && wb == 0.f)) {
            // Rows that see nothing (their O may hold anything).
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = wa == 0.f && wb == 0.f ? 0.f : o[e];
          }
          if (p.n_split == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *staged(stage, lane, ((c >> 3) & 4) + e) =
                  make_uint4(pack2<kBF16>(o[8 * e], o[8 * e + 1]),
                             pack2<kBF16>(o[8 * e + 2], o[8 * e + 3]),
                             pack2<kBF16>(o[8 * e + 4], o[8 * e + 5]),
                             pack2<kBF16>(o[8 * e + 6], o[8 * e + 7]));
            if (c & 32)
              store(static_cast<uint8_t*>(p.out) + 2 * (c - 32), 2 * kHeadDim);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *staged(stage, lane, e) =
                  make_uint4(__float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                             __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3]));
            store(reinterpret_cast<uint8_t*>(p.part_o) + 4 * (w.split * kHeadDim + c),
                  4 * kHeadDim * p.n_split);
          }
        }
        if (ok && w.solo) meet();
        if (p.n_split > 1 && !(w.solo && x == 1)) {
          if (r < rows)
            p.part_lse[(row0 + static_cast<int64_t>(r_tok) * p.h_q + (r - r_tok * G)) * p.n_split +
                       w.split] = bad ? DECATTN_POISON_LSE : l == 0.f ? kNegInf : m + lg2(l);
        }
      }
      if (ok) release_item(k);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpTmem) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) {
    // Never leave the CTA with copies in flight (after an abort there may be
    // some): the last copy into each ring slot is waited for.
    if (made_by[2] > 0) mbar_wait(bar(kBarQ), (made_by[2] - 1) & 1, p.err_flag);
    const int made_k = made_by[0], made_v = made_by[1];
    auto was_made = [&](int e) { return (e >> 1) < ((e & 1) ? made_v : made_k); };
    const int end = 2 * max(made_k, made_v);
    for (int e = max(0, end - 2 * kRing); e < end; ++e)
      if (was_made(e) && !was_made(e + kRing) &&
          !mbar_wait(bar(kBarFull + e % kRing), (e / kRing) & 1, p.err_flag))
        break;
  }
}

// Joins the splits of a row: out = sum_s w_s o_s / sum_s w_s, w_s = 2^(lse_s -
// max).  One warp per (token, head); tokens outside every sequence stay as
// they are, splits with nothing to see (lse = -inf) have no partial to read,
// a bad sequence (+inf) gives zeros, and a split with NaN scores (lse NaN) NaN.
template <bool kBF16>
__global__ void __launch_bounds__(256) gqa_prefill_combine_kernel(const PrefillParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.tokens) * p.h_q) return;
  const int tok = static_cast<int>(row / p.h_q);
  int lo = 0, hi = p.batch;  // the sequence whose rows hold tok
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid] <= tok) lo = mid; else hi = mid;
  }
  const int a = p.q_start[lo], e = p.q_start[lo + 1];
  if (tok < a || tok >= e || !rows_fit(p, a, e)) return;
  const float* lse = p.part_lse + row * p.n_split;
  float mx = kNegInf;  // (the maximum of the numbers: NaN does not count)
  bool some = false;
  for (int s = lane; s < p.n_split; s += 32) {
    mx = fmaxf(mx, lse[s]);
    some |= lse[s] != kNegInf;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * kHeadDim);
  if (!__any_sync(0xffffffffu, some) || mx == DECATTN_POISON_LSE) {
    dst[lane] = make_uint2(0, 0);
    return;
  }
  const float4* po = reinterpret_cast<const float4*>(p.part_o + row * p.n_split * kHeadDim);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int s0 = 0; s0 < p.n_split; s0 += 4) {
    float wt[4];
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u;
      const float at = s < p.n_split ? lse[s] : kNegInf;
      wt[u] = at != kNegInf ? ex2(at - mx) : 0.f;
      x[u] = at != kNegInf ? po[s * (kHeadDim / 4) + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      sum += wt[u];
      acc.x = fmaf(wt[u], x[u].x, acc.x);
      acc.y = fmaf(wt[u], x[u].y, acc.y);
      acc.z = fmaf(wt[u], x[u].z, acc.z);
      acc.w = fmaf(wt[u], x[u].w, acc.w);
    }
  }
  const float inv = 1.f / sum;
  dst[lane] = make_uint2(pack2<kBF16>(acc.x * inv, acc.y * inv),
                         pack2<kBF16>(acc.z * inv, acc.w * inv));
}

template <bool kBF16, bool kF8>
cudaError_t launch_t(const PrefillParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, cudaStream_t stream) {
  auto kern = gqa_prefill_kernel<kBF16, kF8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(p.n_items) * p.n_split * p.h_kv;
  kern<<<grid, kThreads, kSmemBytes, stream>>>(tq, tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.n_split == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.tokens) * p.h_q + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gqa_prefill_combine_kernel<kBF16>, p);
}

}  // namespace

cudaError_t launch_gqa_prefill(const PrefillParams& p, const CUtensorMap& tm_q,
                               const CUtensorMap& tm_k, const CUtensorMap& tm_v, bool bf16,
                               bool fp8, cudaStream_t stream) {
  if (fp8)
    return bf16 ? launch_t<true, true>(p, tm_q, tm_k, tm_v, stream)
                : launch_t<false, true>(p, tm_q, tm_k, tm_v, stream);
  return bf16 ? launch_t<true, false>(p, tm_q, tm_k, tm_v, stream)
              : launch_t<false, false>(p, tm_q, tm_k, tm_v, stream);
}

}  // namespace decattn
