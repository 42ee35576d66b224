// api.cu -- the C ABI of libdecattn: argument checks, split planning,
// workspace carving, TMA descriptor construction and kernel dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "decattn.h"
#include "internal.h"

namespace decattn {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 2-D tensor map over a row-major [outer, inner] tensor of element type dt
// whose rows are row_bytes apart; boxes of box_inner x box_outer elements,
// 128-byte swizzle.
bool make_map_2d_t(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t inner,
                   uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The same over a 16-bit (fp16 / bf16) tensor.
bool make_map_2d(CUtensorMap* m, const void* base, bool bf16, uint64_t inner, uint64_t outer,
                 uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer) {
  return make_map_2d_t(m, base,
                       bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                       inner, outer, row_bytes, box_inner, box_outer);
}

// 3-D tensor map over a row-major [n2, n1, n0] 16-bit tensor (n0 innermost),
// boxes of b0 x b1 x b2 elements, 128-byte swizzle.
bool make_map_3d(CUtensorMap* m, const void* base, bool bf16, uint64_t n0, uint64_t n1,
                 uint64_t n2, uint32_t b0, uint32_t b1, uint32_t b2,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {n0, n1, n2};
  cuuint64_t strides[2] = {n0 * 2, n0 * n1 * 2};
  cuuint32_t box[3] = {b0, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D tensor map with explicit byte strides for dimensions 1 and 2 (they
// need not increase), boxes of b0 x b1 x b2 elements, 128-byte swizzle.
bool make_map_3d_strided(CUtensorMap* m, const void* base, bool bf16, uint64_t n0, uint64_t n1,
                         uint64_t n2, uint64_t stride1, uint64_t stride2, uint32_t b0,
                         uint32_t b1, uint32_t b2) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {n0, n1, n2};
  cuuint64_t strides[2] = {stride1, stride2};
  cuuint32_t box[3] = {b0, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

int device_sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return -1;
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (dev < 64) cache[dev] = n;
  return n;
}

}  // namespace

// Token chunk per split: a multiple of kTile covering max_seq_len in at most
// n_split chunks.  Returns the number of chunks actually used.
int resolve_splits(int max_seq_len, int n_split, int* tokens_per_split) {
  const int tiles = max_seq_len > 0 ? (max_seq_len + kTile - 1) / kTile : 1;
  if (n_split < 1) n_split = 1;
  if (n_split > tiles) n_split = tiles;
  const int tiles_per = (tiles + n_split - 1) / n_split;
  *tokens_per_split = tiles_per * kTile;
  return (tiles + tiles_per - 1) / tiles_per;
}

// A window of every token there can be hides nothing: the kernels' plain case.
int useful_window(int window, int max_seq_len) { return window < max_seq_len ? window : 0; }

// A sliding window of W tokens starts at a block (or 64-token) boundary at
// most min(block_size, 64) - 1 tokens before the window: the longest token
// range any sequence streams.
int window_span(int max_seq_len, int window, int block_size) {
  if (window <= 0) return max_seq_len;
  const int64_t span = static_cast<int64_t>(window) + (block_size < kTile ? block_size : kTile) - 1;
  return span < max_seq_len ? static_cast<int>(span) : max_seq_len;
}

// A window with kept first tokens streams its window's range and the sinks'
// own 64-token tiles; once both cover every length, the whole sequence.
int sinks_span(int max_seq_len, int window, int sinks, int block_size) {
  const int span = window_span(max_seq_len, window, block_size);
  if (window <= 0 || sinks <= 0) return span;
  if (static_cast<int64_t>(window) + sinks >= max_seq_len) return max_seq_len;
  const int64_t both = (static_cast<int64_t>(sinks) + kTile - 1) / kTile * kTile + span;
  return static_cast<int>(both < 0x7fffffc0 ? both : 0x7fffffc0);
}

namespace {

// Split count for `units` independent (sequence[, KV head]) work units on
// `slots` resident CTAs, for the latency-bound 8-bit-cache consumers of
// wide groups, which gain from more CTAs in flight: one split per unit once
// there are 1.5 waves of CTAs; otherwise split each sequence until about two
// waves exist, keeping at least two 64-token tiles per split (measured on the
// 70B-shaped layer with the 16-row padded consumer: 2 splits 211 us, 1 split
// 233 us).
int plan_splits(int units, int max_seq_len, int slots) {
  const int tiles = max_seq_len > 0 ? (max_seq_len + kTile - 1) / kTile : 1;
  if (units < 1) units = 1;
  if (slots < 1) slots = 1;
  if (2 * units >= 3 * slots) return 1;
  int ns = (2 * slots + units - 1) / units;
  int cap = tiles / 2 > 1 ? tiles / 2 : 1;
  if (cap > DECATTN_MAX_SPLITS) cap = DECATTN_MAX_SPLITS;
  if (ns > cap) ns = cap;
  int tps = 0;
  return resolve_splits(max_seq_len, ns, &tps);
}

// Split count for the 16-bit GQA partial kernel: fill at most ~85 % of one
// wave of resident CTAs, with at least 8 tiles (512 tokens) per split.  A
// wave that overflows by a few CTAs costs a second pass over the whole
// per-CTA time, and short splits only add partials.  Measured on GB300
// (2 CTAs per SM, 304 slots): B=1 x 8 KV heads at S=131072, 32 splits
// 92.7 us / 38 splits 96.1 / 40 splits 133.9 / 76 splits 109.1; B=4, 8 splits
// 314 us / 10 splits 456 / 19 splits 325; Llama-3.1-8B MQA (16 units,
// S <= 4096), 8 splits 32 us / 32 splits 59; its GQA-8 (128 units), 2-3
// splits 44-45 us / 5 splits 50.
int plan_splits_one_wave(int units, int max_seq_len, int slots, int min_tiles = 8) {
  const int tiles = max_seq_len > 0 ? (max_seq_len + kTile - 1) / kTile : 1;
  if (units < 1) units = 1;
  if (slots < 1) slots = 1;
  int ns = static_cast<int>((static_cast<int64_t>(slots) * 85) / (100 * static_cast<int64_t>(units)));
  int cap = tiles / min_tiles > 1 ? tiles / min_tiles : 1;
  if (cap > DECATTN_MAX_SPLITS) cap = DECATTN_MAX_SPLITS;
  if (ns > cap) ns = cap;
  if (ns < 1) ns = 1;
  int tps = 0;
  return resolve_splits(max_seq_len, ns, &tps);
}

}  // namespace

int plan_gqa_splits(int batch, int h_q, int h_kv, int max_seq_len, int num_sms) {
  // GQA partial kernels: two resident CTAs per SM, both the mma.sync one
  // (3-stage ring of 32 KB, up to 16 query heads per KV head) and the
  // tcgen05 one for wider groups (2-stage K and V rings, ~100 KB).  The
  // tcgen05 kernel's splits may be as short as 4 tiles: with few units
  // (Llama-3.1-8B MQA at B = 16, 16 units, S <= 4096) 16 splits ran 20.7 us
  // against 22.9 for the 8 that 8-tile splits allow (L2 flushed).
  const int group = h_kv > 0 ? h_q / h_kv : 1;
  return plan_splits_one_wave(batch * h_kv, max_seq_len, num_sms * 2, group > kWideGroup ? 4 : 8);
}

int plan_gqa_fp8_splits(int batch, int h_q, int h_kv, int max_seq_len, int num_sms) {
  // Up to 8 query heads per KV head the 8-bit-cache kernel (transposed
  // consumer, 95 registers, three 16 KB stages) runs four CTAs per SM and,
  // like the 16-bit kernel, wants at most one wave (70B-shaped layer, 512
  // units on 608 slots: 1 split 160 us, 2 splits 171, 4 splits 185; at
  // B=16, 4 splits 48.4 us, 3 splits 50.0, 8 splits 55.6).  Groups of 9..16
  // run two CTAs per SM; from ~0.85 of a wave of units on, their
  // latency-bound consumers prefer about two waves.  Wider groups go to the
  // tensor-core kernel (two CTAs per SM), which, like its 16-bit form, wants
  // one wave.
  const int group = h_kv > 0 ? h_q / h_kv : 1;
  const int per_sm = (group >= 2 && group <= 8) ? 4 : 2;
  const int slots = num_sms * per_sm;
  const int64_t units = static_cast<int64_t>(batch) * h_kv;
  // (The tensor-core kernel's splits may again be 4 tiles long: MQA with 32
  // query heads at B = 16, S = 4096, 16 splits 18.7 us against 20.7 for 8.)
  if (per_sm == 4 || group > 16 || units * 100 < static_cast<int64_t>(slots) * 85)
    return plan_splits_one_wave(batch * h_kv, max_seq_len, slots, group > kWideGroup ? 4 : 8);
  return plan_splits(batch * h_kv, max_seq_len, slots);
}

// A window with kept first tokens, up to 16 query heads per KV head: two to eight
// splits merge within their cluster (no second launch), so they may be as short as
// two tiles while they are two thirds of a wave; from six tiles on, where it begins
// to pay.  Splits chosen so against the rules above, us: 18 sequences, 5 heads on 1,
// window 1335 (16-bit / e4m3) 8: 11.2 / 9.2, 2: 18.2 / 16.6; 4, 64 on 8, 1024: 6:
// 11.5, 2: 14.6; 2, 32 on 32, 1000: 3: 9.7, 2: 11.0 (8, two waves: 13.2); 8, 32 on 8,
// 2048, e4m3 4 / 6 / 8: 11.2 / 10.9 / 11.4; 3, 12 on 4, 200 (5 tiles) 1: 6.6, 2: 7.0.
int plan_sinks_splits(int batch, int h_q, int h_kv, int span, int num_sms, bool fp8) {
  const int base = fp8 ? plan_gqa_fp8_splits(batch, h_q, h_kv, span, num_sms)
                       : plan_gqa_splits(batch, h_q, h_kv, span, num_sms);
  const int group = h_kv > 0 ? h_q / h_kv : 1, tiles = span / kTile + (span % kTile > 0);
  const int64_t units = static_cast<int64_t>(batch) * h_kv;
  if (group > kWideGroup || tiles < 6 || units < 1) return base;
  const int slots = num_sms * (fp8 && group >= 2 && group <= 8 ? 4 : 2);
  const int64_t wave = static_cast<int64_t>(slots) * 65 / 100 / units;
  const int most = static_cast<int>(std::min<int64_t>(wave, std::min(8, tiles / 2)));
  return std::max(base, most);
}

// Listed blocks: as a window's with kept tokens.  Wide groups' splits may be as short
// as two tiles (5 sequences, 32 heads on 1, e4m3, 33 tiles: 17 splits 19.6 us, 7 21.6).
int plan_blocks_splits(int batch, int h_q, int h_kv, int span, int num_sms, bool fp8) {
  const int group = h_kv > 0 ? h_q / h_kv : 1;
  if (group > kWideGroup) return plan_splits_one_wave(batch * h_kv, span, num_sms * 2, 2);
  return plan_sinks_splits(batch, fp8 && group == 1 ? 2 * h_kv : h_q, h_kv, span, num_sms, fp8);
}

// With the scores kept: as a plain decode's, but that MHA over an 8-bit cache runs on
// the same consumer as groups of 2 to 8, four CTAs an SM.
int plan_weights_splits(int batch, int h_q, int h_kv, int max_seq_len, int num_sms, bool fp8) {
  if (!fp8) return plan_gqa_splits(batch, h_q, h_kv, max_seq_len, num_sms);
  return plan_gqa_fp8_splits(batch, h_q == h_kv ? 2 * h_kv : h_q, h_kv, max_seq_len, num_sms);
}

int plan_mla_splits(int batch, int max_seq_len, int num_sms) {
  // MLA partial kernel: one CTA pair per two SMs, all pairs resident at
  // once, each streaming an equal share of the batch's 64-token tiles.  Use
  // every SM pair, but give each pair at least two tiles of the host's
  // upper bound (batch x tiles of max_seq_len) so that tiny batches do not
  // pay a partial + combine for nothing.
  const long long slots = num_sms / 2 > 0 ? num_sms / 2 : 1;
  const long long tiles =
      static_cast<long long>(batch) * (max_seq_len > 0 ? (max_seq_len + kTile - 1) / kTile : 1);
  long long pairs = tiles / 2;
  if (pairs > slots) pairs = slots;
  if (pairs > DECATTN_MAX_SPLITS) pairs = DECATTN_MAX_SPLITS;
  return pairs < 1 ? 1 : static_cast<int>(pairs);
}

size_t mla_workspace_bytes(int batch, int n_pairs, size_t* off_lse, size_t* off_o) {
  if (batch < 1 || n_pairs < 1 || n_pairs > DECATTN_MAX_SPLITS) return 0;
  if (n_pairs == 1) return 0;
  const size_t slots = 2 * static_cast<size_t>(n_pairs);
  // header, per-sequence first tiles (batch + 1), pair slice starts (n_pairs + 1),
  // per-sequence first cost positions (batch)
  const size_t hdr =
      align_up((static_cast<size_t>(kHdrPref) + 2 * batch + 1 + n_pairs + 1) * sizeof(int));
  const size_t lse = align_up(slots * kMlaHeads * sizeof(float));
  const size_t o = align_up(slots * kMlaHeads * kMlaDc * sizeof(float));
  if (off_lse) *off_lse = hdr;
  if (off_o) *off_o = hdr + lse;
  return hdr + lse + o;
}

}  // namespace decattn

using namespace decattn;

extern "C" {

const char* decattn_status_string(int status) {
  switch (status) {
    case DECATTN_OK: return "ok";
    case DECATTN_ERR_INVALID_ARG: return "invalid argument";
    case DECATTN_ERR_UNSUPPORTED: return "unsupported configuration";
    case DECATTN_ERR_WORKSPACE: return "workspace missing or too small";
    case DECATTN_ERR_CUDA: return "CUDA error";
    default: return "unknown status";
  }
}

int decattn_version(void) { return 100; }

int decattn_selftest_wait_timeout(int* err_flag, int* result, int limit_us, void* stream) {
  if (!err_flag || !result || !aligned(err_flag, 4) || !aligned(result, 4) || limit_us < 1 ||
      limit_us > 100000)
    return DECATTN_ERR_INVALID_ARG;
  const cudaError_t e = launch_wait_selftest(err_flag, result, static_cast<uint64_t>(limit_us) * 1000,
                                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int decattn_selftest_warp_wait(int* err_flag, int* result, int limit_us, void* stream) {
  if (!err_flag || !result || !aligned(err_flag, 4) || !aligned(result, 4) || limit_us < 1 ||
      limit_us > 100000)
    return DECATTN_ERR_INVALID_ARG;
  const cudaError_t e =
      launch_warp_wait_selftest(err_flag, result, static_cast<uint64_t>(limit_us) * 1000,
                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int decattn_selftest_gave_up(int* err_flag, float* result, int limit_us, void* stream) {
  if (!err_flag || !result || !aligned(err_flag, 4) || !aligned(result, 4) || limit_us < 1 ||
      limit_us > 100000)
    return DECATTN_ERR_INVALID_ARG;
  const cudaError_t e =
      launch_gave_up_selftest(err_flag, result, static_cast<uint64_t>(limit_us) * 1000,
                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int64_t decattn_kv_bytes_per_token(int n_layers, int n_kv, int d_head, int bytes) {
  if (n_layers < 0 || n_kv < 0 || d_head < 0 || bytes < 0) return -1;
  return static_cast<int64_t>(n_layers) * n_kv * d_head * 2 * bytes;
}

int64_t decattn_mla_bytes_per_token(int n_layers, int d_c, int d_rope, int bytes) {
  if (n_layers < 0 || d_c < 0 || d_rope < 0 || bytes < 0) return -1;
  return static_cast<int64_t>(n_layers) * (d_c + d_rope) * bytes;
}

size_t gqa_decode_workspace_size(int batch, int h_q, int d_head, int num_splits) {
  if (batch < 1 || h_q < 1 || d_head < 1 || num_splits < 1 || num_splits > DECATTN_MAX_SPLITS)
    return 0;
  if (num_splits == 1) return 0;
  const size_t rows = static_cast<size_t>(batch) * h_q * num_splits;
  return align_up(rows * d_head * sizeof(float)) + align_up(rows * sizeof(float));
}

size_t mla_decode_workspace_size(int batch, int num_splits) {
  return mla_workspace_bytes(batch, num_splits, nullptr, nullptr);
}

int gqa_decode_plan_splits(int batch, int h_q, int h_kv, int d_head, int max_seq_len,
                           int num_sms) {
  if (batch < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || d_head < 1 || max_seq_len < 0)
    return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  return plan_gqa_splits(batch, h_q, h_kv, max_seq_len, num_sms);
}

int gqa_decode_fp8kv_plan_splits(int batch, int h_q, int h_kv, int d_head, int max_seq_len,
                                 int num_sms) {
  if (batch < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || d_head < 1 || max_seq_len < 0)
    return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  return plan_gqa_fp8_splits(batch, h_q, h_kv, max_seq_len, num_sms);
}

int gqa_decode_window_plan_splits(int batch, int h_q, int h_kv, int d_head, int max_seq_len,
                                  int window, int block_size, int kv_bytes, int num_sms) {
  if (batch < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || d_head < 1 || max_seq_len < 0 ||
      window < 1 || !is_pow2(block_size) || (kv_bytes != 1 && kv_bytes != 2))
    return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  const int span = window_span(max_seq_len, window, block_size);
  return kv_bytes == 1 ? plan_gqa_fp8_splits(batch, h_q, h_kv, span, num_sms)
                       : plan_gqa_splits(batch, h_q, h_kv, span, num_sms);
}

int gqa_decode_sinks_plan_splits(int batch, int h_q, int h_kv, int d_head, int max_seq_len,
                                 int window, int sinks, int block_size, int kv_bytes,
                                 int num_sms) {
  if (batch < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || d_head < 1 || max_seq_len < 0 ||
      window < 1 || sinks < 0 || !is_pow2(block_size) || (kv_bytes != 1 && kv_bytes != 2))
    return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  if (sinks > 0) window = useful_window(window, max_seq_len);
  const int span = sinks_span(max_seq_len, window, sinks, block_size);
  if (sinks > 0 && window > 0)
    return plan_sinks_splits(batch, h_q, h_kv, span, num_sms, kv_bytes == 1);
  return kv_bytes == 1 ? plan_gqa_fp8_splits(batch, h_q, h_kv, span, num_sms)
                       : plan_gqa_splits(batch, h_q, h_kv, span, num_sms);
}

int gqa_decode_blocks_plan_splits(int batch, int h_q, int h_kv, int d_head, int max_seq_len,
                                  int count, int block_size, int kv_bytes, int num_sms) {
  if (batch < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || d_head < 1 || max_seq_len < 0 ||
      count < 1 || !is_pow2(block_size) || (kv_bytes != 1 && kv_bytes != 2))
    return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  return plan_blocks_splits(batch, h_q, h_kv, static_cast<int>(std::min<int64_t>(
                                max_seq_len, static_cast<int64_t>(count) * block_size)),
                            num_sms, kv_bytes == 1);
}

int gqa_decode_weights_plan_splits(int batch, int h_q, int h_kv, int d_head, int max_seq_len,
                                   int kv_bytes, int num_sms) {
  if (batch < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || d_head < 1 || max_seq_len < 0 ||
      (kv_bytes != 1 && kv_bytes != 2))
    return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  return plan_weights_splits(batch, h_q, h_kv, max_seq_len, num_sms, kv_bytes == 1);
}

size_t gqa_decode_weights_workspace_size(int batch, int h_q, int d_head, int max_seq_len,
                                         int num_splits) {
  if (batch < 1 || h_q < 1 || d_head < 1 || max_seq_len < 0 || num_splits < 1 ||
      num_splits > DECATTN_MAX_SPLITS)
    return 0;
  const size_t rows = static_cast<size_t>(batch) * h_q;
  const size_t stride = (std::max<size_t>(1, max_seq_len) + kTile - 1) / kTile * kTile;
  return (num_splits > 1 ? align_up(rows * num_splits * d_head * sizeof(float)) : 0) +
         align_up(rows * num_splits * sizeof(float)) + align_up(rows * stride * sizeof(float));
}

int mla_decode_plan_splits(int batch, int max_seq_len, int num_sms) {
  if (batch < 1 || max_seq_len < 0) return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  return plan_mla_splits(batch, max_seq_len, num_sms);
}

static int check_launch(const decattn_launch* L, bool mla) {
  if (!L) return DECATTN_ERR_INVALID_ARG;
  if (L->batch < 1 || L->num_blocks < 1 || L->max_blocks_per_seq < 1 || L->max_seq_len < 0)
    return DECATTN_ERR_INVALID_ARG;
  if (L->dtype != DECATTN_FP16 && L->dtype != DECATTN_BF16) return DECATTN_ERR_INVALID_ARG;
  if (L->num_splits < 0 || L->num_splits > DECATTN_MAX_SPLITS) return DECATTN_ERR_INVALID_ARG;
  if (!is_pow2(L->block_size)) return DECATTN_ERR_INVALID_ARG;
  if (L->block_size < 8 || L->block_size > (mla ? 64 : 256)) return DECATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(L->max_seq_len) >
      static_cast<int64_t>(L->max_blocks_per_seq) * L->block_size)
    return DECATTN_ERR_INVALID_ARG;
  if (static_cast<int64_t>(L->num_blocks) * L->block_size > 0x7fffffffLL)
    return DECATTN_ERR_UNSUPPORTED;
  if (L->workspace && !aligned(L->workspace, 16)) return DECATTN_ERR_INVALID_ARG;
  if (L->err_flag && !aligned(L->err_flag, 4)) return DECATTN_ERR_INVALID_ARG;
  return DECATTN_OK;
}

}  // extern "C"

namespace decattn {

int gqa_check_args(const void* q, const void* k_cache, const void* v_cache,
                   const float* k_scale, const float* v_scale, bool fp8,
                   const int32_t* block_table, const int32_t* seq_lens, const void* out, int h_q,
                   int h_kv, int d_head, float scale, int window, const decattn_launch* L) {
  int st = check_launch(L, false);
  if (st != DECATTN_OK) return st;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return DECATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return DECATTN_ERR_INVALID_ARG;
  if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
    return DECATTN_ERR_INVALID_ARG;
  if (h_q < 1 || h_kv < 1 || h_q % h_kv != 0) return DECATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return DECATTN_ERR_INVALID_ARG;
  if (d_head != kHeadDim) return DECATTN_ERR_UNSUPPORTED;
  if (h_q / h_kv > 64) return DECATTN_ERR_UNSUPPORTED;
  if (window < 0) return DECATTN_ERR_INVALID_ARG;
  return DECATTN_OK;
}

}  // namespace decattn

extern "C" {

// What the forms over listed blocks and with token weights have beside a decode's
// arguments.
struct DecodeMore {
  const int32_t* selected = nullptr;
  int count = 0;
  float* weights = nullptr;
  const int32_t* weighed_lens = nullptr;
  float decay = 1.f;
};

static int64_t scores_stride(int max_seq_len) {
  return (std::max<int64_t>(1, max_seq_len) + kTile - 1) / kTile * kTile;
}

// The longest token range that listed blocks make up.
static int listed_span(int max_seq_len, int count, int block_size) {
  return static_cast<int>(std::min<int64_t>(max_seq_len, static_cast<int64_t>(count) * block_size));
}

// gqa_decode and gqa_decode_fp8kv share everything but the cache element type
// (and the 8-bit cache's per-KV-head scales).
static int gqa_decode_impl(const void* q, const void* k_cache, const void* v_cache,
                           const float* k_scale, const float* v_scale, bool fp8,
                           const int32_t* block_table, const int32_t* seq_lens, void* out,
                           int h_q, int h_kv, int d_head, float scale, int window, int sinks,
                           const decattn_launch* L, const DecodeMore& more = {}) {
  const int st = gqa_check_args(q, k_cache, v_cache, k_scale, v_scale, fp8, block_table,
                                seq_lens, out, h_q, h_kv, d_head, scale, window, L);
  if (st != DECATTN_OK) return st;
  if (sinks > 0) window = useful_window(window, L->max_seq_len);
  const int span = more.selected ? listed_span(L->max_seq_len, more.count, L->block_size)
                                 : sinks_span(L->max_seq_len, window, sinks, L->block_size);
  int n_split = L->num_splits;
  if (n_split == 0) {
    const int sms = device_sm_count();
    if (sms <= 0) return DECATTN_ERR_CUDA;
    n_split = more.selected           ? plan_blocks_splits(L->batch, h_q, h_kv, span, sms, fp8)
              : more.weights          ? plan_weights_splits(L->batch, h_q, h_kv, span, sms, fp8)
              : sinks > 0 && window > 0 ? plan_sinks_splits(L->batch, h_q, h_kv, span, sms, fp8)
              : fp8                   ? plan_gqa_fp8_splits(L->batch, h_q, h_kv, span, sms)
                                      : plan_gqa_splits(L->batch, h_q, h_kv, span, sms);
  }
  int tps = 0;
  const int eff = resolve_splits(span, n_split, &tps);

  GqaParams p{};
  p.q = q;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.err_flag = L->err_flag;
  p.batch = L->batch;
  p.h_q = h_q;
  p.h_kv = h_kv;
  p.group = h_q / h_kv;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  p.max_seq_len = L->max_seq_len;
  p.n_split = eff;
  p.tokens_per_split = tps;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.window = window;
  p.sinks = window > 0 ? sinks : 0;
  // (A cluster has at most eight CTAs; wide groups have a kernel of their own.)
  p.joint = (p.sinks > 0 || more.selected) && eff > 1 && eff <= 8 && p.group <= kWideGroup;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.selected = more.selected;
  p.n_listed = more.count;
  if (eff > 1 || more.weights) {
    const size_t need =
        more.weights
            ? gqa_decode_weights_workspace_size(L->batch, h_q, d_head, L->max_seq_len, eff)
            : gqa_decode_workspace_size(L->batch, h_q, d_head, eff);
    if (!L->workspace || L->workspace_bytes < need) return DECATTN_ERR_WORKSPACE;
    const size_t rows = static_cast<size_t>(L->batch) * h_q * eff;
    char* ws = static_cast<char*>(L->workspace);
    if (eff > 1) {
      p.part_o = reinterpret_cast<float*>(ws);
      ws += align_up(rows * d_head * sizeof(float));
    }
    p.part_lse = reinterpret_cast<float*>(ws);
    if (more.weights) {
      p.scores = reinterpret_cast<float*>(ws + align_up(rows * sizeof(float)));
      p.score_stride = scores_stride(L->max_seq_len);
      p.weights = more.weights;
      p.weighed_lens = more.weighed_lens;
      p.decay = more.decay;
    }
  }

  const bool bf16 = L->dtype == DECATTN_BF16;
  const uint64_t rows_total = static_cast<uint64_t>(L->num_blocks) * L->block_size;
  const uint32_t box_rows = static_cast<uint32_t>(L->block_size < kTile ? L->block_size : kTile);
  CUtensorMap tk, tv;
  if (fp8) {
    // One byte per element: a token's 128-d head is one 128-byte box row.
    const uint64_t row_bytes = static_cast<uint64_t>(h_kv) * kHeadDim;
    if (!make_map_2d_t(&tk, k_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, row_bytes, rows_total,
                       row_bytes, kHeadDim, box_rows) ||
        !make_map_2d_t(&tv, v_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, row_bytes, rows_total,
                       row_bytes, kHeadDim, box_rows))
      return DECATTN_ERR_CUDA;
  } else if (h_q / h_kv <= kWideGroup) {
    // The CUDA-core / mma.sync consumers: a 3-D view [2 h_kv halves][rows][64]
    // (strides: a token row, then 128 B per 64-column half), so that one box
    // brings box_rows rows of both halves of a KV head (landing half-major).
    const uint64_t row_bytes = static_cast<uint64_t>(h_kv) * kHeadDim * 2;
    if (!make_map_3d_strided(&tk, k_cache, bf16, 64, rows_total, 2 * static_cast<uint64_t>(h_kv),
                             row_bytes, 128, 64, box_rows, 2) ||
        !make_map_3d_strided(&tv, v_cache, bf16, 64, rows_total, 2 * static_cast<uint64_t>(h_kv),
                             row_bytes, 128, 64, box_rows, 2))
      return DECATTN_ERR_CUDA;
  } else {
    // The tcgen05 kernel of wide groups: 2-D boxes of one 64-column half.
    const uint64_t row_bytes = static_cast<uint64_t>(h_kv) * kHeadDim * 2;
    if (!make_map_2d(&tk, k_cache, bf16, static_cast<uint64_t>(h_kv) * kHeadDim, rows_total,
                     row_bytes, 64, box_rows) ||
        !make_map_2d(&tv, v_cache, bf16, static_cast<uint64_t>(h_kv) * kHeadDim, rows_total,
                     row_bytes, 64, box_rows))
      return DECATTN_ERR_CUDA;
  }

  cudaStream_t stream = static_cast<cudaStream_t>(L->stream);
  const cudaError_t e = fp8 ? launch_gqa_partial_fp8(p, tk, tv, bf16, stream)
                            : launch_gqa_partial(p, tk, tv, bf16, 0, stream);
  if (e != cudaSuccess) return DECATTN_ERR_CUDA;
  if (more.weights) {
    const int sms = device_sm_count();
    if (sms <= 0) return DECATTN_ERR_CUDA;
    return launch_weigh(p, bf16, sms, stream) == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
  }
  if (eff > 1 && !p.joint) {
    CombineParams c{p.part_o, p.part_lse, out, L->batch * h_q, eff};
    if (launch_combine(c, kHeadDim, bf16, stream) != cudaSuccess) return DECATTN_ERR_CUDA;
  }
  return DECATTN_OK;
}

int gqa_decode(const void* q, const void* k_cache, const void* v_cache,
               const int32_t* block_table, const int32_t* seq_lens, void* out, int h_q, int h_kv,
               int d_head, float scale, const decattn_launch* L) {
  return gqa_decode_impl(q, k_cache, v_cache, nullptr, nullptr, false, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, 0, 0, L);
}

int gqa_decode_fp8kv(const void* q, const void* k_cache, const void* v_cache,
                     const float* k_scale, const float* v_scale, const int32_t* block_table,
                     const int32_t* seq_lens, void* out, int h_q, int h_kv, int d_head,
                     float scale, const decattn_launch* L) {
  return gqa_decode_impl(q, k_cache, v_cache, k_scale, v_scale, true, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, 0, 0, L);
}

int gqa_decode_window(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_table, const int32_t* seq_lens, void* out, int h_q,
                      int h_kv, int d_head, float scale, int window, const decattn_launch* L) {
  if (window < 1) return DECATTN_ERR_INVALID_ARG;
  return gqa_decode_impl(q, k_cache, v_cache, nullptr, nullptr, false, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, window, 0, L);
}

int gqa_decode_fp8kv_window(const void* q, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale,
                            const int32_t* block_table, const int32_t* seq_lens, void* out,
                            int h_q, int h_kv, int d_head, float scale, int window,
                            const decattn_launch* L) {
  if (window < 1) return DECATTN_ERR_INVALID_ARG;
  return gqa_decode_impl(q, k_cache, v_cache, k_scale, v_scale, true, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, window, 0, L);
}

int gqa_decode_sinks(const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_table, const int32_t* seq_lens, void* out, int h_q,
                     int h_kv, int d_head, float scale, int window, int sinks,
                     const decattn_launch* L) {
  if (window < 1 || sinks < 0) return DECATTN_ERR_INVALID_ARG;
  return gqa_decode_impl(q, k_cache, v_cache, nullptr, nullptr, false, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, window, sinks, L);
}

int gqa_decode_fp8kv_sinks(const void* q, const void* k_cache, const void* v_cache,
                           const float* k_scale, const float* v_scale,
                           const int32_t* block_table, const int32_t* seq_lens, void* out,
                           int h_q, int h_kv, int d_head, float scale, int window, int sinks,
                           const decattn_launch* L) {
  if (window < 1 || sinks < 0) return DECATTN_ERR_INVALID_ARG;
  return gqa_decode_impl(q, k_cache, v_cache, k_scale, v_scale, true, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, window, sinks, L);
}

// Lengths (of sequences, of lists) beyond which a 32-bit position has no room for a CTA's step.
static bool too_many(int n) { return n > 0x7fffffff - 65536; }
static bool too_long(const decattn_launch* L) { return L && too_many(L->max_seq_len); }

static int decode_blocks(const void* q, const void* k_cache, const void* v_cache,
                         const float* k_scale, const float* v_scale, bool fp8,
                         const int32_t* block_table, const int32_t* seq_lens,
                         const int32_t* selected, void* out, int h_q, int h_kv, int d_head,
                         float scale, int count, const decattn_launch* L) {
  if (!selected || !aligned(selected, 4) || count < 1) return DECATTN_ERR_INVALID_ARG;
  if (too_long(L) || too_many(count)) return DECATTN_ERR_UNSUPPORTED;
  DecodeMore more;
  more.selected = selected;
  more.count = count;
  return gqa_decode_impl(q, k_cache, v_cache, k_scale, v_scale, fp8, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, 0, 0, L, more);
}

int gqa_decode_blocks(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_table, const int32_t* seq_lens,
                      const int32_t* selected, void* out, int h_q, int h_kv, int d_head,
                      float scale, int count, const decattn_launch* L) {
  return decode_blocks(q, k_cache, v_cache, nullptr, nullptr, false, block_table, seq_lens,
                       selected, out, h_q, h_kv, d_head, scale, count, L);
}

int gqa_decode_fp8kv_blocks(const void* q, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale,
                            const int32_t* block_table, const int32_t* seq_lens,
                            const int32_t* selected, void* out, int h_q, int h_kv, int d_head,
                            float scale, int count, const decattn_launch* L) {
  return decode_blocks(q, k_cache, v_cache, k_scale, v_scale, true, block_table, seq_lens,
                       selected, out, h_q, h_kv, d_head, scale, count, L);
}

static int decode_weights(const void* q, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, bool fp8,
                          const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* weighed_lens, float* weights, void* out, int h_q,
                          int h_kv, int d_head, float scale, float decay,
                          const decattn_launch* L) {
  if (!weights || !aligned(weights, 16) || !aligned(weighed_lens, 4) || !std::isfinite(decay))
    return DECATTN_ERR_INVALID_ARG;
  if (too_long(L)) return DECATTN_ERR_UNSUPPORTED;
  DecodeMore more;
  more.weights = weights;
  more.weighed_lens = weighed_lens;
  more.decay = decay;
  return gqa_decode_impl(q, k_cache, v_cache, k_scale, v_scale, fp8, block_table, seq_lens, out,
                         h_q, h_kv, d_head, scale, 0, 0, L, more);
}

int gqa_decode_weights(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* seq_lens,
                       const int32_t* weighed_lens, float* weights, void* out, int h_q, int h_kv,
                       int d_head, float scale, float decay, const decattn_launch* L) {
  return decode_weights(q, k_cache, v_cache, nullptr, nullptr, false, block_table, seq_lens,
                        weighed_lens, weights, out, h_q, h_kv, d_head, scale, decay, L);
}

int gqa_decode_fp8kv_weights(const void* q, const void* k_cache, const void* v_cache,
                             const float* k_scale, const float* v_scale,
                             const int32_t* block_table, const int32_t* seq_lens,
                             const int32_t* weighed_lens, float* weights, void* out, int h_q,
                             int h_kv, int d_head, float scale, float decay,
                             const decattn_launch* L) {
  return decode_weights(q, k_cache, v_cache, k_scale, v_scale, true, block_table, seq_lens,
                        weighed_lens, weights, out, h_q, h_kv, d_head, scale, decay, L);
}

int gqa_block_bounds(const void* k_cache, const int32_t* block_table, const int32_t* first_lens,
                     const int32_t* seq_lens, void* bounds, int h_kv, int d_head, int kv_bytes,
                     const decattn_launch* L) {
  const int st = check_launch(L, false);
  if (st != DECATTN_OK) return st;
  if (!k_cache || !block_table || !seq_lens || !bounds || k_cache == bounds)
    return DECATTN_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) ||
      !aligned(first_lens, 4) || !aligned(seq_lens, 4))
    return DECATTN_ERR_INVALID_ARG;
  if (h_kv < 1 || h_kv > 1024 || (kv_bytes != 1 && kv_bytes != 2)) return DECATTN_ERR_INVALID_ARG;
  if (d_head != kHeadDim || too_long(L)) return DECATTN_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return DECATTN_ERR_CUDA;
  BoundsParams p{};
  p.k_cache = k_cache;
  p.block_table = block_table;
  p.first_lens = first_lens;
  p.seq_lens = seq_lens;
  p.bounds = bounds;
  p.err_flag = L->err_flag;
  p.batch = L->batch;
  p.h_kv = h_kv;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  p.max_seq_len = L->max_seq_len;
  const cudaError_t e = launch_block_bounds(p, kv_bytes == 1, L->dtype == DECATTN_BF16, sms,
                                            static_cast<cudaStream_t>(L->stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

static int64_t select_blocks_of(int max_seq_len, int block_size) {
  return (static_cast<int64_t>(max_seq_len) + block_size - 1) / block_size;
}

size_t gqa_select_workspace_size(int batch, int h_kv, int max_seq_len, int block_size, int count) {
  if (batch < 1 || h_kv < 1 || max_seq_len < 0 || !is_pow2(block_size) || count < 1) return 0;
  const int64_t blocks = select_blocks_of(max_seq_len, block_size);
  if (blocks <= count) return 0;
  const size_t units = static_cast<size_t>(batch) * h_kv, stride = (blocks + 15) / 16 * 16;
  return align_up(units * stride * sizeof(uint64_t)) + align_up(units * stride * sizeof(float)) +
         align_up(units * (stride / 16) * sizeof(uint4));
}

int gqa_select_blocks(const void* q, const void* bounds, const int32_t* block_table,
                      const int32_t* seq_lens, int32_t* selected, int h_q, int h_kv, int d_head,
                      int kv_bytes, int count, int first, int last, const decattn_launch* L) {
  const int st = check_launch(L, false);
  if (st != DECATTN_OK) return st;
  if (!q || !bounds || !block_table || !seq_lens || !selected) return DECATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(selected, 4))
    return DECATTN_ERR_INVALID_ARG;
  if (h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || (kv_bytes != 1 && kv_bytes != 2))
    return DECATTN_ERR_INVALID_ARG;
  if (count < 1 || first < 0 || last < 0 || static_cast<int64_t>(first) + last > count)
    return DECATTN_ERR_INVALID_ARG;
  if (d_head != kHeadDim || h_q / h_kv > 64 || L->batch > 65535 || h_kv > 65535 || too_long(L) ||
      too_many(count))
    return DECATTN_ERR_UNSUPPORTED;
  const int64_t blocks = select_blocks_of(L->max_seq_len, L->block_size);
  SelectParams p{};
  p.q = q;
  p.bounds = bounds;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.selected = selected;
  p.err_flag = L->err_flag;
  p.score_stride = (blocks + 15) / 16 * 16;
  p.batch = L->batch;
  p.h_kv = h_kv;
  p.group = h_q / h_kv;
  p.count = count;
  p.first = first;
  p.last = last;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  p.max_seq_len = L->max_seq_len;
  const size_t need =
      gqa_select_workspace_size(L->batch, h_kv, L->max_seq_len, L->block_size, count);
  if (need > 0 && (!L->workspace || L->workspace_bytes < need)) return DECATTN_ERR_WORKSPACE;
  const int sms = device_sm_count();
  if (sms <= 0) return DECATTN_ERR_CUDA;
  plan_choice(p, static_cast<int>(blocks), sms);
  if (blocks > count) {
    plan_scores(p, static_cast<int>(blocks), sms);
    const size_t all = static_cast<size_t>(L->batch) * h_kv * p.score_stride;
    char* ws = static_cast<char*>(L->workspace);
    p.exact = reinterpret_cast<uint64_t*>(ws);
    ws += align_up(all * sizeof(uint64_t));
    p.scores = reinterpret_cast<float*>(ws);
    ws += align_up(all * sizeof(float));
    p.parts = reinterpret_cast<uint4*>(ws);
  }
  const cudaError_t e = launch_select_blocks(p, kv_bytes == 1, L->dtype == DECATTN_BF16,
                                             static_cast<cudaStream_t>(L->stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int gqa_kv_evict(void* k_cache, void* v_cache, float* weights, const int32_t* block_table,
                 const int32_t* seq_lens, int32_t* new_lens, int32_t* kept, int h_kv, int d_head,
                 int kv_bytes, int keep, int recent, int limit, const decattn_launch* L) {
  const int st = check_launch(L, false);
  if (st != DECATTN_OK) return st;
  if (!k_cache || !v_cache || !weights || !block_table || !seq_lens || !new_lens || !kept ||
      k_cache == v_cache || new_lens == seq_lens)
    return DECATTN_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(new_lens, 4) ||
      !aligned(kept, 4))
    return DECATTN_ERR_INVALID_ARG;
  if (h_kv < 1 || h_kv > 1024 || (kv_bytes != 1 && kv_bytes != 2)) return DECATTN_ERR_INVALID_ARG;
  if (keep < 1 || recent < 0 || recent > keep || limit < keep) return DECATTN_ERR_INVALID_ARG;
  if (d_head != kHeadDim || L->batch > 65535 || too_long(L) || too_many(keep))
    return DECATTN_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return DECATTN_ERR_CUDA;
  EvictParams p{};
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.weights = weights;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.kept = kept;
  p.err_flag = L->err_flag;
  p.batch = L->batch;
  p.h_kv = h_kv;
  p.head_bytes = kHeadDim * kv_bytes;
  p.keep = keep;
  p.recent = recent;
  p.limit = limit;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  p.max_seq_len = L->max_seq_len;
  const cudaError_t e = launch_kv_evict(p, sms, static_cast<cudaStream_t>(L->stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int mla_decode(const void* q_absorbed, const void* q_rope, const void* latent_cache,
               const int32_t* block_table, const int32_t* seq_lens, void* out, float scale,
               const decattn_launch* L) {
  int st = check_launch(L, true);
  if (st != DECATTN_OK) return st;
  if (!q_absorbed || !q_rope || !latent_cache || !block_table || !seq_lens || !out)
    return DECATTN_ERR_INVALID_ARG;
  if (!aligned(q_absorbed, 16) || !aligned(q_rope, 16) || !aligned(latent_cache, 16) ||
      !aligned(out, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return DECATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return DECATTN_ERR_INVALID_ARG;

  int n_pairs = L->num_splits;
  if (n_pairs == 0) {
    const int sms = device_sm_count();
    if (sms <= 0) return DECATTN_ERR_CUDA;
    n_pairs = plan_mla_splits(L->batch, L->max_seq_len, sms);
  }

  MlaParams p{};
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.err_flag = L->err_flag;
  p.batch = L->batch;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  p.max_seq_len = L->max_seq_len;
  p.n_pairs = n_pairs;
  p.scale_log2 = scale * 1.4426950408889634f;
  if (n_pairs > 1) {
    size_t off_lse = 0, off_o = 0;
    const size_t need = mla_workspace_bytes(L->batch, n_pairs, &off_lse, &off_o);
    if (!L->workspace || L->workspace_bytes < need) return DECATTN_ERR_WORKSPACE;
    char* ws = static_cast<char*>(L->workspace);
    p.ws_hdr = reinterpret_cast<int*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + off_lse);
    p.part_o = reinterpret_cast<float*>(ws + off_o);
  }

  const bool bf16 = L->dtype == DECATTN_BF16;
  const uint64_t c_rows = static_cast<uint64_t>(L->num_blocks) * L->block_size;
  const uint64_t q_rows = static_cast<uint64_t>(L->batch) * kMlaHeads;
  CUtensorMap tqa, tc, tc4, tout, tpo;
  if (!make_map_2d(&tqa, q_absorbed, bf16, kMlaDc, q_rows, kMlaDc * 2, 64, kMlaHeads) ||
      !make_map_2d(&tc, latent_cache, bf16, kMlaWidth, c_rows, kMlaWidth * 2, 64,
                   static_cast<uint32_t>(L->block_size < 64 ? L->block_size : 64)) ||
      !make_map_2d(&tout, out, bf16, kMlaDc, q_rows, kMlaDc * 2, 64, kMlaHeads))
    return DECATTN_ERR_CUDA;
  // check_launch caps MLA blocks at 64 rows, so block size 64 is exactly the
  // case in which the kernel takes one 64-row box per tile and copies four
  // chunks at once through tc4.
  if (L->block_size >= 64) {
    if (!make_map_3d_strided(&tc4, latent_cache, bf16, 64, c_rows, kMlaWidth / 64, kMlaWidth * 2,
                             128, 64, 64, 4))
      return DECATTN_ERR_CUDA;
  } else {
    tc4 = tc;  // never used: smaller blocks take one 2-D copy per chunk and block
  }
  if (n_pairs > 1) {
    if (!make_map_2d_t(&tpo, p.part_o, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, kMlaDc,
                       2ull * n_pairs * kMlaHeads, kMlaDc * 4, 32, kMlaHeads))
      return DECATTN_ERR_CUDA;
  } else {
    tpo = tout;  // never used: every segment of a single pair is whole
  }
  p.q_abs = q_absorbed;
  p.q_rope = q_rope;

  cudaStream_t stream = static_cast<cudaStream_t>(L->stream);
  cudaError_t e = launch_mla_partial(p, tqa, tc, tc4, tout, tpo, bf16, stream);
  if (e == cudaErrorNotSupported) return DECATTN_ERR_UNSUPPORTED;
  if (e != cudaSuccess) return DECATTN_ERR_CUDA;
  if (n_pairs > 1) {
    MlaCombineParams c{p.part_o, p.part_lse, p.ws_hdr, out, L->batch, n_pairs};
    if (launch_mla_combine(c, bf16, stream) != cudaSuccess) return DECATTN_ERR_CUDA;
  }
  return DECATTN_OK;
}

// The decode step's cache write (gqa_kv_append, gqa_kv_append_fp8kv,
// mla_kv_append): host checks, then one launch for K and V.
static int kv_append_impl(const void* k_new, const void* v_new, const float* k_scale,
                          const float* v_scale, bool e4m3, const int32_t* positions,
                          const int32_t* block_table, void* k_cache, void* v_cache, int row_elems,
                          int head_elems, bool mla, const decattn_launch* L) {
  if (!L) return DECATTN_ERR_INVALID_ARG;
  if (L->batch < 1 || L->num_blocks < 1 || L->max_blocks_per_seq < 1)
    return DECATTN_ERR_INVALID_ARG;
  if (L->dtype != DECATTN_FP16 && L->dtype != DECATTN_BF16) return DECATTN_ERR_INVALID_ARG;
  if (!is_pow2(L->block_size)) return DECATTN_ERR_INVALID_ARG;
  if (L->block_size < 8 || L->block_size > (mla ? 64 : 256)) return DECATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(L->num_blocks) * L->block_size > 0x7fffffffLL)
    return DECATTN_ERR_UNSUPPORTED;
  if (!k_new || !k_cache || !positions || !block_table) return DECATTN_ERR_INVALID_ARG;
  if (!mla && (!v_new || !v_cache)) return DECATTN_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(k_cache, 16) || !aligned(positions, 4) ||
      !aligned(block_table, 4) || (v_new && !aligned(v_new, 16)) ||
      (v_cache && !aligned(v_cache, 16)))
    return DECATTN_ERR_INVALID_ARG;
  if (e4m3 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
    return DECATTN_ERR_INVALID_ARG;
  if (L->err_flag && !aligned(L->err_flag, 4)) return DECATTN_ERR_INVALID_ARG;

  AppendParams p{};
  p.k_new = k_new;
  p.v_new = mla ? nullptr : v_new;
  p.positions = positions;
  p.block_table = block_table;
  p.k_cache = k_cache;
  p.v_cache = mla ? nullptr : v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err_flag = L->err_flag;
  p.batch = L->batch;
  p.row_elems = row_elems;
  p.head_elems = head_elems;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  const cudaError_t e = launch_append(p, e4m3, L->dtype == DECATTN_BF16,
                                      static_cast<cudaStream_t>(L->stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int gqa_kv_append(const void* k_new, const void* v_new, const int32_t* positions,
                  const int32_t* block_table, void* k_cache, void* v_cache, int h_kv, int d_head,
                  const decattn_launch* L) {
  if (h_kv < 1 || h_kv > 1024) return DECATTN_ERR_INVALID_ARG;
  if (d_head != kHeadDim) return DECATTN_ERR_UNSUPPORTED;
  return kv_append_impl(k_new, v_new, nullptr, nullptr, false, positions, block_table, k_cache,
                        v_cache, h_kv * kHeadDim, kHeadDim, false, L);
}

int gqa_kv_append_fp8kv(const void* k_new, const void* v_new, const float* k_scale,
                        const float* v_scale, const int32_t* positions,
                        const int32_t* block_table, void* k_cache, void* v_cache, int h_kv,
                        int d_head, const decattn_launch* L) {
  if (h_kv < 1 || h_kv > 1024) return DECATTN_ERR_INVALID_ARG;
  if (d_head != kHeadDim) return DECATTN_ERR_UNSUPPORTED;
  return kv_append_impl(k_new, v_new, k_scale, v_scale, true, positions, block_table, k_cache,
                        v_cache, h_kv * kHeadDim, kHeadDim, false, L);
}

int mla_kv_append(const void* latent_new, const int32_t* positions, const int32_t* block_table,
                  void* latent_cache, const decattn_launch* L) {
  return kv_append_impl(latent_new, nullptr, nullptr, nullptr, false, positions, block_table,
                        latent_cache, nullptr, kMlaWidth, kMlaWidth, true, L);
}

int paged_plan(const int32_t* cached_lens, const int32_t* new_lens, int32_t* block_table,
               int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out,
               int32_t* seq_lens, int32_t* q_start, int32_t* slots, int32_t* positions,
               int max_tokens, const decattn_launch* L) {
  if (!L) return DECATTN_ERR_INVALID_ARG;
  if (L->batch < 1 || L->num_blocks < 1 || L->max_blocks_per_seq < 1 || max_tokens < 0)
    return DECATTN_ERR_INVALID_ARG;
  if (!is_pow2(L->block_size)) return DECATTN_ERR_INVALID_ARG;
  if (L->block_size < 8 || L->block_size > 256 || L->batch > kPlanMaxBatch)
    return DECATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(L->num_blocks) * L->block_size > 0x7fffffffLL ||
      static_cast<int64_t>(L->max_blocks_per_seq) * L->block_size > 0x7fffffffLL - 256)
    return DECATTN_ERR_UNSUPPORTED;
  const void* all[] = {cached_lens, new_lens, block_table, free_blocks, free_count,
                       free_count_out, seq_lens, q_start};
  for (const void* a : all)
    if (!a || !aligned(a, 4)) return DECATTN_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!slots || !positions)) return DECATTN_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(positions, 4)) return DECATTN_ERR_INVALID_ARG;
  if (L->err_flag && !aligned(L->err_flag, 4)) return DECATTN_ERR_INVALID_ARG;
  PlanParams p{};
  p.cached_lens = cached_lens;
  p.new_lens = new_lens;
  p.block_table = block_table;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.seq_lens = seq_lens;
  p.q_start = q_start;
  p.slots = slots;
  p.positions = positions;
  p.err_flag = L->err_flag;
  p.batch = L->batch;
  p.max_tokens = max_tokens;
  p.in_place = seq_lens == cached_lens || free_count_out == free_count;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  const cudaError_t e = launch_paged_plan(p, static_cast<cudaStream_t>(L->stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int decattn_rope_fill(decattn_rope* rope, const double* inv_freq, int rot_dim,
                      const int* sections, int n_axes, int interleaved) {
  if (!rope || !inv_freq || n_axes < 1 || n_axes > 8 || (interleaved != 0 && interleaved != 1))
    return DECATTN_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > kHeadDim || rot_dim % 16 != 0) return DECATTN_ERR_UNSUPPORTED;
  if (!sections && n_axes != 1) return DECATTN_ERR_INVALID_ARG;
  const int pairs = rot_dim / 2;
  int64_t sum = 0;
  for (int a = 0; sections && a < n_axes; ++a) {
    if (sections[a] < 0) return DECATTN_ERR_INVALID_ARG;
    sum += sections[a];
  }
  if (sections && sum != pairs) return DECATTN_ERR_INVALID_ARG;
  for (int i = 0; i < pairs; ++i)
    if (!std::isfinite(inv_freq[i])) return DECATTN_ERR_INVALID_ARG;
  *rope = decattn_rope{};
  rope->rot_dim = rot_dim;
  rope->n_axes = n_axes;
  rope->interleaved = interleaved;
  int axis = 0, left = sections ? sections[0] : pairs;
  for (int i = 0; i < pairs; ++i) {
    while (left == 0) left = sections[++axis];
    --left;
    rope->axis[i] = static_cast<uint8_t>(axis);
    // Turns per position modulo one turn, as a 64-bit fraction.  The double
    // product's relative error of 2^-53 is the frequency's own precision.
    double turns = inv_freq[i] / 6.283185307179586476925286766559;
    turns -= std::floor(turns);
    const double scaled = std::ldexp(turns, 64);  // <= 2^64; exact
    rope->turns[i] = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
  }
  return DECATTN_OK;
}

static int rope_append_impl(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, const float* k_scale,
                            const float* v_scale, bool e4m3, const int32_t* positions,
                            const decattn_rope* rope, const int32_t* slots, void* q_out,
                            void* k_cache, void* v_cache, int tokens, int h_q, int h_kv,
                            int d_head, const decattn_launch* L) {
  if (!L || !rope) return DECATTN_ERR_INVALID_ARG;
  if (L->num_blocks < 1 || tokens < 0) return DECATTN_ERR_INVALID_ARG;
  if (L->dtype != DECATTN_FP16 && L->dtype != DECATTN_BF16) return DECATTN_ERR_INVALID_ARG;
  if (!is_pow2(L->block_size)) return DECATTN_ERR_INVALID_ARG;
  if (L->block_size < 8 || L->block_size > 256) return DECATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(L->num_blocks) * L->block_size > 0x7fffffffLL)
    return DECATTN_ERR_UNSUPPORTED;
  if (h_q < 1 || h_kv < 1 || h_q > (1 << 20) || h_kv > 1024) return DECATTN_ERR_INVALID_ARG;
  if (d_head != kHeadDim) return DECATTN_ERR_UNSUPPORTED;
  if (rope->rot_dim < 16 || rope->rot_dim > kHeadDim || rope->rot_dim % 16 != 0)
    return DECATTN_ERR_UNSUPPORTED;
  if (rope->n_axes < 1 || rope->n_axes > 8 || (rope->interleaved != 0 && rope->interleaved != 1))
    return DECATTN_ERR_INVALID_ARG;
  for (int i = 0; i < rope->rot_dim / 2; ++i)
    if (rope->axis[i] >= rope->n_axes) return DECATTN_ERR_INVALID_ARG;
  if (L->err_flag && !aligned(L->err_flag, 4)) return DECATTN_ERR_INVALID_ARG;
  if (tokens == 0) return DECATTN_OK;
  if (!q || !k_new || !v_new || !positions || !slots || !q_out || !k_cache || !v_cache)
    return DECATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(positions, 4) ||
      !aligned(slots, 4))
    return DECATTN_ERR_INVALID_ARG;
  if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 ||
      q_stride < static_cast<int64_t>(h_q) * kHeadDim ||
      k_stride < static_cast<int64_t>(h_kv) * kHeadDim ||
      v_stride < static_cast<int64_t>(h_kv) * kHeadDim)
    return DECATTN_ERR_INVALID_ARG;
  // In place only where every row stays where it is.
  if (q_out == q && q_stride != static_cast<int64_t>(h_q) * kHeadDim)
    return DECATTN_ERR_INVALID_ARG;
  if (e4m3 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
    return DECATTN_ERR_INVALID_ARG;
  RopeParams p{};
  p.q = q;
  p.k = k_new;
  p.v = v_new;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.positions = positions;
  p.slots = slots;
  p.err_flag = L->err_flag;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.tokens = tokens;
  p.h_q = h_q;
  p.h_kv = h_kv;
  p.num_slots = L->num_blocks * L->block_size;
  p.rope = *rope;
  const cudaError_t e = launch_rope_append(p, e4m3, L->dtype == DECATTN_BF16,
                                           static_cast<cudaStream_t>(L->stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int gqa_rope_append(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                    int64_t k_stride, int64_t v_stride, const int32_t* positions,
                    const decattn_rope* rope, const int32_t* slots, void* q_out, void* k_cache,
                    void* v_cache, int tokens, int h_q, int h_kv, int d_head,
                    const decattn_launch* L) {
  return rope_append_impl(q, k_new, v_new, q_stride, k_stride, v_stride, nullptr, nullptr, false,
                          positions, rope, slots, q_out, k_cache, v_cache, tokens, h_q, h_kv,
                          d_head, L);
}

int gqa_rope_append_fp8kv(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                          int64_t k_stride, int64_t v_stride, const float* k_scale,
                          const float* v_scale, const int32_t* positions,
                          const decattn_rope* rope, const int32_t* slots, void* q_out,
                          void* k_cache, void* v_cache, int tokens, int h_q, int h_kv,
                          int d_head, const decattn_launch* L) {
  return rope_append_impl(q, k_new, v_new, q_stride, k_stride, v_stride, k_scale, v_scale, true,
                          positions, rope, slots, q_out, k_cache, v_cache, tokens, h_q, h_kv,
                          d_head, L);
}

// Pieces (of two Q tiles) that a step's rows can at most be cut into.
static int64_t prefill_items(int batch, int tokens, int max_q_len, int group) {
  const int tpi = 2 * (128 / group);
  const int64_t by_rows = static_cast<int64_t>(tokens) / tpi + batch;
  const int64_t by_seq = static_cast<int64_t>(batch) *
                         ((static_cast<int64_t>(max_q_len) + tpi - 1) / tpi);
  return by_rows < by_seq ? by_rows : by_seq;
}

static int plan_prefill_splits(int batch, int tokens, int max_q_len, int h_q, int h_kv,
                               int max_seq_len, int window, int sinks, int sms) {
  const int64_t units = prefill_items(batch, tokens, max_q_len, h_q / h_kv) * h_kv;
  int64_t span = max_seq_len;
  if (window > 0) {
    const int64_t seen = static_cast<int64_t>(window) + max_q_len + sinks + 256;
    if (seen < span) span = seen;
  }
  const int64_t tiles = (span + 127) / 128;
  // One wave of one CTA per SM at most, and the number that takes least by this
  // count, in ns: a CTA's tiles (one Q tile's, two Q tiles'), and from two splits on
  // the combine, its chain over the splits and its traffic.  Measured, 8 KV heads:
  // 64 heads, 4 tokens over an 8k cache with 4 / 8 / 12 / 19 splits 31.0 / 25.0 /
  // 23.1 / 25.0 us, over 2k with 1 / 2 / 4 / 8 24.1 / 20.0 / 16.7 / 15.2, 8 over
  // 131k with 8 / 12 / 19 / 24 136 / 103 / 96 / 125 (24: a second wave), 2 x 64
  // over 8k with 2 / 3 / 4 / 6 66 / 52 / 44 / 60; 32 heads, 2 x 128 over 1k with
  // 1 / 2 / 4 24.9 / 23.0 / 21.0, 8 x 64 over 500 with 1 / 2 16.4 / 20.4.
  const int64_t tile_ns = max_q_len <= 128 / (h_q / h_kv) ? 950 : 1700;
  int64_t most = units > 0 ? sms / units : 1, ns = 1, best = tiles * tile_ns;
  if (most > tiles) most = tiles;
  if (most > DECATTN_MAX_SPLITS) most = DECATTN_MAX_SPLITS;
  for (int64_t n = 2; n <= most; ++n) {
    const int64_t cost = (tiles + n - 1) / n * tile_ns + 2000 + 300 * n +
                         static_cast<int64_t>(tokens) * h_q * n / 12;
    if (cost < best) {
      best = cost;
      ns = n;
    }
  }
  return static_cast<int>(ns);
}

size_t gqa_prefill_workspace_size(int tokens, int h_q, int d_head, int num_splits) {
  return gqa_decode_workspace_size(tokens, h_q, d_head, num_splits);
}

int gqa_prefill_plan_splits(int batch, int tokens, int max_q_len, int h_q, int h_kv, int d_head,
                            int max_seq_len, int window, int sinks, int num_sms) {
  if (batch < 1 || tokens < 0 || max_q_len < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 ||
      h_q / h_kv > 64 || d_head < 1 || max_seq_len < 0 || window < 0 || sinks < 0)
    return DECATTN_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return DECATTN_ERR_CUDA;
  return plan_prefill_splits(batch, tokens, max_q_len, h_q, h_kv, max_seq_len, window, sinks,
                             num_sms);
}

static int gqa_prefill_impl(const void* q, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale, bool fp8,
                            const int32_t* block_table, const int32_t* q_start,
                            const int32_t* seq_lens, void* out, int tokens, int max_q_len,
                            int h_q, int h_kv, int d_head, float scale, int window, int sinks,
                            const decattn_launch* L) {
  if (tokens < 0 || max_q_len < 1 || sinks < 0) return DECATTN_ERR_INVALID_ARG;
  if (tokens == 0) {
    // No row to compute: q and out may be null, the rest is still checked.
    static const uint4 nothing{};
    q = q ? q : &nothing;
    out = out ? out : const_cast<uint4*>(&nothing);
  }
  const int st = gqa_check_args(q, k_cache, v_cache, k_scale, v_scale, fp8, block_table,
                                seq_lens, out, h_q, h_kv, d_head, scale, window, L);
  if (st != DECATTN_OK) return st;
  window = useful_window(window, L->max_seq_len);
  if (!q_start || !aligned(q_start, 4)) return DECATTN_ERR_INVALID_ARG;
  // (Tile offsets and the step behind the last tile stay within 31 bits.)
  if (L->max_seq_len > 0x7fffffff - 4096) return DECATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return DECATTN_OK;
  const int group = h_q / h_kv;
  int sms = 0, ns = L->num_splits;
  if (ns == 0) {
    sms = device_sm_count();
    if (sms <= 0) return DECATTN_ERR_CUDA;
    ns = plan_prefill_splits(L->batch, tokens, max_q_len, h_q, h_kv, L->max_seq_len, window,
                             sinks, sms);
  }
  const int64_t items = prefill_items(L->batch, tokens, max_q_len, group);
  if (items * h_kv * ns > 0x7fffffffLL || static_cast<int64_t>(tokens) * h_q > 0x7fffffffLL)
    return DECATTN_ERR_UNSUPPORTED;
  PrefillParams p{};
  p.q = q;
  p.block_table = block_table;
  p.q_start = q_start;
  p.seq_lens = seq_lens;
  p.out = out;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err_flag = L->err_flag;
  p.batch = L->batch;
  p.tokens = tokens;
  p.max_q_len = max_q_len;
  p.h_q = h_q;
  p.h_kv = h_kv;
  p.group = group;
  p.block_size = L->block_size;
  p.log2_block_size = ilog2(L->block_size);
  p.num_blocks = L->num_blocks;
  p.max_blocks_per_seq = L->max_blocks_per_seq;
  p.max_seq_len = L->max_seq_len;
  p.window = window;
  p.sinks = window > 0 ? sinks : 0;
  p.tokens_per_tile = 128 / group;
  p.n_items = static_cast<int>(items);
  p.n_split = ns;
  p.negate = scale < 0.f ? 1 : 0;
  // A zero scale (equal weights) is a scale that no score can feel: the
  // kernel's masked scores are -inf, and -inf times 0 would be NaN.
  const float mag = std::fabs(scale) * 1.4426950408889634f;
  p.scale_log2 = mag > 1e-37f ? mag : 1e-37f;
  if (ns > 1) {
    const size_t need = gqa_prefill_workspace_size(tokens, h_q, d_head, ns);
    if (!L->workspace || L->workspace_bytes < need) return DECATTN_ERR_WORKSPACE;
    p.part_o = static_cast<float*>(L->workspace);
    p.part_lse = reinterpret_cast<float*>(
        static_cast<char*>(L->workspace) +
        align_up(static_cast<size_t>(tokens) * h_q * ns * d_head * sizeof(float)));
  }
  if (sms == 0) sms = device_sm_count();
  if (sms <= 0) return DECATTN_ERR_CUDA;
  p.once = max_q_len <= 2 * p.tokens_per_tile ? 1 : 0;
  p.steal = items * h_kv * ns > sms ? 1 : 0;
  const bool bf16 = L->dtype == DECATTN_BF16;
  const uint64_t rows_total = static_cast<uint64_t>(L->num_blocks) * L->block_size;
  const uint32_t box_rows = static_cast<uint32_t>(L->block_size < 128 ? L->block_size : 128);
  const uint64_t width = static_cast<uint64_t>(h_kv) * kHeadDim;
  CUtensorMap tq, tk, tv;
  if (!make_map_3d(&tq, q, bf16, kHeadDim, static_cast<uint64_t>(h_q),
                   static_cast<uint64_t>(tokens), 64, static_cast<uint32_t>(group),
                   static_cast<uint32_t>(p.tokens_per_tile)) ||
      !(fp8 ? make_map_2d_t(&tk, k_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, width, rows_total, width,
                            kHeadDim, box_rows) &&
                  make_map_2d_t(&tv, v_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, width, rows_total,
                                width, kHeadDim, box_rows)
            : make_map_2d(&tk, k_cache, bf16, width, rows_total, width * 2, 64, box_rows) &&
                  make_map_2d(&tv, v_cache, bf16, width, rows_total, width * 2, 64, box_rows)))
    return DECATTN_ERR_CUDA;
  const cudaError_t e =
      launch_gqa_prefill(p, tq, tk, tv, bf16, fp8, static_cast<cudaStream_t>(L->stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int gqa_prefill(const void* q, const void* k_cache, const void* v_cache,
                const int32_t* block_table, const int32_t* q_start, const int32_t* seq_lens,
                void* out, int tokens, int max_q_len, int h_q, int h_kv, int d_head, float scale,
                int window, int sinks, const decattn_launch* L) {
  return gqa_prefill_impl(q, k_cache, v_cache, nullptr, nullptr, false, block_table, q_start,
                          seq_lens, out, tokens, max_q_len, h_q, h_kv, d_head, scale, window,
                          sinks, L);
}

int gqa_prefill_fp8kv(const void* q, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale, const int32_t* block_table,
                      const int32_t* q_start, const int32_t* seq_lens, void* out, int tokens,
                      int max_q_len, int h_q, int h_kv, int d_head, float scale, int window,
                      int sinks, const decattn_launch* L) {
  return gqa_prefill_impl(q, k_cache, v_cache, k_scale, v_scale, true, block_table, q_start,
                          seq_lens, out, tokens, max_q_len, h_q, h_kv, d_head, scale, window,
                          sinks, L);
}

// MLA's absorption GEMMs: Y[b, i, :] = X[b, i, :] W_i^T for every head i.
static int head_gemm_impl(const void* x, const void* w, void* y, int batch, int heads, int m,
                          int k, int dtype, int* err_flag, void* stream) {
  if (!x || !w || !y) return DECATTN_ERR_INVALID_ARG;
  if (batch < 1 || heads < 1 || m < 1 || k < 1) return DECATTN_ERR_INVALID_ARG;
  if (dtype != DECATTN_FP16 && dtype != DECATTN_BF16) return DECATTN_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16)) return DECATTN_ERR_INVALID_ARG;
  if (err_flag && !aligned(err_flag, 4)) return DECATTN_ERR_INVALID_ARG;
  if (m % 128 != 0 || k % 64 != 0 || heads > 65535) return DECATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(heads) * m > 0x7fffffffLL ||
      static_cast<int64_t>(batch) * heads * m > (1LL << 40))
    return DECATTN_ERR_UNSUPPORTED;
  HeadGemmParams p{};
  p.out = y;
  p.err_flag = err_flag;
  p.batch = batch;
  p.heads = heads;
  p.m = m;
  p.k = k;
  const int b16 = (batch + 15) / 16 * 16;
  p.n_tile = b16 < 256 ? b16 : 256;
  if ((batch + p.n_tile - 1) / p.n_tile > 65535) return DECATTN_ERR_UNSUPPORTED;
  // Ring stages: up to 8, within ~100 KB of shared memory, so that two CTAs
  // fit an SM and a call launched right after this one (a programmatic
  // dependent) can start streaming its weights while this one finishes
  // (DeepSeek-V2 out GEMM, B = 32, 8 layers' weights in turn: 6.99 us with
  // 8 stages and one CTA per SM).
  const int stage_bytes = 128 * 128 + p.n_tile * 128;
  int stages = (100 * 1024) / stage_bytes;
  stages = stages < 2 ? 2 : (stages > 8 ? 8 : stages);
  p.stages = k / 64 < stages ? k / 64 : stages;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.n_tile) p.tmem_cols *= 2;
  const bool bf16 = dtype == DECATTN_BF16;
  CUtensorMap tw, tx, ty;
  if (!make_map_2d(&tw, w, bf16, static_cast<uint64_t>(k), static_cast<uint64_t>(heads) * m,
                   static_cast<uint64_t>(k) * 2, 64, 128) ||
      !make_map_3d(&tx, x, bf16, static_cast<uint64_t>(k), static_cast<uint64_t>(heads),
                   static_cast<uint64_t>(batch), 64, 1, static_cast<uint32_t>(p.n_tile)) ||
      !make_map_3d(&ty, y, bf16, static_cast<uint64_t>(m), static_cast<uint64_t>(heads),
                   static_cast<uint64_t>(batch), 64, 1, static_cast<uint32_t>(p.n_tile),
                   CU_TENSOR_MAP_SWIZZLE_NONE))
    return DECATTN_ERR_CUDA;
  const cudaError_t e = launch_head_gemm(p, tw, tx, ty, bf16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DECATTN_OK : DECATTN_ERR_CUDA;
}

int mla_absorb_q(const void* q_nope, const void* w_uk, void* q_abs, int batch, int n_heads,
                 int d_h, int d_c, int dtype, int* err_flag, void* stream) {
  return head_gemm_impl(q_nope, w_uk, q_abs, batch, n_heads, d_c, d_h, dtype, err_flag, stream);
}

int mla_unabsorb_out(const void* o_lat, const void* w_uv_t, void* out, int batch, int n_heads,
                     int d_c, int d_v, int dtype, int* err_flag, void* stream) {
  return head_gemm_impl(o_lat, w_uv_t, out, batch, n_heads, d_v, d_c, dtype, err_flag, stream);
}

}  // extern "C"
