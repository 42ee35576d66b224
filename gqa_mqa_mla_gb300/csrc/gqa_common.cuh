// gqa_common.cuh -- the per-CTA token range and bad-data handling shared by
// the GQA partial kernels (one CTA per split, KV head j and sequence b).
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace decattn {

// Token range [t_begin, t_end) of split `split` of sequence b, the window
// start w0 ("07 · MHA/MQA/GQA/MLA quick learn": each token attends only to
// the last W tokens), and this thread's share of the validity checks.
// Tiles start at the block (or 64-token) boundary holding w0; blocks wholly
// before the window are never read.  `bad` is this thread's verdict only: the
// caller ORs it over the CTA (block ids are checked strided by threadIdx.x).
//
// kSinks: the sequence's first s_end = min(sinks, w0) tokens stay visible
// too.  Its tiles are then those of [0, s_end) followed by those from the
// window's boundary on, numbered through and dealt out to the splits in that
// order; a tile holds tokens of one of the two ranges only, so no token is
// counted twice where both ranges meet in one block.  With sinks >= w0 the
// ranges join: plain attention over the whole sequence.
struct GqaTile {
  int t0;    // first token
  int skip;  // rows [skip, nval) of the tile's 64 are attended
  int nval;
};

template <bool kSinks>
struct GqaSpan {
  int w0, t_begin, t_end, bad;
  int n_tiles;
  // kSinks only, in tokens counted from this split's first tile: one past the
  // last sink, the window's start and end; and the first token of the split's
  // tiles if they are sinks' (sink0) or the window's (win0).  (Few values: at
  // 175 registers instead of 168 the 16-bit kernel ran one CTA per SM, not
  // two, 211 us instead of 165 at 64 x 4100 tokens of 8 KV heads.)
  int s_rel, w_rel, e_rel, sink0, win0;

  DECATTN_DEV GqaTile tile(int it) const {
    GqaTile r;
    if constexpr (kSinks) {
      const int o = it * kTile;
      const bool sink = o < s_rel;
      r.t0 = (sink ? sink0 : win0) + o;
      r.skip = sink ? 0 : max(0, w_rel - o);
      r.nval = min(kTile, (sink ? s_rel : e_rel) - o);
    } else {
      r.t0 = t_begin + it * kTile;
      r.skip = max(0, w0 - r.t0);
      r.nval = min(kTile, t_end - r.t0);
    }
    return r;
  }
  DECATTN_DEV bool empty() const { return kSinks ? n_tiles <= 0 : t_end <= t_begin; }
  // One past the last token whose block may be read.
  DECATTN_DEV int end() const { return kSinks ? win0 + e_rel : t_end; }
};

// 1 (and the flag) if a block id of tokens [t0, t1) is out of range.
DECATTN_DEV int gqa_bad_blocks(const GqaParams& p, int b, int t0, int t1) {
  int bad = 0;
  const int32_t* bt = p.block_table + static_cast<size_t>(b) * p.max_blocks_per_seq;
  const int k1 = (t1 - 1) >> p.log2_block_size;
  for (int k = (t0 >> p.log2_block_size) + threadIdx.x; k <= k1; k += blockDim.x) {
    const int id = bt[k];
    if (id < 0 || id >= p.num_blocks) {
      bad = 1;
      flag_error(p.err_flag, kFlagBadBlock);
    }
  }
  return bad;
}

template <bool kSinks = false>
DECATTN_DEV GqaSpan<kSinks> gqa_span(const GqaParams& p, int split, int j, int b) {
  GqaSpan<kSinks> r;
  const int seq_len = p.seq_lens[b];
  r.bad = 0;
  if (seq_len < 0 || seq_len > p.max_seq_len) {
    r.bad = 1;
    if (threadIdx.x == 0 && split == 0 && j == 0) flag_error(p.err_flag, kFlagBadSeqLen);
  }
  r.w0 = (p.window > 0 && seq_len > p.window) ? seq_len - p.window : 0;
  if (kSinks && p.sinks >= r.w0) r.w0 = 0;
  const int base = r.w0 & ~((p.block_size < kTile ? p.block_size : kTile) - 1);
  if constexpr (kSinks) {
    r.t_begin = r.t_end = 0;
    r.n_tiles = 0;
    if (r.bad) return r;
    const int s_end = min(p.sinks, r.w0);
    const int sink_tiles = (s_end + kTile - 1) / kTile;
    const int total = sink_tiles + (seq_len - base + kTile - 1) / kTile;
    const int per = p.tokens_per_split / kTile;
    const int tile0 = min(split * per, total);
    r.n_tiles = min(per, total - tile0);
    if (r.n_tiles <= 0) return r;
    r.sink0 = tile0 * kTile;
    r.win0 = base + (tile0 - sink_tiles) * kTile;
    r.s_rel = s_end - r.sink0;
    r.w_rel = r.w0 - r.win0;
    r.e_rel = seq_len - r.win0;
    const int end = tile0 + r.n_tiles;
    if (tile0 < sink_tiles) r.bad |= gqa_bad_blocks(p, b, r.sink0, min(s_end, end * kTile));
    if (end > sink_tiles)
      r.bad |= gqa_bad_blocks(p, b, base + max(0, tile0 - sink_tiles) * kTile,
                              min(seq_len, base + (end - sink_tiles) * kTile));
  } else {
    r.t_begin = base + split * p.tokens_per_split;
    r.t_end = r.bad ? r.t_begin : min(seq_len, r.t_begin + p.tokens_per_split);
    if (!r.bad && r.t_end > r.t_begin) r.bad = gqa_bad_blocks(p, b, r.t_begin, r.t_end);
    r.n_tiles = (r.t_end - r.t_begin + kTile - 1) / kTile;
  }
  return r;
}

// Rows row0 .. row0 + rows - 1 of a CTA that met bad data (zeros plus the
// poison marker for the combine) or an empty token range (zeros, lse = -inf).
DECATTN_DEV void gqa_write_empty(const GqaParams& p, size_t row0, int rows, int split, bool bad) {
  for (int e = threadIdx.x; e < rows * kHeadDim; e += blockDim.x) {
    const int r = e / kHeadDim, d = e % kHeadDim;
    if (p.n_split == 1) {
      static_cast<uint16_t*>(p.out)[(row0 + r) * kHeadDim + d] = 0;
    } else {
      p.part_o[((row0 + r) * p.n_split + split) * kHeadDim + d] = 0.f;
      if (d == 0)
        p.part_lse[(row0 + r) * p.n_split + split] = bad ? DECATTN_POISON_LSE : -__builtin_huge_valf();
    }
  }
}

}  // namespace decattn
