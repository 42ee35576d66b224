// rope_append.cu -- rotary positions with one or several axes on a step's
// queries and keys, and the write of its keys and values into the paged cache.
//
// Pair i of a head, (x, y) = (h[i], h[i + r/2]) or (h[2i], h[2i + 1]) of the
// first r dimensions, is turned by the angle  pos[axis(i), t] * f_i:
//   x' = x cos - y sin,   y' = x sin + y cos
// (time, height and width positions of images and video: each pair follows
// one axis).  The angle is reduced exactly: f_i is stored in turns as a
// 64-bit fraction F_i = f_i / (2 pi) * 2^64, and pos * F_i modulo 2^64 is the
// phase of a position however far (the multiplication drops whole turns);
// its top 32 bits, rounded, go to sincospif, so the angle is off by at most
// 2^-25 of a half turn.  Products are in fp32, each result rounded once.
//
// Bound by HBM: q, k and v are read once, q_out and the cache rows written
// once.  A CTA takes one token (few tokens: latency) up to four: its
// threads make the tokens' sines and cosines, which the heads share through
// shared memory; a head's 128 values are eight threads' work, two 16-byte
// pieces each, so that a thread holds both halves of its eight pairs, and the
// next head's pieces are on their way while one is turned.
#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                       // threads per head
constexpr int kHeads = kThreads / kLanes;       // heads at a time

template <bool kBF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2<kBF16>(in[k]);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}

template <bool kBF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<kBF16>(x[0], x[1]), pack2<kBF16>(x[2], x[3]), pack2<kBF16>(x[4], x[5]),
                    pack2<kBF16>(x[6], x[7]));
}

// fp32(x) / s as e4m3 codes, as the single-token cache write quantises.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float s) {
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * k], s), __fdiv_rn(x[2 * k + 1], s));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// kNext: pairs of neighbours (2i, 2i + 1); else pairs half the rotated width apart.
template <bool kBF16, bool kF8, bool kNext, int kTok>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float4 cs[kTok][32];  // (cos, sin) of pairs 2 i and 2 i + 1
  __shared__ int slots[kTok];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTok;
  const int n_tok = min(kTok, static_cast<int>(p.tokens - t0));
  const int pairs = p.rope.rot_dim >> 1;
  const int u = threadIdx.x % kLanes;
  const bool turned = 8 * u < pairs;  // this thread's eight pairs (8 u .. 8 u + 7) are rotated
  // The thread's two 8-element pieces of a head: neighbours, or half the
  // rotated width apart; past the rotated part, neighbours again.
  const int e0 = kNext ? 16 * u : turned ? 8 * u : 16 * u;
  const int e1 = kNext ? e0 + 8 : turned ? e0 + pairs : e0 + 8;
  const int heads = p.h_q + 2 * p.h_kv;

  auto source = [&](int tl, int h) -> const uint16_t* {
    const int64_t t = t0 + tl;
    if (h < p.h_q) return static_cast<const uint16_t*>(p.q) + t * p.q_stride + h * kHeadDim;
    h -= p.h_q;
    if (h < p.h_kv) return static_cast<const uint16_t*>(p.k) + t * p.k_stride + h * kHeadDim;
    return static_cast<const uint16_t*>(p.v) + t * p.v_stride + (h - p.h_kv) * kHeadDim;
  };
  // Units of work: the heads (q, k, v) of the CTA's tokens, one after another.
  int tl = 0, h = threadIdx.x / kLanes;
  auto wrap = [&](int& at, int& head) {
    while (head >= heads) {
      head -= heads;
      ++at;
    }
  };
  wrap(tl, h);
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (tl < n_tok) {
    const uint16_t* src = source(tl, h);
    w0 = *reinterpret_cast<const uint4*>(src + e0);
    w1 = *reinterpret_cast<const uint4*>(src + e1);
  }
  for (int i = threadIdx.x; i < kTok * 64; i += kThreads) {
    const int at = i >> 6, pair = i & 63;
    if (at < n_tok && pair < pairs) {
      const int pos = p.positions[p.rope.axis[pair] * static_cast<int64_t>(p.tokens) + t0 + at];
      const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.rope.turns[pair];
      const int half_turns = static_cast<int>(static_cast<uint32_t>((phase + 0x80000000ull) >> 32));
      float sn, cn;
      sincospif(static_cast<float>(half_turns) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31
      reinterpret_cast<float2*>(&cs[at][0])[pair] = make_float2(cn, sn);
    }
  }
  if (threadIdx.x < n_tok) {
    const int slot = p.slots[t0 + threadIdx.x];
    if (slot >= p.num_slots) flag_error(p.err_flag, kFlagBadBlock);
    slots[threadIdx.x] = slot < p.num_slots ? slot : -1;
  }
  __syncthreads();

  // With one or two tokens a CTA a thread keeps its pairs' sines and cosines from
  // head to head (64 tokens 3.2 -> 2.95 us, 1111 into an 8-bit cache 6.9 -> 6.5);
  // with four it has them for two or three heads only, and the registers cost
  // more CTAs than the reads (8192 tokens 55.1 -> 57.7).
  constexpr bool kHold = kTok <= 2;
  float4 held[4] = {};
  int held_of = -1;
#pragma unroll 1
  while (tl < n_tok) {
    if (kHold && turned && tl != held_of) {
#pragma unroll
      for (int j = 0; j < 4; ++j) held[j] = cs[tl][4 * u + j];
      held_of = tl;
    }
    int tn = tl, hn = h + kHeads;
    wrap(tn, hn);
    uint4 n0 = make_uint4(0, 0, 0, 0), n1 = n0;
    if (tn < n_tok) {
      const uint16_t* src = source(tn, hn);
      n0 = *reinterpret_cast<const uint4*>(src + e0);
      n1 = *reinterpret_cast<const uint4*>(src + e1);
    }
    const bool is_q = h < p.h_q, is_v = h >= p.h_q + p.h_kv;
    float a[8], b[8];
    unpack8<kBF16>(w0, a);
    unpack8<kBF16>(w1, b);
    if (turned && !is_v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 f = kHold ? held[j] : cs[tl][4 * u + j];  // pairs 8 u + 2 j and the next
        // Their places: neighbours in one piece, or place 2 j (2 j + 1) of both.
        float& x0 = kNext ? (j < 2 ? a : b)[4 * (j & 1)] : a[2 * j];
        float& y0 = kNext ? (j < 2 ? a : b)[4 * (j & 1) + 1] : b[2 * j];
        float& x1 = kNext ? (j < 2 ? a : b)[4 * (j & 1) + 2] : a[2 * j + 1];
        float& y1 = kNext ? (j < 2 ? a : b)[4 * (j & 1) + 3] : b[2 * j + 1];
        const float p0 = x0 * f.x - y0 * f.y, q0 = x0 * f.y + y0 * f.x;
        const float p1 = x1 * f.z - y1 * f.w, q1 = x1 * f.w + y1 * f.z;
        x0 = p0;
        y0 = q0;
        x1 = p1;
        y1 = q1;
      }
    }
    if (is_q) {
      uint16_t* dst = static_cast<uint16_t*>(p.q_out) +
                      ((t0 + tl) * p.h_q + h) * static_cast<int64_t>(kHeadDim);
      *reinterpret_cast<uint4*>(dst + e0) = pack8<kBF16>(a);
      *reinterpret_cast<uint4*>(dst + e1) = pack8<kBF16>(b);
    } else if (slots[tl] >= 0) {
      const int hh = is_v ? h - p.h_q - p.h_kv : h - p.h_q;
      const int64_t row = (static_cast<int64_t>(slots[tl]) * p.h_kv + hh) * kHeadDim;
      if constexpr (kF8) {
        const float sc = (is_v ? p.v_scale : p.k_scale)[hh];
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + row;
        *reinterpret_cast<uint2*>(dst + e0) = quant8(a, sc);
        *reinterpret_cast<uint2*>(dst + e1) = quant8(b, sc);
      } else {
        uint16_t* dst = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + row;
        *reinterpret_cast<uint4*>(dst + e0) = pack8<kBF16>(a);
        *reinterpret_cast<uint4*>(dst + e1) = pack8<kBF16>(b);
      }
    }
    tl = tn;
    h = hn;
    w0 = n0;
    w1 = n1;
  }
}

template <bool kBF16, bool kF8, bool kNext>
void launch_n(const RopeParams& p, cudaStream_t stream) {
  // A CTA's tokens: as few as put all CTAs on the GPU at once (four per SM
  // of 152), at most four.  64 + 8 + 8 heads in bf16, by 1 / 2 / 4 tokens a
  // CTA (before `held`): 300 tokens 3.9 / 4.2 / 6.1 us, 1111 12.4 / 10.4 / 12.3,
  // 2048 18.6 / 18.1 / 17.5, 8192 60.7 / 54.9 / 55.4 (6.1 TB/s); 8 tokens 62.7.
  constexpr int kSlots = 4 * 152;
  auto go = [&](auto kern, int tok) {
    kern<<<static_cast<unsigned>((p.tokens + tok - 1) / tok), kThreads, 0, stream>>>(p);
  };
  if (p.tokens <= kSlots)
    go(rope_append_kernel<kBF16, kF8, kNext, 1>, 1);
  else if (p.tokens <= 2 * kSlots)
    go(rope_append_kernel<kBF16, kF8, kNext, 2>, 2);
  else
    go(rope_append_kernel<kBF16, kF8, kNext, 4>, 4);
}

template <bool kBF16, bool kF8>
void launch_t(const RopeParams& p, cudaStream_t stream) {
  p.rope.interleaved ? launch_n<kBF16, kF8, true>(p, stream)
                     : launch_n<kBF16, kF8, false>(p, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool e4m3, bool bf16, cudaStream_t stream) {
  if (e4m3)
    bf16 ? launch_t<true, true>(p, stream) : launch_t<false, true>(p, stream);
  else
    bf16 ? launch_t<true, false>(p, stream) : launch_t<false, false>(p, stream);
  return cudaGetLastError();
}

}  // namespace decattn
