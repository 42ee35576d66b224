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
// once.  One CTA takes one token: 64 threads make the token's sines and
// cosines, shared by all heads through shared memory; a head's 128 values
// are eight threads' work, two 16-byte pieces each, so that a thread holds
// both halves of its eight pairs.
#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                       // threads per head
constexpr int kHeads = kThreads / kLanes;       // heads per pass of a CTA

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
template <bool kBF16, bool kF8, bool kNext>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[64];
  const int64_t t = blockIdx.x;
  const int pairs = p.rope.rot_dim >> 1;
  if (threadIdx.x < pairs) {
    const int i = threadIdx.x;
    const int pos = p.positions[p.rope.axis[i] * static_cast<int64_t>(p.tokens) + t];
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.rope.turns[i];
    const int half_turns = static_cast<int>(static_cast<uint32_t>((phase + 0x80000000ull) >> 32));
    float s, c;
    sincospif(static_cast<float>(half_turns) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cs[i] = make_float2(c, s);
  }
  const int slot = p.slots[t];
  const bool in_cache = slot >= 0 && slot < p.num_slots;
  if (threadIdx.x == 0 && slot >= p.num_slots) flag_error(p.err_flag, kFlagBadBlock);
  __syncthreads();

  const int u = threadIdx.x % kLanes;
  const bool turned = 8 * u < pairs;  // this thread's eight pairs (8 u .. 8 u + 7) are rotated
  // The thread's two 8-element pieces of a head: neighbours, or half the
  // rotated width apart; past the rotated part, neighbours again.
  const int e0 = kNext ? 16 * u : turned ? 8 * u : 16 * u;
  const int e1 = kNext ? e0 + 8 : turned ? e0 + pairs : e0 + 8;
  float c[8], s[8];
  if (turned) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = cs[8 * u + k];
      c[k] = f.x;
      s[k] = f.y;
    }
  }
  const int n_heads = p.h_q + (in_cache ? 2 * p.h_kv : 0);
#pragma unroll 2
  for (int h = threadIdx.x / kLanes; h < n_heads; h += kHeads) {
    const bool is_q = h < p.h_q, is_v = h >= p.h_q + p.h_kv;
    const int hh = is_q ? h : is_v ? h - p.h_q - p.h_kv : h - p.h_q;
    const uint16_t* src = static_cast<const uint16_t*>(is_q ? p.q : is_v ? p.v : p.k) +
                          t * (is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride) +
                          hh * kHeadDim;
    const uint4 w0 = *reinterpret_cast<const uint4*>(src + e0);
    const uint4 w1 = *reinterpret_cast<const uint4*>(src + e1);
    float a[8], b[8];
    unpack8<kBF16>(w0, a);
    unpack8<kBF16>(w1, b);
    if (turned && !is_v) {
      if constexpr (kNext) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = a[2 * k], y = a[2 * k + 1];
          a[2 * k] = x * c[k] - y * s[k];
          a[2 * k + 1] = x * s[k] + y * c[k];
          const float z = b[2 * k], w = b[2 * k + 1];
          b[2 * k] = z * c[4 + k] - w * s[4 + k];
          b[2 * k + 1] = z * s[4 + k] + w * c[4 + k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float x = a[k], y = b[k];
          a[k] = x * c[k] - y * s[k];
          b[k] = x * s[k] + y * c[k];
        }
      }
    }
    if (is_q) {
      uint16_t* dst = static_cast<uint16_t*>(p.q_out) +
                      (t * p.h_q + hh) * static_cast<int64_t>(kHeadDim);
      *reinterpret_cast<uint4*>(dst + e0) = pack8<kBF16>(a);
      *reinterpret_cast<uint4*>(dst + e1) = pack8<kBF16>(b);
    } else {
      const int64_t row = (static_cast<int64_t>(slot) * p.h_kv + hh) * kHeadDim;
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
  }
}

template <bool kBF16, bool kF8>
void launch_t(const RopeParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.tokens));
  if (p.rope.interleaved)
    rope_append_kernel<kBF16, kF8, true><<<grid, kThreads, 0, stream>>>(p);
  else
    rope_append_kernel<kBF16, kF8, false><<<grid, kThreads, 0, stream>>>(p);
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
