// Head norms of queries and keys and the rotation by position, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w      (w absent: y = x)
//   pairs (y_j, y_{j + rot/2}), or (y_2j, y_{2j+1}) interleaved, j < rot / 2:
//   (a, b) -> (a cos - b sin, b cos + a sin), angle = position * inv_freq[j]
//
// Bytes bound the kernel: every vector is read and written once, and the
// arithmetic is a few operations per element.  Sixteen lanes share a vector; a
// lane takes two groups of four coordinates, placed so that the partners of a
// rotation are in one lane (coordinates 4 l .. and rot / 2 + 4 l .. , or eight
// neighbours), and the norm is four shuffles.  Each sixteen lanes keep to one
// token, whose cosines and sines then stay in registers for all its heads, and
// have four vectors in flight.
//
// Angles: position * inv_freq loses its fraction of a turn in 32 bits at far
// positions.  inv_freq / (2 pi) is kept as a 64-bit fixed-point fraction of a
// turn, so the product with the position is exact modulo one turn (an integer
// multiplication that wraps), and what is rounded is an angle within an eighth
// of a turn of a quarter-turn multiple.  The fractions are formed once per
// CTA, cosines and sines once per token and CTA: all heads share them.
#include <cuda_bf16.h>

#include "kernels.h"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeVecs = kRopeThreads / 16;      // vectors side by side in a CTA
constexpr int kRopeTokens = 4;                    // most tokens a CTA takes at a time
constexpr int kRopeUnroll = 4;                    // vectors a lane has in flight

// Four coordinates, as loaded (streamed: nothing is read twice) and as floats.
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  // (the one rounding to the output type)
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    __stcs(reinterpret_cast<uint2*>(p),
           make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
  }
};
template <>
struct Four<float> {
  float4 w;
  __device__ __forceinline__ void load(const float* p) { w = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w; }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  }
};

// cos and sin of turns / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(unsigned long long turns) {
  const unsigned long long shifted = turns + (1ull << 61);      // nearest quarter turn
  const int quarter = static_cast<int>(shifted >> 62);
  const long long rest = static_cast<long long>(shifted & ((1ull << 62) - 1)) - (1ll << 61);
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);       // half turns, |.| <= 1/4
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// What a lane keeps for its token: where its coordinates are, its pairs'
// cosines and sines, whether they turn.
struct LaneTurn {
  int a, b;                  // coordinates a .. a + 3 and b .. b + 3
  float2 cs[4];
  bool turned, interleaved;
};

// The heads first, first + step, .. of one token's tensor (x, out: this token's
// rows; live: whether the token is there).  The loop is the same for every lane.
template <typename T>
__device__ __forceinline__ void turn_heads(const T* x, T* out, int heads, int first, int step, bool live, const T* weight,
                                           float eps, const LaneTurn& l) {
  float wa[4], wb[4];
  if (weight != nullptr) {
    Four<T> w;
    w.load(weight + l.a);
    w.get(wa);
    w.load(weight + l.b);
    w.get(wb);
  }
  for (int h0 = first - first % step; h0 < heads; h0 += step * kRopeUnroll) {
    Four<T> xa[kRopeUnroll], xb[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + first % step + u * step;
      if (live && h < heads) {
        xa[u].load(x + h * kDim + l.a);
        xb[u].load(x + h * kDim + l.b);
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + first % step + u * step;
      float a[4], b[4];
      xa[u].get(a);
      xb[u].get(b);
      if (weight != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        const float r = 1.0f / sqrtf(ss * (1.0f / kDim) + eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] *= r * wa[i];
          b[i] *= r * wb[i];
        }
      }
      if (l.turned) {
        if (l.interleaved) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p = a[2 * i], q = a[2 * i + 1], s = b[2 * i], t = b[2 * i + 1];
            a[2 * i] = p * l.cs[i].x - q * l.cs[i].y;
            a[2 * i + 1] = q * l.cs[i].x + p * l.cs[i].y;
            b[2 * i] = s * l.cs[i + 2].x - t * l.cs[i + 2].y;
            b[2 * i + 1] = t * l.cs[i + 2].x + s * l.cs[i + 2].y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = a[i], q = b[i];
            a[i] = p * l.cs[i].x - q * l.cs[i].y;
            b[i] = q * l.cs[i].x + p * l.cs[i].y;
          }
        }
      }
      if (live && h < heads) {
        Four<T>::store(out + h * kDim + l.a, a);
        Four<T>::store(out + h * kDim + l.b, b);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(NormRopeArgs a) {
  __shared__ unsigned long long freq_s[kDim / 2];
  __shared__ float2 turn_s[kRopeTokens][kDim / 2];
  const int tid = threadIdx.x, l16 = tid & 15, vec = tid >> 4;
  const int half = a.rot_dim / 2, tokens = a.group_tokens;
  if (tid < half) {
    double f = a.inv_freq[tid] * 0.15915494309189533577;        // turns per position
    f -= floor(f);
    freq_s[tid] = __double2ull_rn(f * 0x1p63) << 1;             // (f < 1: 63 bits hold it)
  }
  LaneTurn l;
  l.turned = 8 * l16 < a.rot_dim;
  l.interleaved = a.interleaved;
  l.a = l.turned && !a.interleaved ? 4 * l16 : 8 * l16;
  l.b = l.turned && !a.interleaved ? half + 4 * l16 : 8 * l16 + 4;
  const int t = vec % tokens, first = vec / tokens, step = kRopeVecs / tokens;   // its token, its heads
  const T* const q = static_cast<const T*>(a.q);
  const T* const k = static_cast<const T*>(a.k);
  T* const q_out = static_cast<T*>(a.q_out);
  T* const k_out = static_cast<T*>(a.k_out);
  const int n_groups = a.n_tokens / tokens + (a.n_tokens % tokens != 0);
  for (int group = blockIdx.x; group < n_groups; group += gridDim.x) {
    const int t0 = group * tokens;
    if (half > 0) {
      __syncthreads();                            // freq_s written; the previous tokens' angles read
      for (int i = tid; i < tokens * half; i += kRopeThreads) {
        const int u = i / half, j = i - u * half;
        if (t0 + u < a.n_tokens)
          turn_s[u][j] = cos_sin(freq_s[j] * static_cast<unsigned long long>(static_cast<long long>(a.positions[t0 + u])));
      }
      __syncthreads();
    }
    const bool live = t0 + t < a.n_tokens && (a.positions == nullptr || a.positions[t0 + t] >= 0);
    if (l.turned)
#pragma unroll
      for (int i = 0; i < 4; ++i) l.cs[i] = turn_s[t][4 * l16 + i];
    const long long row = live ? t0 + t : 0;
    turn_heads(q + row * a.q_stride, q_out + row * a.q_out_stride, a.n_q, first, step, live,
               static_cast<const T*>(a.q_weight), a.eps, l);
    turn_heads(k + row * a.k_stride, k_out + row * a.k_out_stride, a.n_kv, first, step, live,
               static_cast<const T*>(a.k_weight), a.eps, l);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& args, bool bf16, int num_sms, cudaStream_t stream) {
  // few tokens: one per CTA, so that a decode step's heads spread over the SMs;
  // otherwise four, whose angles are one per thread
  NormRopeArgs a = args;
  a.group_tokens = a.n_tokens <= 8 * num_sms ? 1 : kRopeTokens;
  const int n_groups = a.n_tokens / a.group_tokens + (a.n_tokens % a.group_tokens != 0);
  const int grid = n_groups < num_sms * 8 ? n_groups : num_sms * 8;   // 8 CTAs of 256 threads fill an SM
  if (bf16) norm_rope_kernel<__nv_bfloat16><<<grid, kRopeThreads, 0, stream>>>(a);
  else norm_rope_kernel<float><<<grid, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
