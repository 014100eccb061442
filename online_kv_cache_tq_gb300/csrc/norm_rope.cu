// Head norms of queries and keys and the rotation by position, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w      (w absent: y = x)
//   pairs (y_j, y_{j + rot/2}), or (y_2j, y_{2j+1}) interleaved, j < rot / 2:
//   (a, b) -> (a cos - b sin, b cos + a sin), angle = position * inv_freq[j]
//
// Bytes bound the kernel: every vector is read and written once, and the
// arithmetic is a few operations per element.  Sixteen lanes share a vector,
// eight coordinates each (one 16-byte load at bf16), so the norm is four
// shuffles and a half-rotation's partner sits rot / 16 lanes away.  A lane
// keeps several vectors in flight.
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
constexpr int kRopeTokens = 4;                    // most tokens whose angles a CTA forms at a time
constexpr int kRopeUnroll = 2;                    // vectors a lane has in flight

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// The one rounding to the output type.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

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

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(NormRopeArgs a) {
  __shared__ unsigned long long freq_s[kDim / 2];
  __shared__ float2 turn_s[kRopeTokens][kDim / 2];
  __shared__ int pos_s[kRopeTokens];
  const int tid = threadIdx.x, l16 = tid & 15;
  const int half = a.rot_dim / 2, heads = a.n_q + a.n_kv;
  if (tid < half) {
    double f = a.inv_freq[tid] * 0.15915494309189533577;        // turns per position
    f -= floor(f);
    freq_s[tid] = __double2ull_rn(f * 0x1p63) << 1;             // (f < 1: 63 bits hold it)
  }
  // coordinates of this lane: c0 .. c0 + 7; rotated pairs' partner lane
  const int c0 = l16 * 8;
  const bool turned = c0 < a.rot_dim;
  const bool upper = !a.interleaved && c0 >= half;
  const int partner = turned && !a.interleaved ? (upper ? l16 - half / 8 : l16 + half / 8) : l16;
  const int j0 = a.interleaved ? c0 / 2 : (upper ? c0 - half : c0);

  const T* const q = static_cast<const T*>(a.q);
  const T* const k = static_cast<const T*>(a.k);
  T* const q_out = static_cast<T*>(a.q_out);
  T* const k_out = static_cast<T*>(a.k_out);
  const int n_groups = a.n_tokens / a.group_tokens + (a.n_tokens % a.group_tokens != 0);
  for (int group = blockIdx.x; group < n_groups; group += gridDim.x) {
    const int t0 = group * a.group_tokens;
    const int nt = min(a.group_tokens, a.n_tokens - t0);
    __syncthreads();                              // freq_s written; the previous group's angles read
    if (tid < kRopeTokens) pos_s[tid] = tid < nt ? (a.positions != nullptr ? a.positions[t0 + tid] : 0) : -1;
    for (int i = tid; i < nt * half; i += kRopeThreads) {
      const int t = i / half, j = i - t * half;
      const int pos = a.positions[t0 + t];
      turn_s[t][j] = cos_sin(freq_s[j] * static_cast<unsigned long long>(static_cast<long long>(pos)));
    }
    __syncthreads();
    const int n_vec = nt * heads;
    for (int base = 0; base < n_vec; base += kRopeVecs * kRopeUnroll) {   // (uniform: whole warps shuffle)
      float x[kRopeUnroll][8];
      int tok[kRopeUnroll];
      T* dst[kRopeUnroll];
      const T* wgt[kRopeUnroll];
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int v = base + u * kRopeVecs + (tid >> 4);
        dst[u] = nullptr;
        tok[u] = 0;
        wgt[u] = nullptr;
        if (v < n_vec) {
          const int t = v / heads, h = v - t * heads;
          tok[u] = t;
          if (pos_s[t] >= 0) {
            const long long row = t0 + t;
            const bool is_q = h < a.n_q;
            const T* src = is_q ? q + row * a.q_stride + h * kDim : k + row * a.k_stride + (h - a.n_q) * kDim;
            dst[u] = is_q ? q_out + row * a.q_out_stride + h * kDim : k_out + row * a.k_out_stride + (h - a.n_q) * kDim;
            wgt[u] = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
            load8(src + c0, x[u]);
          }
        }
        if (dst[u] == nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if (wgt[u] != nullptr) {
          const float r = 1.0f / sqrtf(ss * (1.0f / kDim) + a.eps);
          float w[8];
          load8(wgt[u] + c0, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[u][i] = x[u][i] * r * w[i];
        }
        if (half > 0) {
          const float2* const cs = turn_s[tok[u]] + j0;
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (turned) {
                const float2 w = cs[i];
                const float p = x[u][2 * i], o = x[u][2 * i + 1];
                x[u][2 * i] = p * w.x - o * w.y;
                x[u][2 * i + 1] = o * w.x + p * w.y;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float o = __shfl_sync(0xffffffffu, x[u][i], partner, 16);
              if (turned) {
                const float2 w = cs[i];
                x[u][i] = x[u][i] * w.x + (upper ? o * w.y : -(o * w.y));
              }
            }
          }
        }
        if (dst[u] != nullptr) store8(dst[u] + c0, x[u]);
      }
    }
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
