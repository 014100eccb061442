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
// neighbours), and the norm is four shuffles.  Sixteen lanes take a run of one
// token's heads: each lane forms the four cosines and sines of its pairs once
// and keeps them in registers, and there is no barrier between runs.  A lane
// has 64 bytes in flight.  32768 tokens x 72 heads, bf16: 207 us, 5.8 TB/s, 0.86 of
// a plain copy (a partner eight lanes away and barriers between tokens: 430 us;
// partners in one lane: 315 us).
//
// Angles: position * inv_freq loses its fraction of a turn in 32 bits at far
// positions.  inv_freq / (2 pi) is kept as a 64-bit fixed-point fraction of a
// turn, so the product with the position is exact modulo one turn (an integer
// multiplication that wraps), and what is rounded is an angle within an eighth
// of a turn of a quarter-turn multiple.
#include <cuda_bf16.h>

#include "kernels.h"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeVecs = kRopeThreads / 16;      // runs side by side in a CTA
template <typename T>
constexpr int kRopeUnroll = sizeof(T) == 2 ? 4 : 2;   // vectors a lane has in flight

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

// cos and sin of position * freq / 2^64 turns.  The top 32 bits of the product
// (modulo a turn) are a quarter turn's number and an angle within an eighth
// of a turn of it, for which the Taylor series to the 9th and 10th power
// leave less than 2e-9.
__device__ __forceinline__ float2 cos_sin(unsigned long long freq, unsigned pos) {
  const unsigned turn = static_cast<unsigned>(freq >> 32) * pos + __umulhi(static_cast<unsigned>(freq), pos);
  const unsigned shifted = turn + (1u << 29);                   // nearest quarter turn
  const int rest = static_cast<int>(shifted & 0x3fffffffu) - (1 << 29);
  const float x = static_cast<float>(rest) * 1.46291807926715968e-9f;   // 2 pi / 2^32
  const float z = x * x;
  const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float cc = shifted & (1u << 30) ? -s : c, ss = shifted & (1u << 30) ? c : s;
  return shifted & (1u << 31) ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

// The rotation of a lane's four pairs.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&a)[4], float (&b)[4], const float2 (&cs)[4]) {
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float p = a[2 * i], q = a[2 * i + 1], s = b[2 * i], t = b[2 * i + 1];
      a[2 * i] = p * cs[i].x - q * cs[i].y;
      a[2 * i + 1] = q * cs[i].x + p * cs[i].y;
      b[2 * i] = s * cs[i + 2].x - t * cs[i + 2].y;
      b[2 * i + 1] = t * cs[i + 2].x + s * cs[i + 2].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = a[i], q = b[i];
      a[i] = p * cs[i].x - q * cs[i].y;
      b[i] = q * cs[i].x + p * cs[i].y;
    }
  }
}

// A vector whose squares leave fp32's range (rare): read again and scaled by
// the power of two that brings its largest coordinate near 1 (2^100 at most, so
// that the scaled eps stays a number).
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void far_vector(const T* x, T* out, const float (&wa)[4], const float (&wb)[4], float eps,
                                           int ca, int cb, bool turned, const float2 (&cs)[4]) {
  const unsigned lanes = 0xffffu << (threadIdx.x & 16);
  Four<T> w;
  float a[4], b[4], top = 0.f, ss = 0.f;
  w.load(x + ca);
  w.get(a);
  w.load(x + cb);
  w.get(b);
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, d));
  const int e = max(-100, min(126, static_cast<int>(__float_as_uint(top) >> 23) - 127));
  const float down = __uint_as_float(static_cast<unsigned>(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] *= down;
    b[i] *= down;
    ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) ss += __shfl_xor_sync(lanes, ss, d);
  const float r = 1.0f / sqrtf(ss * (1.0f / kDim) + eps * down * down);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] *= r * wa[i];
    b[i] *= r * wb[i];
  }
  if (turned) turn<INTERLEAVED>(a, b, cs);
  Four<T>::store(out + ca, a);
  Four<T>::store(out + cb, b);
}

// Heads h0 .. h1 - 1 of one tensor of a token (x, out: its rows), coordinates
// ca .. ca + 3 and cb .. cb + 3 of each; cs: the lane's four pairs.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void turn_heads(const T* x, T* out, int h0, int h1, const T* weight, float eps, int ca, int cb,
                                           bool turned, const float2 (&cs)[4]) {
  if (h0 >= h1) return;
  float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
  if (weight != nullptr) {
    Four<T> w;
    w.load(weight + ca);
    w.get(wa);
    w.load(weight + cb);
    w.get(wb);
  }
  const unsigned lanes = 0xffffu << (threadIdx.x & 16);
  for (int h = h0; h < h1; h += kRopeUnroll<T>) {
    Four<T> xa[kRopeUnroll<T>], xb[kRopeUnroll<T>];
#pragma unroll
    for (int u = 0; u < kRopeUnroll<T>; ++u) {
      const T* const p = x + min(h + u, h1 - 1) * kDim;   // (the last one again where there are no more)
      xa[u].load(p + ca);
      xb[u].load(p + cb);
    }
    unsigned far = 0;                             // vectors that `far_vector` does
#pragma unroll
    for (int u = 0; u < kRopeUnroll<T>; ++u) {
      float a[4], b[4];
      xa[u].get(a);
      xb[u].get(b);
      if (weight != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) ss += __shfl_xor_sync(lanes, ss, d);
        // (all sixteen lanes; beside an eps of 2^-118 and more, squares that vanish do not count)
        if (!(ss < 0x1p120f) || (ss < 0x1p-100f && eps < 0x1p-118f)) far |= 1u << u;
        const float r = 1.0f / sqrtf(ss * (1.0f / kDim) + eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] *= r * wa[i];
          b[i] *= r * wb[i];
        }
      }
      if (turned) turn<INTERLEAVED>(a, b, cs);
      if (h + u < h1 && !(far >> u & 1u)) {
        T* const p = out + (h + u) * kDim;
        Four<T>::store(p + ca, a);
        Four<T>::store(p + cb, b);
      }
    }
#pragma unroll 1
    for (int u = 0; far != 0; ++u, far >>= 1) {
      if ((far & 1u) && h + u < h1)
        far_vector<T, INTERLEAVED>(x + (h + u) * kDim, out + (h + u) * kDim, wa, wb, eps, ca, cb, turned, cs);
    }
  }
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 4) norm_rope_kernel(NormRopeArgs a) {
  __shared__ unsigned long long freq_s[kDim / 2];
  const int tid = threadIdx.x, l16 = tid & 15;
  const int half = a.rot_dim / 2;
  if (tid < half) {
    double f = a.inv_freq[tid] * 0.15915494309189533577;        // turns per position
    f -= floor(f);
    freq_s[tid] = __double2ull_rn(f * 0x1p63) << 1;             // (f < 1: 63 bits hold it)
  }
  __syncthreads();
  const bool turned = 8 * l16 < a.rot_dim;
  const int ca = turned && !INTERLEAVED ? 4 * l16 : 8 * l16;
  const int cb = turned && !INTERLEAVED ? half + 4 * l16 : 8 * l16 + 4;
  const int heads = a.n_q + a.n_kv;
  // The halves of a warp take the same heads of neighbouring tokens, so that
  // they stay together.
  const int warps = kRopeThreads / 32;
  const long long n_runs = (static_cast<long long>(a.n_tokens) + 1) / 2 * a.token_runs;
  for (long long run = static_cast<long long>(blockIdx.x) * warps + (tid >> 5); run < n_runs;
       run += static_cast<long long>(gridDim.x) * warps) {
    const long long token_pair = run / a.token_runs, token = 2 * token_pair + ((tid >> 4) & 1);
    const int h0 = static_cast<int>(run - token_pair * a.token_runs) * a.run_heads, h1 = min(h0 + a.run_heads, heads);
    if (token >= a.n_tokens) continue;            // (all sixteen lanes, here and below)
    float2 cs[4] = {};
    if (a.positions != nullptr) {
      const int pos = a.positions[token];
      if (pos < 0) continue;
      if (turned)
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = cos_sin(freq_s[4 * l16 + i], static_cast<unsigned>(pos));
    }
    turn_heads<T, INTERLEAVED>(static_cast<const T*>(a.q) + token * a.q_stride,
                               static_cast<T*>(a.q_out) + token * a.q_out_stride, h0, min(h1, a.n_q),
                               static_cast<const T*>(a.q_weight), a.eps, ca, cb, turned, cs);
    turn_heads<T, INTERLEAVED>(static_cast<const T*>(a.k) + token * a.k_stride,
                               static_cast<T*>(a.k_out) + token * a.k_out_stride, max(h0 - a.n_q, 0), h1 - a.n_q,
                               static_cast<const T*>(a.k_weight), a.eps, ca, cb, turned, cs);
  }
}

template <typename T>
void launch_type(const NormRopeArgs& a, int grid, cudaStream_t stream) {
  if (a.interleaved) norm_rope_kernel<T, true><<<grid, kRopeThreads, 0, stream>>>(a);
  else norm_rope_kernel<T, false><<<grid, kRopeThreads, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& args, bool bf16, int num_sms, cudaStream_t stream) {
  // A token's heads are cut into runs so that the last round of runs over the
  // GPU's sixteen-lane slots weighs little: six rounds where runs of eight
  // heads allow it (32768 tokens of 72 heads: runs of 36 take 212 us, of 72
  // 220 us, of 8 227 us; 5001 tokens of 40 fp32 heads: runs of 8 take 44 us, of
  // 40 47 us); fewer heads than eight only where that leaves slots empty, down
  // to what a lane has in flight (a decode step).
  NormRopeArgs a = args;
  const int heads = a.n_q + a.n_kv;
  const long long slots = 4ll * num_sms * kRopeVecs;
  const int least = bf16 ? kRopeUnroll<__nv_bfloat16> : kRopeUnroll<float>;
  const long long eights = (heads + 7) / 8, most = (heads + least - 1) / least;
  long long runs = (6 * slots + a.n_tokens - 1) / a.n_tokens;
  if (runs > eights) runs = a.n_tokens * eights >= slots ? eights : most;
  a.run_heads = static_cast<int>((heads + runs - 1) / runs + least - 1) / least * least;
  a.token_runs = (heads + a.run_heads - 1) / a.run_heads;
  const int warps = kRopeThreads / 32;
  const long long ctas = ((static_cast<long long>(a.n_tokens) + 1) / 2 * a.token_runs + warps - 1) / warps;
  const int grid = static_cast<int>(ctas < 4ll * num_sms ? ctas : 4ll * num_sms);
  if (bf16) launch_type<__nv_bfloat16>(a, grid, stream);
  else launch_type<float>(a, grid, stream);
  return cudaGetLastError();
}

}  // namespace tq
