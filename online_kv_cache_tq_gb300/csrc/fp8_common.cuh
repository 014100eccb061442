// Device code shared by the kernels of the 8-bit cache: e4m3 conversions, and
// the runs of a call's tokens that lie in one cache block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernels.h"

namespace tq {
namespace {

// Two e4m3 codes of a register's low half as floats, and back (saturating).
__device__ __forceinline__ __half2 fp8_halves(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3));
}
__device__ __forceinline__ float2 fp8_floats(uint32_t two) { return __half22float2(fp8_halves(two)); }
__device__ __forceinline__ uint32_t fp8_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t fp8_four(float a, float b, float c, float d) {
  return fp8_pair(a, b) | fp8_pair(c, d) << 16;
}
constexpr uint32_t kFp8NaN4 = 0x7f7f7f7fu;

// 2^e of a scale, and its exponent (scales are powers of two).
__device__ __forceinline__ float fp8_power(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ int fp8_exponent(float scale) {
  const int e = static_cast<int>((__float_as_uint(scale) >> 23) & 255u) - 127;
  return min(kFp8MaxExp, max(kFp8MinExp, e));
}
// The least e (within the scales' range) with 448 2^e >= amax: 448 = 1.75 * 2^8.
__device__ __forceinline__ int fp8_scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax > 0.f ? min(kFp8MaxExp, max(kFp8MinExp, e)) : kFp8MinExp;
}
// Four codes times 2^-k, rounded once more: 2^-k and the products are exact in
// fp16 as far down as e4m3 tells values from zero.
__device__ __forceinline__ uint32_t fp8_rescale(uint32_t four, __half2 factor) {
  const __half2 lo = __hmul2(fp8_halves(four), factor), hi = __hmul2(fp8_halves(four >> 16), factor);
  return __nv_cvt_halfraw2_to_fp8x2(__half2_raw(lo), __NV_SATFINITE, __NV_E4M3) |
         static_cast<uint32_t>(__nv_cvt_halfraw2_to_fp8x2(__half2_raw(hi), __NV_SATFINITE, __NV_E4M3)) << 16;
}

// A run: tokens `row` .. `row + len - 1` of the call, at offsets off, off + 1,
// .. of one cache block.
struct Fp8Run {
  int row, block, off, len;
};
constexpr int kFp8Window = 64;    // most tokens of a CTA's window

// The runs that begin among tokens w0 .. w0 + window - 1 of the call, into
// `runs` (at most a run per token), in no order; returns how many.  Called by
// the whole CTA; a sequence whose rows or length are out of range, and a block
// id outside the cache, are recorded and left out.
//
// The sequences of the window's first and last token come from counts over
// query_start, one round of loads for as many sequences as the CTA has
// threads; a token's own sequence is then searched between those two.
__device__ __forceinline__ int fp8_find_runs(const Fp8Cache& c, int w0, int window, Fp8Run* runs, int* scratch) {
  const int tid = threadIdx.x;
  if (tid < 3) scratch[tid] = 0;
  __syncthreads();
  int before = 0, upto = 0;
  for (int b = tid; b < c.batch; b += blockDim.x) {
    const int s = c.query_start[b];
    before += s <= w0;
    upto += s <= w0 + window - 1;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  upto = __reduce_add_sync(0xffffffffu, upto);
  if ((tid & 31) == 0) {
    atomicAdd(&scratch[0], before);
    atomicAdd(&scratch[1], upto);
  }
  __syncthreads();
  const int t = w0 + tid;
  if (tid < window && t < c.n_tokens) {
    int lo = max(0, scratch[0] - 1), hi = max(lo, scratch[1] - 1);   // the last sequence that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (c.query_start[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int s0 = c.query_start[lo], s1 = c.query_start[lo + 1];
    if (s0 <= t && t < s1) {                      // (else a row that belongs to no sequence)
      const int ctx = c.context_lens[lo], n = s1 - s0;
      if (s0 < 0 || s1 > c.n_tokens || ctx < n || ctx > static_cast<long long>(c.max_blocks) * c.block_size) {
        atomicCAS(c.error, 0, kErrContext);
      } else {
        const int pos = ctx - n + t - s0, col = pos / c.block_size, off = pos - col * c.block_size;
        if (t == s0 || off == 0) {
          const long long id = c.block_table ? c.block_table[static_cast<long long>(lo) * c.max_blocks + col]
                                             : static_cast<long long>(lo) * c.max_blocks + col;
          if (id < 0 || id >= c.num_blocks) {
            atomicCAS(c.error, 0, kErrBlock);
          } else {
            const int i = atomicAdd(&scratch[2], 1);
            runs[i] = Fp8Run{t, static_cast<int>(id), off, min(c.block_size - off, s1 - t)};
          }
        }
      }
    }
  }
  __syncthreads();
  return scratch[2];
}

// 4 x 4 words over four neighbouring lanes (lane & 3): lane i's word j goes to
// lane j's word i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const int lane = threadIdx.x & 3;
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & s) continue;
      // words j and j + s: a lane without bit s gives the latter, one with it the former
      const bool up = lane & s;
      const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? w[j] : w[j + s], s);
      if (up) w[j] = other;
      else w[j + s] = other;
    }
  }
}
// 4 x 4 bytes of four words: byte j of word i goes to byte i of word j.
__device__ __forceinline__ void transpose_bytes(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  out[0] = __byte_perm(a, b, 0x5410);
  out[1] = __byte_perm(a, b, 0x7632);
  out[2] = __byte_perm(c, d, 0x5410);
  out[3] = __byte_perm(c, d, 0x7632);
}

}  // namespace
}  // namespace tq
