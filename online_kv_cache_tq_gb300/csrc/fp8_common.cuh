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
// Four floats times `scale` as codes, to nearest even, saturating.
__device__ __forceinline__ uint32_t fp8_four(float a, float b, float c, float d);
__device__ __forceinline__ uint32_t fp8_four_scaled(float a, float b, float c, float d, float scale) {
  const float2 s = make_float2(scale, scale);
  const float2 lo = __fmul2_rn(make_float2(a, b), s), hi = __fmul2_rn(make_float2(c, d), s);
  return fp8_four(lo.x, lo.y, hi.x, hi.y);
}
// Four floats as codes, to nearest even, saturating.
__device__ __forceinline__ uint32_t fp8_four(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
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

// A sequence's rows, checked: n rows from s0 on, its last positions up to ctx.
// n is 0 where something is out of range (recorded by the CTA that `record`s).
__device__ __forceinline__ int3 fp8_sequence(const Fp8Cache& c, int b, bool record) {
  const int s0 = c.query_start[b], s1 = c.query_start[b + 1], ctx = c.context_lens[b];
  const bool ok = s0 >= 0 && s0 <= s1 && s1 <= c.n_tokens && ctx >= s1 - s0 &&
                  ctx <= static_cast<long long>(c.max_blocks) * c.block_size;
  if (!ok && s0 != s1 && record) atomicCAS(c.error, 0, kErrContext);
  return make_int3(s0, ok ? s1 - s0 : 0, ctx);
}

// The runs of a call, numbered sequence by sequence: what a CTA of THREADS
// threads holds to find one.  Every CTA forms the sums over the batch itself: a
// thread has the sequences tid * chunk .. of the batch.
template <int THREADS>
struct Fp8Runs {
  int first[THREADS + 1];         // runs before the thread's sequences
  int3 seq[THREADS];              // the first of them (fp8_sequence)
  int chunk, most;                // most rows of a sequence
  long long tokens;

  static __device__ __forceinline__ int count(const Fp8Cache& c, const int3& s) {
    return s.y == 0 ? 0 : ((s.z - s.y) % c.block_size + s.y - 1) / c.block_size + 1;
  }
  // By the whole CTA.  Where query_start goes down anywhere (rows could overlap),
  // that is recorded and there are no runs.
  __device__ __forceinline__ void find(const Fp8Cache& c, long long (*warp_s)[2]) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, per = (c.batch + THREADS - 1) / THREADS;
    int top = 0;
    bool down = false;
    long long runs = 0, rows = 0;
    if (tid == 0) most = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= c.batch) break;
      const int3 s = fp8_sequence(c, b, blockIdx.x == 0);
      down = down || c.query_start[b + 1] < c.query_start[b];
      if (i == 0) seq[tid] = s;
      runs += count(c, s);
      rows += s.y;
      top = max(top, s.y);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    long long upto = runs;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
      rows += __shfl_xor_sync(0xffffffffu, rows, d);
    }
    if (lane == 31) warp_s[warp][0] = upto, warp_s[warp][1] = rows;
    const bool ok = !__syncthreads_or(down);      // (then rows are at most n_tokens, and a run has one: the sums below are ints)
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += warp_s[w][0];
      all += warp_s[w][1];
    }
    first[tid + 1] = ok ? static_cast<int>(before + upto) : 0;
    if (lane == 0) atomicMax(&most, top);
    if (tid == 0) {
      first[0] = 0;
      chunk = per;
      tokens = all;
    }
    __syncthreads();
  }
  __device__ __forceinline__ int total() const { return first[THREADS]; }
  // Run g (block -1, recorded: its block is not in the cache).  *from: the thread
  // whose sequences hold it, or one before; moved on to it (callers go upwards).
  __device__ __forceinline__ Fp8Run get(const Fp8Cache& c, int g, int* from) const {
    int lo = *from;                               // the last thread with no more runs than g before it
    if (first[lo + 1] <= g) {
      int hi = THREADS - 1;
      ++lo;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= g) lo = mid;
        else hi = mid - 1;
      }
      *from = lo;
    }
    int b = lo * chunk, at = g - first[lo];
    int3 s = seq[lo];
    if (chunk > 1) {
      for (int n = count(c, s); at >= n; n = count(c, s)) {
        at -= n;
        s = fp8_sequence(c, ++b, false);
      }
    }
    const int past = s.z - s.y, col = past / c.block_size + at, off = at == 0 ? past - col * c.block_size : 0;
    const int pos = col * c.block_size + off;
    const long long entry = static_cast<long long>(b) * c.max_blocks + col;
    long long id = c.block_table ? c.block_table[entry] : entry;
    if (id < 0 || id >= c.num_blocks) {
      atomicCAS(c.error, 0, kErrBlock);
      id = -1;
    }
    return Fp8Run{s.x + pos - past, static_cast<int>(id), off, min(c.block_size - off, s.z - pos)};
  }
};

// What fp8_find_runs shares in a CTA.
constexpr int kFp8Held = 128;     // sequences whose starts and lengths it holds
struct Fp8Finder {
  Fp8Run runs[kFp8Window];
  int count[3];                   // sequences that start up to the window's first and last token; runs
  int start[kFp8Held + 1], ctx[kFp8Held];
};

// The parts of runs that lie among tokens w0 .. w0 + window - 1 of the call, into
// `f.runs` (at most a run per token), in no order; returns how many.  Called by
// the whole CTA; a sequence whose rows or length are out of range, and a block
// id outside the cache, are recorded and left out.  Where query_start goes down
// anywhere, that is recorded and there are no runs.
//
// The sequences of the window's first and last token come from counts over
// query_start; a token's own sequence is then searched between those two.  A
// small batch is held in shared memory, so that the block table's read is the
// second and last that waits for another.
__device__ __forceinline__ int fp8_find_runs(const Fp8Cache& c, int w0, int window, Fp8Finder& f) {
  const int tid = threadIdx.x;
  const bool held = c.batch <= kFp8Held;
  if (tid < 3) f.count[tid] = 0;
  __syncthreads();
  int before = 0, upto = 0;
  bool down = false;
  for (int b = tid; b < c.batch; b += blockDim.x) {
    const int s = c.query_start[b];
    down |= c.query_start[b + 1] < s;
    before += s <= w0;
    upto += s <= w0 + window - 1;
    if (held) f.start[b] = s, f.ctx[b] = c.context_lens[b];
  }
  if (held && tid == 0) f.start[c.batch] = c.query_start[c.batch];
  before = __reduce_add_sync(0xffffffffu, before);
  upto = __reduce_add_sync(0xffffffffu, upto);
  if ((tid & 31) == 0) {
    atomicAdd(&f.count[0], before);
    atomicAdd(&f.count[1], upto);
  }
  if (__syncthreads_or(down)) {
    if (tid == 0) atomicCAS(c.error, 0, kErrContext);
    return 0;
  }
  const int t = w0 + tid;
  if (tid < window && t < c.n_tokens) {
    const int* const start = held ? f.start : c.query_start;
    int lo = max(0, f.count[0] - 1), hi = max(lo, f.count[1] - 1);   // the last sequence that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int s0 = start[lo], s1 = start[lo + 1];
    if (s0 <= t && t < s1) {                      // (else a row that belongs to no sequence)
      const int ctx = held ? f.ctx[lo] : c.context_lens[lo], n = s1 - s0;
      if (s0 < 0 || s1 > c.n_tokens || ctx < n || ctx > static_cast<long long>(c.max_blocks) * c.block_size) {
        atomicCAS(c.error, 0, kErrContext);
      } else {
        const int pos = ctx - n + t - s0, col = pos / c.block_size, off = pos - col * c.block_size;
        if (t == s0 || off == 0 || tid == 0) {
          const long long id = c.block_table ? c.block_table[static_cast<long long>(lo) * c.max_blocks + col]
                                             : static_cast<long long>(lo) * c.max_blocks + col;
          if (id < 0 || id >= c.num_blocks) {
            atomicCAS(c.error, 0, kErrBlock);
          } else {
            const int i = atomicAdd(&f.count[2], 1);
            f.runs[i] = Fp8Run{t, static_cast<int>(id), off, min(c.block_size - off, min(s1, w0 + window) - t)};
          }
        }
      }
    }
  }
  __syncthreads();
  return f.count[2];
}

// 4 x 4 words over four lanes APART apart (i = lane / APART % 4): lane i's word j
// goes to lane j's word i.
template <int APART>
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const int lane = threadIdx.x / APART;
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & s) continue;
      // words j and j + s: a lane without bit s gives the latter, one with it the former
      const bool up = lane & s;
      const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? w[j] : w[j + s], s * APART);
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
