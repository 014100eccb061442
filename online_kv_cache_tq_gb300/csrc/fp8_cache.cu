// Writing the 8-bit cache and reading it back.
//
// Append.  For every (block, KV head) that the call's tokens touch, keys and
// values apart, a = max |x| over the new tokens, and the scale is the least
// 2^e, -40 <= e <= 14, with 448 2^e >= a, or the block's old one if that is
// larger and the block already holds earlier tokens (the run does not begin at
// its first offset).  The codes are rn_e4m3(x 2^-e); where the scale grew, the
// earlier tokens' codes become rn_e4m3(code 2^(e_old - e)).  A power of two
// loses nothing but codes that leave e4m3's normal range.
// The bound is HBM, 2 x 128 x (element + 1) bytes a token and KV head, and the
// latency of a chain (run, table entry, rows, largest, codes) that a stage ahead
// hides: a prompt of 32768 tokens x 8 heads takes 39.1 us in bf16 (5.1 TB/s, 0.77
// of the measured copy; 730 warp instructions for a warp's 16 tokens x 128, 57 %
// of issue), a decode step of 64 sequences 4 us.  Rows kept in registers between
// the two passes took 45 us, read twice from memory 55, staged by bulk copies of
// a row each 55.  A mixed step of 24 sequences x 4 heads, float32, blocks of 96
// tokens: 15.6 us; 20.7 where a run longer than a stage came twice, 28 with windows
// of tokens per CTA instead of runs, because a window's runs come one after another.
//
// Read.  x = code 2^e, exact in either type.  The bound is HBM: 131072 tokens x 8
// heads to bf16 122 us (6.6 TB/s, 0.99), 65536 to float32 103 us (0.97).
#include <algorithm>

#include "fp8_common.cuh"
#include "tc_ptx.cuh"

namespace tq {
namespace {

// Tokens that one warp appends alone.  (Runs of one length, 8 heads, blocks of 64,
// us by a warp | by a CTA: 64 of 2 bf16 5.0 | 6.6, of 4 7.7 | 6.9, of 8 11.2 | 7.2;
// 256 of 4 17.5 | 18.6, of 8 33.8 | 21.0; float32 256 of 4 16.8 | 23.8, of 8 29.7 | 27.5.)
constexpr int kShortRun = 4;
constexpr int kReadCtasPerSm = 32;

template <bool BF16>
struct Eight {                    // eight neighbouring coordinates of a row as they lie in memory
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    w[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (!BF16) w[1] = *reinterpret_cast<const uint4*>(p + 16);
  }
  __device__ __forceinline__ void floats(float (&v)[8]) const {
    if constexpr (BF16) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[4 * i] = __uint_as_float(w[i].x), v[4 * i + 1] = __uint_as_float(w[i].y);
        v[4 * i + 2] = __uint_as_float(w[i].z), v[4 * i + 3] = __uint_as_float(w[i].w);
      }
    }
  }
};

// Byte of (token, coordinate) in a block's keys and values of a KV head.
__device__ __forceinline__ int key_byte(int token, int coord) {
  return (token >> 3) * 1024 + (coord >> 4) * 128 + (token & 7) * 16 + (coord & 15);
}
__device__ __forceinline__ int value_byte(int token, int coord) {
  return (token >> 4) * 2048 + coord * 16 + (token & 15);
}

// Codes of the tokens before offset `off` times 2^-k, by `threads` threads.
__device__ __forceinline__ void rescale_block(uint8_t* block, bool values, int off, int k, int tid, int threads) {
  const __half2 factor = __float2half2_rn(fp8_power(-k));
  uint4* const p = reinterpret_cast<uint4*>(block);
  const int count = values ? (off + 15) / 16 * 128 : (off + 7) / 8 * 64;
  for (int i = tid; i < count; i += threads) {
    const int mine = values ? min(16, off - (i >> 7) * 16) : (i >> 6) * 8 + (i & 7) < off ? 16 : 0;   // bytes
    if (mine == 0) continue;
    const uint4 old = p[i];
    const uint32_t u[4] = {old.x, old.y, old.z, old.w};
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(4, max(0, mine - 4 * j));
      const uint32_t mask = n == 4 ? 0xffffffffu : (1u << (8 * n)) - 1u;
      w[j] = (fp8_rescale(u[j], factor) & mask) | (u[j] & ~mask);
    }
    p[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The scale of a run whose new tokens have magnitudes up to `amax`; *grown: by
// how many powers of two the earlier tokens' codes have to shrink.
__device__ __forceinline__ int run_exponent(float amax, int off, float old_scale, int* grown) {
  const int e = fp8_scale_exponent(amax);
  *grown = 0;
  if (off == 0) return e;
  const int old = fp8_exponent(old_scale);
  if (e > old) *grown = e - old;
  return max(e, old);
}

// A run of at most kShortRun tokens, by one warp: four coordinates a lane.
template <bool BF16>
__device__ __forceinline__ void append_short(const Fp8Run& r, const void* rows, long long stride, int head,
                                             uint8_t* block, float* scale, bool values) {
  const int lane = threadIdx.x & 31;
  const float old = r.off > 0 ? *scale : 0.f;
  float x[kShortRun][4];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kShortRun; ++i) {
    if (i >= r.len) break;
    const long long at = (static_cast<long long>(r.row) + i) * stride + head * kDim + 4 * lane;
    if constexpr (BF16) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(rows) + at));
      x[i][0] = __uint_as_float(u.x << 16), x[i][1] = __uint_as_float(u.x & 0xffff0000u);
      x[i][2] = __uint_as_float(u.y << 16), x[i][3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
      const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(rows) + at));
      x[i][0] = u.x, x[i][1] = u.y, x[i][2] = u.z, x[i][3] = u.w;
    }
  }
  uint32_t nans = 0;                              // tokens with a NaN, by bit: they do not count
#pragma unroll
  for (int i = 0; i < kShortRun; ++i)
    if (i < r.len) {
      // (a sum of magnitudes is NaN only if one of them is)
      const float all = (fabsf(x[i][0]) + fabsf(x[i][1])) + (fabsf(x[i][2]) + fabsf(x[i][3]));
      const bool nan = __any_sync(0xffffffffu, all != all);
      nans |= nan ? 1u << i : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = nan ? amax : fmaxf(amax, fabsf(x[i][j]));
    }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  int grown;
  const int e = run_exponent(amax, r.off, old, &grown);
  if (grown > 0) {
    rescale_block(block, values, r.off, grown, lane, 32);
    __syncwarp();
  }
  if (lane == 0 && (r.off == 0 || grown > 0)) *scale = fp8_power(e);
  const float down = fp8_power(-e);
#pragma unroll
  for (int i = 0; i < kShortRun; ++i) {
    if (i >= r.len) break;
    const uint32_t w = nans >> i & 1u ? kFp8NaN4 : fp8_four_scaled(x[i][0], x[i][1], x[i][2], x[i][3], down);
    const int token = r.off + i;
    if (!values) {
      *reinterpret_cast<uint32_t*>(block + key_byte(token, 4 * lane)) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) block[value_byte(token, 4 * lane + j)] = static_cast<uint8_t>(w >> (8 * j));
    }
  }
}

// ---- longer runs ---------------------------------------------------------------
//
// A CTA takes 64 tokens of a (run, tensor, KV head) at a time: their rows come
// into shared memory by asynchronous copies, a stage ahead of the work on them.  Runs of
// one stage are searched for their largest magnitude and converted where they
// lie.  With blocks of up to 128 tokens the two stages are one, without copies
// ahead (prefetching the next rows to L2 gains nothing); with longer ones a run's
// rows come twice.
constexpr int kStageTokens = 64;
template <bool BF16>
struct Stage {
  static constexpr int kThreads = BF16 ? 128 : 256, kWarps = kThreads / 32;
  static constexpr int kPieces = kDim * (BF16 ? 2 : 4) / 16;   // of a row, 16 bytes each
  static constexpr int kRows = kThreads / kPieces;             // that the threads take at a time
  static constexpr int kRow = kDim * (BF16 ? 2 : 4), kPitch = kRow + 16;   // (16: rows in different banks)
  static constexpr int kBytes = kStageTokens * kPitch;
};

// One pass over a stage's tokens.
struct Step {
  Fp8Run r;
  int field;                     // tensor and KV head
  int base;                      // block offset of the stage's first token
  bool search, write;
  bool valid;
};

// The largest magnitude among rows [lo, hi) of a stage over a thread's share of
// them, as bits; vectors with a NaN do not count, but set *nan.  By whole warps:
// one has a row, or two side by side (bf16).
template <bool BF16>
__device__ __forceinline__ uint32_t largest_bits(const uint8_t* stage, int lo, int hi, bool* nan) {
  using S = Stage<BF16>;
  const int row = lo + threadIdx.x / S::kPieces;
  const uint8_t* const mine = stage + row * S::kPitch + threadIdx.x % S::kPieces * 16;
  uint32_t top = 0;
  float odd = 0.f;                                // NaN after a NaN (or infinity)
  {
    const uint8_t* p = mine;
#pragma unroll 4
    for (int r = row; r < hi; r += S::kRows, p += S::kRows * S::kPitch) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
          top = __vmaxu2(top, u[j] & 0x7fff7fffu);
        } else {
          const float x = __uint_as_float(u[j]);
          top = __float_as_uint(fmaxf(__uint_as_float(top), fabsf(x)));
          odd = fmaf(x, 0.f, odd);
        }
      }
    }
  }
  if (BF16) top = max(top << 16, top & 0xffff0000u);
  if (!__any_sync(0xffffffffu, BF16 ? top > 0x7f800000u : odd != odd)) return top;
  float most = 0.f;                               // once more, row by row
  const uint8_t* p = mine;
  const int first = lo + threadIdx.x / 32 * (32 / S::kPieces);   // (the same for the warp)
  const uint32_t neighbours = (S::kPieces == 32 ? 0xffffffffu : 0xffffu) << (threadIdx.x & 31 & ~(S::kPieces - 1));
#pragma unroll 1
  for (int r = first; r < hi; r += S::kRows, p += S::kRows * S::kPitch) {
    float own = 0.f;
    bool bad = false;
    if (r + row - first < hi) {
#pragma unroll 1
      for (int j = 0; j < (BF16 ? 8 : 4); ++j) {
        const float x = BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[j]) : reinterpret_cast<const float*>(p)[j];
        bad = bad || x != x;
        own = fmaxf(own, fabsf(x));
      }
    }
    bad = (__ballot_sync(0xffffffffu, bad) & neighbours) != 0;
    *nan = *nan || bad;
    if (!bad) most = fmaxf(most, own);
  }
  return __float_as_uint(most);
}

// Codes of a stage's tokens that are in the run.  A warp has sixteen
// tokens (float32: a half of their coordinates).
// Keys: eight tokens by four chunks of sixteen coordinates a round, a core matrix
// (128 bytes) per eight lanes.  Values: a lane has four tokens (lane / 8) of eight
// coordinates (lane % 8) twice; lanes eight apart exchange their words to have
// sixteen tokens of a coordinate each.  nan: the run's tokens by bit, or null.
template <bool BF16>
__device__ __forceinline__ void write_codes(const uint8_t* stage, const Fp8Run& r, int base, uint8_t* block, bool values,
                                            float down, const uint8_t* nan) {
  constexpr int kParts = Stage<BF16>::kWarps / 4, kEach = 2 / kParts;   // warps of sixteen tokens, halves of the coordinates each
  const int warp = threadIdx.x >> 5 & 3, part = threadIdx.x >> 7, lane = threadIdx.x & 31;
  const int end = r.off + r.len, unit = base + 16 * warp;     // the warp's first token
  if (unit >= end || unit + 16 <= r.off) return;
  const uint8_t* const rows = stage + 16 * warp * Stage<BF16>::kPitch;
  constexpr int kEight = 8 * (BF16 ? 2 : 4);      // bytes of eight coordinates
  if (!values) {
#pragma unroll
    for (int k = 0; k < 2 * kEach; ++k) {
      const int i = k + 2 * kEach * part;
      const int at = 8 * (i & 1) + (lane & 7), chunk = 4 * (i >> 1) + (lane >> 3), token = unit + at;
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Eight<BF16> x;
        float v[8];
        x.load(rows + at * Stage<BF16>::kPitch + (2 * chunk + h) * kEight);
        x.floats(v);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[2 * h + j] = fp8_four_scaled(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], down);
      }
      if (nan != nullptr && nan[16 * warp + at]) w[0] = w[1] = w[2] = w[3] = kFp8NaN4;
      if (token >= r.off && token < end)
        *reinterpret_cast<uint4*>(block + key_byte(token, 16 * chunk)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
  const int quad = lane >> 3, piece = lane & 7;
  uint32_t fix = 0;                               // bytes of the lane's four tokens that are NaN
  if (nan != nullptr)
    for (int i = 0; i < 4; ++i) fix |= nan[16 * warp + 4 * quad + i] ? 0xffu << (8 * i) : 0u;
#pragma unroll
  for (int g = 0; g < kEach; ++g) {
    const int h = g + kEach * part;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Eight<BF16> x;
      x.load(rows + (4 * quad + i) * Stage<BF16>::kPitch + (piece + 8 * h) * kEight);
      x.floats(v[i]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 4 * c + j;
        w[j] = (fp8_four_scaled(v[0][k], v[1][k], v[2][k], v[3][k], down) & ~fix) | (kFp8NaN4 & fix);
      }
      transpose4<8>(w);
      uint8_t* const dst = block + value_byte(unit, 8 * piece + 64 * h + 4 * c + quad);
      if (unit >= r.off && unit + 16 <= end) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (unit + i >= r.off && unit + i < end) dst[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
      }
    }
  }
}

// Items are (run, tensor, KV head), the heads of a run side by side as in memory;
// the CTAs take every gridDim.x-th.  Where the call's runs are short on average a
// warp takes an item, and the CTA those among its warps' that are not.
template <bool BF16, bool WHOLE>
constexpr int kAppendCtas = BF16 ? 6 : WHOLE ? 4 : 3;   // of an SM, by their stages (float32, blocks of 96: four 15.9 us, three 16.9)

// WHOLE: the two stages are one (blocks of 65 to 128 tokens).
template <bool BF16, bool WHOLE>
__global__ void __launch_bounds__(Stage<BF16>::kThreads, kAppendCtas<BF16, WHOLE>) fp8_append_kernel(Fp8RowsArgs a) {
  constexpr int kThreads = Stage<BF16>::kThreads, kWarps = Stage<BF16>::kWarps;
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ Fp8Runs<kThreads> runs;
  __shared__ long long warp_s[kWarps][2];
  __shared__ uint32_t top_s[kWarps];
  __shared__ uint8_t nan_s[2 * kStageTokens];
  const Fp8Cache& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  runs.find(c, warp_s);
  const bool shorts = runs.tokens <= static_cast<long long>(kShortRun) * runs.total();
  auto values_of = [&](int field) { return a.rows[0] == nullptr || field >= c.n_kv; };
  auto head_of = [&](int field) { return field >= c.n_kv ? field - c.n_kv : field; };
  auto vector_of = [&](const Fp8Run& r, int field) { return static_cast<long long>(r.block) * c.n_kv + head_of(field); };

  // an item's run and field, moved on by a number of items
  struct Item {
    int g, field;
  };
  auto move = [&](Item& it, unsigned by) {
    const unsigned f = it.field + by, over = f / a.fields;
    it.g += over;
    it.field = f - over * a.fields;
  };
  const int total = runs.total();
  int from = 0;
  if (shorts) {
    Item it{0, 0};
    move(it, blockIdx.x * kWarps + warp);
    for (; it.g < total; move(it, gridDim.x * kWarps)) {
      const Fp8Run r = runs.get(c, it.g, &from);
      if (r.block < 0 || r.len > kShortRun) continue;
      const bool values = values_of(it.field);
      append_short<BF16>(r, a.rows[values], a.stride[values], head_of(it.field),
                         (values ? c.v : c.k) + vector_of(r, it.field) * c.block_size * kDim,
                         (values ? c.v_scale : c.k_scale) + vector_of(r, it.field), values);
    }
    if (runs.most <= kShortRun) return;           // (there are no others)
    from = 0;
  }
  // The steps over the CTA's (longer) runs, one after another.
  constexpr int span = WHOLE ? 2 * kStageTokens : kStageTokens;
  Item at{0, 0};
  move(at, blockIdx.x);
  auto first_step = [&]() {                       // of the item or those behind it
    Step s;
    s.valid = false;
    for (; at.g < total && !s.valid; move(at, gridDim.x)) {
      s.field = at.field;
      s.r = runs.get(c, at.g, &from);
      if (s.r.block < 0 || (shorts && s.r.len <= kShortRun)) continue;
      s.base = s.r.off & ~15;
      s.search = s.valid = true;
      s.write = s.r.off + s.r.len - s.base <= span;
    }
    return s;
  };
  auto step_after = [&](const Step& s) {
    Step n = s;
    const int first = s.r.off & ~15, end = s.r.off + s.r.len;
    n.base += span;
    if (n.base < end) return n;                   // more of the run in this pass
    if (s.write) return first_step();
    n.base = first;                               // found the largest: now the codes
    n.search = false;
    n.write = true;
    return n;
  };
  auto copy = [&](const Step& s, int k) {         // its rows, sixteen bytes a thread at a time
    if (s.valid) {
      constexpr int kPieces = Stage<BF16>::kPieces, kElem = BF16 ? 2 : 4;
      const bool values = values_of(s.field);
      const int lo = max(s.r.off, s.base), hi = min(s.r.off + s.r.len, s.base + span);
      const long long pitch = a.stride[values] * kElem;
      const uint8_t* src = static_cast<const uint8_t*>(a.rows[values]) + head_of(s.field) * Stage<BF16>::kRow +
                           (s.r.row + static_cast<long long>(lo + tid / kPieces - s.r.off)) * pitch + tid % kPieces * 16;
      uint8_t* dst = stages + (k & 1) * Stage<BF16>::kBytes + (lo + tid / kPieces - s.base) * Stage<BF16>::kPitch + tid % kPieces * 16;
      constexpr int kRows = Stage<BF16>::kRows;
#pragma unroll 8
      for (int t = lo + tid / kPieces; t < hi; t += kRows) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
        src += kRows * pitch;
        dst += kRows * Stage<BF16>::kPitch;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Step now = first_step();
  copy(now, 0);
  uint32_t top = 0;
  bool nan = false;
  float down = 1.f;
  for (int k = 0; now.valid; ++k) {
    const Step next = step_after(now);
    if (!WHOLE) copy(next, k + 1);
    const uint8_t* const stage = stages + (WHOLE ? 0 : k & 1) * Stage<BF16>::kBytes;
    const bool values = values_of(now.field);
    const long long vec = vector_of(now.r, now.field);
    uint8_t* const block = (values ? c.v : c.k) + vec * c.block_size * kDim;
    float* const scale = (values ? c.v_scale : c.k_scale) + vec;
    const float old = now.search && now.r.off > 0 ? *scale : 0.f;
    const int lo = max(now.r.off, now.base) - now.base, hi = min(now.r.off + now.r.len, now.base + span) - now.base;
    if (WHOLE) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    if (now.search) {
      if (now.base == (now.r.off & ~15)) top = 0, nan = false;
      top = max(top, largest_bits<BF16>(stage, lo, hi, &nan));
      if (now.base + span >= now.r.off + now.r.len) {
        // the run's scale
        const uint32_t most = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) top_s[warp] = most;
        nan = __syncthreads_or(nan);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = max(top, top_s[w]);
        int grown;
        const int e = run_exponent(__uint_as_float(top), now.r.off, old, &grown);
        if (grown > 0) {
          rescale_block(block, values, now.r.off, grown, tid, kThreads);
          __syncthreads();
        }
        if (tid == 0 && (now.r.off == 0 || grown > 0)) *scale = fp8_power(e);
        down = fp8_power(-e);
      }
    }
    if (now.write) {
      if (nan) {                                  // which tokens have one (the same for the whole CTA)
        if (tid < span) {
          bool here = false;
          if (tid >= lo && tid < hi)
            for (int d = 0; d < kDim; ++d) {
              const uint8_t* const p = stage + tid * Stage<BF16>::kPitch;
              const float v = BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[d])
                                   : reinterpret_cast<const float*>(p)[d];
              here = here || v != v;
            }
          nan_s[tid] = here;
        }
        __syncthreads();
      }
      for (int t = 0; t < span; t += kStageTokens)
        write_codes<BF16>(stage + t * Stage<BF16>::kPitch, now.r, now.base + t, block, values, down, nan ? nan_s + t : nullptr);
    }
    __syncthreads();                              // (the stage may be filled again)
    if (WHOLE) copy(next, 0);
    now = next;
  }
}

// ---- reading back --------------------------------------------------------------

template <bool BF16>
constexpr int kReadWarps = BF16 ? 2 : 4;   // (four take 129 us in place of 122 for 131072 tokens in bf16, two 51 in place of 49 for ragged ranges in float32)

// 32 bytes to a row: one store where they are aligned to as many (two of 16 bytes
// that skip 16 each leave half sectors: 131 us in place of 102 for 65536 tokens
// of eight heads in float32).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Eight values as bf16 pairs; eight, or two times eight, to a row.
__device__ __forceinline__ void pack8(const float (&v)[8], uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* rows, long long at, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t w[4];
    pack8(v, w);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(rows) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
    store32(static_cast<float*>(rows) + at, w);
  }
}
template <bool BF16>
__device__ __forceinline__ void store16(void* rows, long long at, const float (&lo)[8], const float (&hi)[8]) {
  if constexpr (BF16) {
    uint32_t w[8];
    pack8(lo, w);
    pack8(hi, w + 4);
    store32(static_cast<__nv_bfloat16*>(rows) + at, w);
  } else {
    store8<BF16>(rows, at, lo);
    store8<BF16>(rows, at + 8, hi);
  }
}
__device__ __forceinline__ void eight_values(uint32_t lo, uint32_t hi, float scale, float (&v)[8]) {
  const uint32_t w[2] = {lo, hi};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = fp8_floats(w[i >> 1] >> (16 * (i & 1)));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

// A CTA has the tokens of a window for one (tensor, KV head), its neighbours the
// others.  A warp takes sixteen tokens at a time, with the append's shares of
// lanes.
template <bool BF16>
__global__ void __launch_bounds__(32 * kReadWarps<BF16>) fp8_read_kernel(Fp8RowsArgs a) {
  __shared__ Fp8Finder found;
  const Fp8Cache& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane & 3, piece = lane >> 2;
  const int field = blockIdx.x % a.fields;
  const int count = fp8_find_runs(c, blockIdx.x / a.fields * a.window, a.window, found);
  int turn = 0;
  const bool values = a.rows[0] == nullptr || field >= c.n_kv;
  const int head = field >= c.n_kv ? field - c.n_kv : field;
  void* const rows = values ? a.rows[1] : a.rows[0];
  const long long stride = values ? a.stride[1] : a.stride[0];
  for (int i = 0; i < count; ++i) {
    const Fp8Run r = found.runs[i];
    const long long vec = static_cast<long long>(r.block) * c.n_kv + head;
    const uint8_t* const block = (values ? c.v : c.k) + vec * c.block_size * kDim;
    const float scale = __ldg((values ? c.v_scale : c.k_scale) + vec);
    const int end = r.off + r.len;
    for (int unit = r.off & ~15; unit < end; unit += 16, ++turn) {
      if (turn % kReadWarps<BF16> != warp) continue;
      auto row_at = [&](int token) { return (static_cast<long long>(r.row) + token - r.off) * stride + head * kDim; };
      if (!values) {
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __ldg(reinterpret_cast<const uint4*>(block + key_byte(unit + 4 * k + quad, 16 * piece)));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int token = unit + 4 * k + quad;
          if (token < r.off || token >= end) continue;
          float lo[8], hi[8];
          eight_values(w[k].x, w[k].y, scale, lo);
          eight_values(w[k].z, w[k].w, scale, hi);
          store16<BF16>(rows, row_at(token) + 16 * piece, lo, hi);
        }
      } else {
        uint4 w[4];                               // coordinates quad and quad + 4 of two pieces
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = __ldg(reinterpret_cast<const uint4*>(block + value_byte(unit, 8 * piece + 64 * (k >> 1) + 4 * (k & 1) + quad)));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t four[2][4];                    // [half of the eight coordinates][token]
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t u[4] = {w[2 * h + k].x, w[2 * h + k].y, w[2 * h + k].z, w[2 * h + k].w};
            transpose4<1>(u);
            transpose_bytes(u, four[k]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int token = unit + 4 * quad + j;
            if (token < r.off || token >= end) continue;
            float v[8];
            eight_values(four[0][j], four[1][j], scale, v);
            store8<BF16>(rows, row_at(token) + 8 * piece + 64 * h, v);
          }
        }
      }
    }
  }
}

// As many CTAs as the SMs have room for, or as there can be items.
template <bool BF16, bool WHOLE>
cudaError_t append(const Fp8RowsArgs& a, cudaStream_t stream) {
  using S = Stage<BF16>;
  const int smem = WHOLE ? a.c.block_size * S::kPitch : 2 * S::kBytes;
  const cudaError_t err =
      cudaFuncSetAttribute(fp8_append_kernel<BF16, WHOLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * S::kBytes);
  if (err != cudaSuccess) return err;
  // (an SM has 228 KB; a CTA takes 1 KB more than it asks for)
  const int fit = std::min<int>(kAppendCtas<BF16, WHOLE>, (228 << 10) / (smem + static_cast<int>(sizeof(Fp8Runs<S::kThreads>)) + 1536));
  const long long runs = std::min<long long>(a.c.n_tokens, a.c.n_tokens / a.c.block_size + 2ll * a.c.batch);
  const long long ctas = std::min<long long>(runs * a.fields, fit * a.num_sms);
  fp8_append_kernel<BF16, WHOLE><<<static_cast<unsigned>(ctas), S::kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

long long windows_of(const Fp8RowsArgs& a) {
  return (static_cast<long long>(a.c.n_tokens) + a.window - 1) / a.window;
}

// Read: windows of 16 tokens, or of 64 where that leaves 32 CTAs an SM (fewer
// searches for the runs).
long long read_grid(Fp8RowsArgs& a) {
  a.fields = ((a.rows[0] != nullptr) + (a.rows[1] != nullptr)) * a.c.n_kv;
  a.window = kFp8Window;
  if (windows_of(a) * a.fields < static_cast<long long>(kReadCtasPerSm) * a.num_sms) a.window = 16;
  return windows_of(a) * a.fields;
}

}  // namespace

cudaError_t launch_fp8_append(const Fp8RowsArgs& args, bool bf16, cudaStream_t stream) {
  Fp8RowsArgs a = args;
  a.fields = ((a.rows[0] != nullptr) + (a.rows[1] != nullptr)) * a.c.n_kv;
  const bool whole = a.c.block_size > kStageTokens && a.c.block_size <= 2 * kStageTokens;
  if (whole) return bf16 ? append<true, true>(a, stream) : append<false, true>(a, stream);
  return bf16 ? append<true, false>(a, stream) : append<false, false>(a, stream);
}

cudaError_t launch_fp8_read(const Fp8RowsArgs& args, bool bf16, cudaStream_t stream) {
  Fp8RowsArgs a = args;
  const long long grid = read_grid(a);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (bf16) fp8_read_kernel<true><<<static_cast<unsigned>(grid), 32 * kReadWarps<true>, 0, stream>>>(a);
  else fp8_read_kernel<false><<<static_cast<unsigned>(grid), 32 * kReadWarps<false>, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
