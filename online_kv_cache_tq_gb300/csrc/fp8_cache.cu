// Writing the 8-bit cache and reading it back.
//
// Append.  For every (block, KV head) that the call's tokens touch, keys and
// values apart, a = max |x| over the new tokens, and the scale is the least
// 2^e, -40 <= e <= 14, with 448 2^e >= a, or the block's old one if that is
// larger and the block already holds earlier tokens (the run does not begin at
// its first offset).  The codes are rn_e4m3(x 2^-e); where the scale grew, the
// earlier tokens' codes become rn_e4m3(code 2^(e_old - e)).  A power of two
// loses nothing but codes that leave e4m3's normal range.
//
// Read.  x = code 2^e, exact in either type.
#include "fp8_common.cuh"

namespace tq {
namespace {

constexpr int kShortRun = 8;      // tokens that one warp appends alone

template <bool BF16>
struct Eight {                    // eight neighbouring coordinates of a row as they lie in memory
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* rows, long long at) {
    const uint4* const p = BF16 ? reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(rows) + at)
                                : reinterpret_cast<const uint4*>(static_cast<const float*>(rows) + at);
    w[0] = __ldg(p);
    if constexpr (!BF16) w[1] = __ldg(p + 1);
  }
  __device__ __forceinline__ void clear() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (!BF16) w[1] = w[0];
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
#pragma unroll
  for (int i = 0; i < kShortRun; ++i)
    if (i < r.len) {
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fabsf(x[i][j]));   // (a NaN is no magnitude)
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
    const bool nan = __any_sync(0xffffffffu, x[i][0] != x[i][0] || x[i][1] != x[i][1] || x[i][2] != x[i][2] || x[i][3] != x[i][3]);
    const uint32_t w = nan ? kFp8NaN4 : fp8_four(x[i][0] * down, x[i][1] * down, x[i][2] * down, x[i][3] * down);
    const int token = r.off + i;
    if (!values) {
      *reinterpret_cast<uint32_t*>(block + key_byte(token, 4 * lane)) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) block[value_byte(token, 4 * lane + j)] = static_cast<uint8_t>(w >> (8 * j));
    }
  }
}

// A longer run, by the CTA: WARPS groups of sixteen tokens at a time.  A thread
// has eight coordinates of four tokens twice.  Keys: tokens 4 i + (lane & 3) of
// the warp's sixteen, coordinates 16 (lane / 4) and the eight behind them, so
// that a row is read and a core matrix written in whole lines.  Values: tokens
// 4 (lane & 3) + i, coordinates 8 (lane / 4) and those 64 on; four lanes
// exchange their words to have sixteen tokens of a coordinate each.
template <bool BF16, int WARPS>
__device__ __forceinline__ void append_long(const Fp8Run& r, const void* rows, long long stride, int head,
                                            uint8_t* block, float* scale, bool values, float* amax_s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane & 3, piece = lane >> 2;
  const float old = r.off > 0 ? *scale : 0.f;
  const int first = r.off & ~15, end = r.off + r.len, step = 16 * WARPS;
  Eight<BF16> x[8];
  auto token_of = [&](int base, int i) { return base + 16 * warp + (values ? 4 * quad + i : 4 * i + quad); };
  auto load = [&](int base) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const int token = token_of(base, m >> 1);
      const int coord = values ? 8 * piece + 64 * (m & 1) : 16 * piece + 8 * (m & 1);
      if (token >= r.off && token < end)
        x[m].load(rows, (static_cast<long long>(r.row) + token - r.off) * stride + head * kDim + coord);
      else x[m].clear();
    }
  };
  float amax = 0.f;
  for (int base = first; base < end; base += step) {
    load(base);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      float v[8];
      x[m].floats(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
    }
  }
  const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
  if (lane == 0) amax_s[warp] = __uint_as_float(bits);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) amax = fmaxf(amax, amax_s[w]);
  int grown;
  const int e = run_exponent(amax, r.off, old, &grown);
  if (grown > 0) rescale_block(block, values, r.off, grown, threadIdx.x, 32 * WARPS);
  __syncthreads();                                // (also: amax_s is read, the next run may write it)
  if (threadIdx.x == 0 && (r.off == 0 || grown > 0)) *scale = fp8_power(e);
  const float down = fp8_power(-e);
  for (int base = first; base < end; base += step) {
    if (end - first > step) load(base);           // (else the one pass is still here)
    uint32_t nan = 0;                             // by i: whether the token's vector has a NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a[8], b[8];
      x[2 * i].floats(a);
      x[2 * i + 1].floats(b);
      bool here = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) here = here || a[j] != a[j] || b[j] != b[j];
      // (a token's eight lanes have the same quad)
      nan |= (__ballot_sync(0xffffffffu, here) & (0x11111111u << quad)) != 0 ? 1u << i : 0u;
    }
    if (!values) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = token_of(base, i);
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[8];
          x[2 * i + h].floats(v);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[2 * h + j] = nan & (1u << i) ? kFp8NaN4
                                           : fp8_four(v[4 * j] * down, v[4 * j + 1] * down, v[4 * j + 2] * down, v[4 * j + 3] * down);
        }
        if (token >= r.off && token < end)
          *reinterpret_cast<uint4*>(block + key_byte(token, 16 * piece)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      const int unit = base + 16 * warp;          // the warp's sixteen tokens
      uint32_t fix = 0;                           // bytes of the lane's four tokens that are NaN
#pragma unroll
      for (int i = 0; i < 4; ++i) fix |= nan & (1u << i) ? 0xffu << (8 * i) : 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i + h].floats(v[i]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = 4 * c + j;
            w[j] = (fp8_four(v[0][k] * down, v[1][k] * down, v[2][k] * down, v[3][k] * down) & ~fix) | (kFp8NaN4 & fix);
          }
          transpose4(w);
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
  }
}

template <bool BF16, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) fp8_append_kernel(Fp8RowsArgs a) {
  __shared__ Fp8Run runs[kFp8Window];
  __shared__ int scratch[3];
  __shared__ float amax_s[WARPS];
  const Fp8Cache& c = a.c;
  const int warp = threadIdx.x >> 5;
  const bool values = a.rows[0] == nullptr || blockIdx.z == 1;
  const int head = blockIdx.y;
  const void* const rows = values ? a.rows[1] : a.rows[0];
  const long long stride = values ? a.stride[1] : a.stride[0];
  const int count = fp8_find_runs(c, blockIdx.x * a.window, a.window, runs, scratch);
  auto block_of = [&](const Fp8Run& r) {
    return (values ? c.v : c.k) + (static_cast<long long>(r.block) * c.n_kv + head) * c.block_size * kDim;
  };
  auto scale_of = [&](const Fp8Run& r) {
    return (values ? c.v_scale : c.k_scale) + static_cast<long long>(r.block) * c.n_kv + head;
  };
  for (int i = warp; i < count; i += WARPS) {
    const Fp8Run r = runs[i];
    if (r.len <= kShortRun) append_short<BF16>(r, rows, stride, head, block_of(r), scale_of(r), values);
  }
  for (int i = 0; i < count; ++i) {
    const Fp8Run r = runs[i];
    if (r.len > kShortRun) append_long<BF16, WARPS>(r, rows, stride, head, block_of(r), scale_of(r), values, amax_s);
  }
}

// ---- reading back --------------------------------------------------------------

constexpr int kReadWarps = 4;

// Eight values to a row.
__device__ __forceinline__ void store8(void* rows, bool bf16, long long at, const float (&v)[8]) {
  if (bf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(rows) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* const p = reinterpret_cast<float4*>(static_cast<float*>(rows) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
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

// A warp takes sixteen tokens at a time, with the append's shares of lanes.
template <bool BF16>
__global__ void __launch_bounds__(32 * kReadWarps) fp8_read_kernel(Fp8RowsArgs a) {
  __shared__ Fp8Run runs[kFp8Window];
  __shared__ int scratch[3];
  const Fp8Cache& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane & 3, piece = lane >> 2;
  const bool values = a.rows[0] == nullptr || blockIdx.z == 1;
  const int head = blockIdx.y;
  void* const rows = values ? a.rows[1] : a.rows[0];
  const long long stride = values ? a.stride[1] : a.stride[0];
  const int count = fp8_find_runs(c, blockIdx.x * a.window, a.window, runs, scratch);
  int turn = 0;
  for (int i = 0; i < count; ++i) {
    const Fp8Run r = runs[i];
    const long long vec = static_cast<long long>(r.block) * c.n_kv + head;
    const uint8_t* const block = (values ? c.v : c.k) + vec * c.block_size * kDim;
    const float scale = __ldg((values ? c.v_scale : c.k_scale) + vec);
    const int end = r.off + r.len;
    for (int unit = r.off & ~15; unit < end; unit += 16, ++turn) {
      if (turn % kReadWarps != warp) continue;
      auto row_at = [&](int token) { return (static_cast<long long>(r.row) + token - r.off) * stride + head * kDim; };
      if (!values) {
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __ldg(reinterpret_cast<const uint4*>(block + key_byte(unit + 4 * k + quad, 16 * piece)));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int token = unit + 4 * k + quad;
          if (token < r.off || token >= end) continue;
          float v[8];
          eight_values(w[k].x, w[k].y, scale, v);
          store8(rows, BF16, row_at(token) + 16 * piece, v);
          eight_values(w[k].z, w[k].w, scale, v);
          store8(rows, BF16, row_at(token) + 16 * piece + 8, v);
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
            transpose4(u);
            transpose_bytes(u, four[k]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int token = unit + 4 * quad + j;
            if (token < r.off || token >= end) continue;
            float v[8];
            eight_values(four[0][j], four[1][j], scale, v);
            store8(rows, BF16, row_at(token) + 8 * piece + 64 * h, v);
          }
        }
      }
    }
  }
}

// Tokens of a window: as few as leave the grid at about 8192 CTAs, so that the
// runs of a decode step spread over many.
int window_of(const Fp8RowsArgs& a, int tensors) {
  int w = 4;
  while (w < kFp8Window && (static_cast<long long>(a.c.n_tokens) + w - 1) / w * a.c.n_kv * tensors > 8192) w *= 2;
  return w;
}

template <bool BF16>
cudaError_t append(const Fp8RowsArgs& a, dim3 grid, cudaStream_t stream) {
  if (a.c.block_size <= 64) fp8_append_kernel<BF16, 4><<<grid, 128, 0, stream>>>(a);
  else fp8_append_kernel<BF16, 8><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

dim3 grid_of(Fp8RowsArgs& a) {
  const int tensors = (a.rows[0] != nullptr) + (a.rows[1] != nullptr);
  a.window = window_of(a, tensors);
  return dim3((a.c.n_tokens + a.window - 1) / a.window, a.c.n_kv, tensors);
}

}  // namespace

cudaError_t launch_fp8_append(const Fp8RowsArgs& args, bool bf16, cudaStream_t stream) {
  Fp8RowsArgs a = args;
  const dim3 grid = grid_of(a);
  return bf16 ? append<true>(a, grid, stream) : append<false>(a, grid, stream);
}

cudaError_t launch_fp8_read(const Fp8RowsArgs& args, bool bf16, cudaStream_t stream) {
  Fp8RowsArgs a = args;
  const dim3 grid = grid_of(a);
  if (bf16) fp8_read_kernel<true><<<grid, 32 * kReadWarps, 0, stream>>>(a);
  else fp8_read_kernel<false><<<grid, 32 * kReadWarps, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
