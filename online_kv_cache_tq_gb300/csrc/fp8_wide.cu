// Many rows per sequence over the 8-bit cache: key tiles (128 tokens of a KV
// head) of such a sequence are expanded once into the operands of the wide form
// (extend_wide.cu): keys as fp16 and values as bf16 numbers, both exactly the
// codes, in the swizzled layout that its products read, with the blocks' scales
// as the columns' factors.  Then a tile serves every row tile of 256 rows.
//
// The bound is memory: 32 KB in and 64.5 KB out a tile; 1008 tiles take 31 us
// (3.1 TB/s).  A chunk of 2048 tokens on 14001, 64/8 heads, takes 867 us with it,
// 1.16 PFLOP/s, where keys with large channels have every tile searched for its
// maximum, and 795 us (1.27) where not.
#include "dependent.cuh"
#include "fp8_common.cuh"
#include "tc_ptx.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;
constexpr int kBlockBytes = kTile * 128;          // a 64-column block of a 128-row operand
constexpr int kExpandThreads = 256;
constexpr int kExpandSmem = 2 * kTile * kDim + kTileImageBytes + 128;   // codes, operands (128: alignment)

// Bytes `i` of two words as two 16-bit halves; eight codes (byte i of eight
// words, or two words) as eight fp16 or bf16 numbers.
__device__ __forceinline__ uint32_t halves(uint32_t two) {
  const __half2 h = fp8_halves(two);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf16s(uint32_t two) {
  const float2 f = fp8_floats(two);
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__global__ void __launch_bounds__(kExpandThreads) fp8_expand_kernel(Fp8Cache c, ExtendArgs a, float to_log2) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ float scale_s[2][4];                 // keys and values, by group of 32 tokens
  __shared__ long long row_s[4];
  __shared__ uint32_t there_s[4], nan_s[2][4];    // tokens by bit
  __shared__ float square_s[2][kTile], reach_s[4];
  uint8_t* const smem = smem_raw + ((128u - (ptx::smem_u32(smem_raw) & 127u)) & 127u);
  uint8_t* const codes = smem;                    // keys, then values
  uint8_t* const image = smem + 2 * kTile * kDim;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  wait_prerequisites();
  const long long total = a.ws_expand[c.batch];
  for (long long g = blockIdx.x; g < total; g += gridDim.x) {
    int lo = 0, hi = c.batch;                     // the last sequence whose tiles start at or before g
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.ws_expand[mid] <= g) lo = mid;
      else hi = mid;
    }
    const int ctx = a.ws_seq[lo].z, tiles = max(1, (ctx + kTile - 1) / kTile);
    const int local = static_cast<int>(g - a.ws_expand[lo]), kvh = local / tiles, pos0 = (local - kvh * tiles) * kTile;
    if (tid < 4) {                                // a group of 32 tokens each
      const int pos = pos0 + 32 * tid, col = pos / c.block_size, off = pos - col * c.block_size;
      long long row = -1;
      uint32_t there = 0;
      if (pos < ctx) {
        const long long at = static_cast<long long>(lo) * c.max_blocks + col;
        const int id = c.block_table ? c.block_table[at] : static_cast<int>(at);
        if (id < 0 || id >= c.num_blocks) {
          atomicCAS(c.error, 0, kErrBlock);
        } else {
          const long long vec = static_cast<long long>(id) * c.n_kv + kvh;
          row = vec * c.block_size + off;
          there = ctx - pos >= 32 ? 0xffffffffu : (1u << (ctx - pos)) - 1u;
          scale_s[0][tid] = c.k_scale[vec];
          scale_s[1][tid] = c.v_scale[vec];
        }
      }
      row_s[tid] = row;
      there_s[tid] = there;
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // (the last tile's image has left)
    __syncthreads();
    {                                             // the codes of the groups: 4 KB of keys and of values each
      const uint4 none = make_uint4(0, 0, 0, 0);
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const long long row = row_s[i & 3];
        w[i] = row < 0 ? none : __ldg(reinterpret_cast<const uint4*>((i < 4 ? c.k : c.v) + row * kDim) + tid);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(codes + (i >> 2) * kTile * kDim + (i & 3) * 32 * kDim)[tid] = w[i];
    }
    __syncthreads();
    if (warp < 4) {                               // vectors that are NaN: all their codes are
      const int t = tid;
      const uint8_t k = codes[(t >> 3) * 1024 + (t & 7) * 16], v = codes[kTile * kDim + (t >> 4) * 2048 + (t & 15)];
      const uint32_t kn = __ballot_sync(0xffffffffu, (k & 127) == 127), vn = __ballot_sync(0xffffffffu, (v & 127) == 127);
      if (lane == 0) nan_s[0][warp] = kn, nan_s[1][warp] = vn;
    }
    __syncthreads();
    // keys: eight lanes a half row of 64 coordinates, rows in expansion order
#pragma unroll 2
    for (int i = tid; i < 2 * kTile * 8; i += kExpandThreads) {
      const int p = i & 7, row = (i >> 3) & (kTile - 1), half = i >> 10, grp = row >> 5, bit = expanded_bit(row & 31);
      const int t = 32 * grp + bit;
      const bool on = (there_s[grp] & ~nan_s[0][grp]) >> bit & 1u;
      uint2 w = *reinterpret_cast<const uint2*>(codes + (t >> 3) * 1024 + (4 * half + (p >> 1)) * 128 + (t & 7) * 16 + 8 * (p & 1));
      if (!on) w = make_uint2(0, 0);
      const uint4 h = make_uint4(halves(w.x), halves(w.x >> 16), halves(w.y), halves(w.y >> 16));
      *reinterpret_cast<uint4*>(image + half * kBlockBytes + row * 128 + ((p ^ (row & 7)) << 4)) = h;
      float square = 0.f;
      const uint32_t u[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[q]));
        square = fmaf(f.x, f.x, fmaf(f.y, f.y, square));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
      if (p == 0) square_s[half][row] = square;
    }
    // values: a coordinate's 32 tokens of a group, as four chunks of eight in expansion order
#pragma unroll
    for (int i = tid; i < 4 * kDim; i += kExpandThreads) {
      const int dim = i & (kDim - 1), grp = i >> 7;
      const uint4* const src = reinterpret_cast<const uint4*>(codes + kTile * kDim + 2 * grp * 2048 + dim * 16);
      const uint4 x = src[0], y = src[kDim];      // (sixteen tokens on: 2048 bytes)
      uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      const uint32_t on = there_s[grp] & ~nan_s[1][grp];
      if (on != 0xffffffffu) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t four = on >> (4 * q) & 15u;
          w[q] &= (four & 1u ? 0xffu : 0u) | (four & 2u ? 0xff00u : 0u) | (four & 4u ? 0xff0000u : 0u) | (four & 8u ? 0xff000000u : 0u);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {               // tokens j, 4 + j, .. 28 + j
        uint32_t out[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) out[q] = bf16s(__byte_perm(w[2 * q], w[2 * q + 1], j | (4 + j) << 4));
        const int p = 4 * (grp & 1) + j;
        *reinterpret_cast<uint4*>(image + kExtendImageBytes + (grp >> 1) * kBlockBytes + dim * 128 + ((p ^ (dim & 7)) << 4)) =
            make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
    ptx::fence_async_shared();
    __syncthreads();
    if (tid == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                   ::"l"(reinterpret_cast<uint64_t>(a.ws_tiles + g * kTileImageBytes)), "r"(ptx::smem_u32(image)),
                     "r"(kTileImageBytes)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    TileMeta* const meta = a.ws_meta + g;
    if (tid < kTile) {                            // by operand row
      const int grp = warp, bit = expanded_bit(lane);
      const bool there = there_s[grp] >> bit & 1u;
      const float nan = __int_as_float(0x7fc00000);
      const float f = !there ? 0.f : nan_s[0][grp] >> bit & 1u ? nan : scale_s[0][grp] * to_log2;
      meta->key_factor[tid] = f;
      meta->value_factor[tid] = !there ? 0.f : nan_s[1][grp] >> bit & 1u ? nan : scale_s[1][grp];
      const float reach = fabsf(f) * sqrtf(square_s[0][tid] + square_s[1][tid]);
      const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(reach) & 0x7fffffffu);   // (a NaN above all)
      if (lane == 0) {
        reach_s[warp] = __uint_as_float(bits);
        meta->valid[warp] = there_s[warp];
      }
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t bits = 0;
      for (int w = 0; w < 4; ++w) bits = max(bits, __float_as_uint(reach_s[w]));
      meta->reach = __uint_as_float(bits);
      uint32_t odd = 0;                           // tokens whose factors are not their block's
      for (int g = 0; g < 4; ++g) odd |= nan_s[0][g] | nan_s[1][g] | ~there_s[g];
      meta->grouped = odd == 0;
    }
    __syncwarp();                                 // (thread 0's neighbours write there_s next)
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // nothing is in flight when the CTA ends
}

}  // namespace

cudaError_t launch_fp8_expand(const Fp8Cache& cache, const ExtendArgs& args, float scale, cudaStream_t stream) {
  cudaError_t err = cudaFuncSetAttribute(fp8_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(fp8_expand_kernel, dim3(2 * args.d.num_sms), kExpandThreads, kExpandSmem, stream, cache, args,
                          scale * 1.4426950408889634f);
}

}  // namespace tq
