// Attention of several new tokens per sequence over the packed cache.
//
// The n new tokens of a sequence are the last n of its context; token i sees
// positions 0 .. context - n + i.  As in a decode step the scores are
//   s_t = scale (n_t <R q, c[code_t]> + gamma_t sqrt(pi/2)/m <S q, 2 bits_t - 1>)
// and the output is R^T sum_t softmax(s)_t n^v_t c^v[code_t].
//
// One CTA per (token, query head): 128 threads are 128 context tokens while
// scores are formed and 128 coordinates while values are added; the running
// maximum and sum of the softmax are fp32.
#include <cuda_bf16.h>

#include "kernels.h"

namespace tq {
namespace {

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

__global__ void __launch_bounds__(kDim) extend_simt_kernel(ExtendArgs a) {
  __shared__ float q_s[kDim], qr_s[kDim], qs_s[kDim], p_s[kDim], o_s[kDim], lev_k[kMaxLevels], lev_v[kMaxLevels];
  __shared__ float red[4];
  __shared__ int off_s[kDim / 32];
  __shared__ long long blk_s[kDim / 32];
  const DecodeArgs& d = a.d;
  const int tid = threadIdx.x;
  const int token = blockIdx.x, head = blockIdx.y, kvh = head / d.group;
  int lo = 0, hi = d.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.query_start[mid] <= token) lo = mid;
    else hi = mid;
  }
  const int s0 = a.query_start[lo], s1 = a.query_start[lo + 1];
  if (token < s0 || token >= s1) return;          // behind the last sequence
  const long long vec = static_cast<long long>(token) * d.n_q + head;
  __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.out) + vec * kDim;
  const int ctx = d.context_lens[lo];
  const bool bad = ctx < 0 || ctx > d.max_context || ctx > static_cast<long long>(d.max_blocks) * d.block_size ||
                   s0 < 0 || s1 > a.n_tokens;
  if (bad && tid == 0) atomicCAS(d.error, 0, kErrContext);
  const int seen = bad ? 0 : ctx - (s1 - s0) + (token - s0) + 1;   // visible positions
  q_s[tid] = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(d.q)[vec * kDim + tid])
                      : static_cast<const float*>(d.q)[vec * kDim + tid];
  if (tid < kMaxLevels) {
    lev_k[tid] = d.tables->k_levels[tid];
    lev_v[tid] = d.tables->v_levels[tid];
  }
  __syncthreads();
  float yr = 0.f, ys = 0.f;
  for (int i = 0; i < kDim; ++i) {
    yr = fmaf(d.Rt[i * kDim + tid], q_s[i], yr);
    ys = fmaf(d.St[i * kDim + tid], q_s[i], ys);
  }
  qr_s[tid] = yr;
  qs_s[tid] = ys;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < seen; t0 += kDim) {
    __syncthreads();
    if (tid < kDim / 32) {                        // (a group of 32 tokens lies within one block)
      const int pos = t0 + 32 * tid;
      long long blk = -1;
      if (pos < seen) {
        const int col = pos / d.block_size;
        blk = d.block_table ? d.block_table[static_cast<long long>(lo) * d.max_blocks + col]
                            : static_cast<long long>(lo) * d.max_blocks + col;
        if (blk < 0 || blk >= d.num_blocks) {
          blk = -1;
          atomicCAS(d.error, 0, kErrBlock);
        }
      }
      blk_s[tid] = blk;
      off_s[tid] = pos % d.block_size;
    }
    __syncthreads();
    const long long blk = blk_s[tid >> 5];
    float s = -INFINITY, nv = 0.f;
    if (t0 + tid < seen && blk >= 0) {
      const long long row = (blk * d.n_kv + kvh) * d.block_size + off_s[tid >> 5] + (tid & 31);
      const uint32_t* const codes = reinterpret_cast<const uint32_t*>(d.k_codes + row * (d.k_bits * 16));
      float dot = 0.f, sgn = 0.f;
      for (int w = 0; w < 4; ++w) {
        uint32_t pl[4] = {0, 0, 0, 0};
        for (int p = 0; p < d.k_bits; ++p) pl[p] = codes[p * 4 + w];
        const uint32_t bits = d.k_qjl ? reinterpret_cast<const uint32_t*>(d.k_qjl + row * 16)[w] : 0u;
        for (int j = 0; j < 32; ++j) {
          const int code = ((pl[0] >> j) & 1) | ((pl[1] >> j) & 1) << 1 | ((pl[2] >> j) & 1) << 2 |
                           ((pl[3] >> j) & 1) << 3;
          dot = fmaf(qr_s[32 * w + j], lev_k[code], dot);
          sgn += (bits >> j) & 1 ? qs_s[32 * w + j] : -qs_s[32 * w + j];
        }
      }
      s = load_norm(d.k_norm, row, d.norm16) * dot;
      if (d.k_qjl) s = fmaf(load_norm(d.k_rnorm, row, d.norm16) * d.qjl_coef, sgn, s);
      s *= d.scale;
      nv = load_norm(d.v_norm, row, d.norm16);
    }
    const float m_new = fmaxf(m, block_max(s, red));
    const float shift = m_new == -INFINITY ? 0.f : m_new;
    const float p = __expf(s - shift);
    p_s[tid] = p == 0.f ? 0.f : p * nv;
    float sum = p;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    const float keep = __expf(m - shift);
    l = l * keep + ((red[0] + red[1]) + (red[2] + red[3]));
    acc *= keep;
    m = m_new;
    for (int g = 0; g < kDim / 32; ++g) {
      if (blk_s[g] < 0) continue;
      const uint32_t* const words = reinterpret_cast<const uint32_t*>(d.v_codes);
      uint32_t pl[4] = {0, 0, 0, 0};
      for (int p = 0; p < d.v_bits; ++p)
        pl[p] = words[transposed_word(blk_s[g], kvh, d.n_kv, d.v_bits, p, tid, d.block_size, off_s[g])];
      for (int t = 0; t < 32; ++t) {
        const int code = ((pl[0] >> t) & 1) | ((pl[1] >> t) & 1) << 1 | ((pl[2] >> t) & 1) << 2 |
                         ((pl[3] >> t) & 1) << 3;
        acc = fmaf(p_s[32 * g + t], lev_v[code], acc);
      }
    }
  }
  o_s[tid] = l == 0.f ? 0.f : acc / l;         // (a NaN in a visible token shows)
  __syncthreads();
  float o = 0.f;
  for (int j = 0; j < kDim; ++j) o = fmaf(d.R[j * kDim + tid], o_s[j], o);
  out[tid] = __float2bfloat16_rn(o);
}

}  // namespace

size_t extend_workspace_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_extend(const ExtendArgs& a, void*, cudaStream_t stream) {
  extend_simt_kernel<<<dim3(a.n_tokens, a.d.n_q), kDim, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
