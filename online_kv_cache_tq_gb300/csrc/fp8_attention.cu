// Attention over the 8-bit cache: a warp per (token, query head), a lane per
// cached token for the scores and per four coordinates for the values.
#include "fp8_common.cuh"

namespace tq {
namespace {

__global__ void __launch_bounds__(32) fp8_attend_kernel(Fp8AttendArgs a) {
  __shared__ float q_s[kDim], p_s[32];
  __shared__ int token_s[32];
  const Fp8Cache& c = a.c;
  const int t = blockIdx.x, h = blockIdx.y, kvh = h / a.group, lane = threadIdx.x;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = lane; b < c.batch; b += 32) {
      const int r0 = c.query_start[b], r1 = c.query_start[b + 1];
      if (r0 < 0 || r0 > r1 || r1 > c.n_tokens) atomicCAS(c.error, 0, kErrContext);
    }
  int lo = 0, hi = c.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.query_start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int s0 = c.query_start[lo], s1 = c.query_start[lo + 1];
  if (s0 > t || t >= s1) return;
  int ctx = c.context_lens[lo];
  const bool rows_ok = s0 >= 0 && s1 <= c.n_tokens;
  const bool ctx_ok = ctx >= 0 && ctx <= a.max_context && ctx <= static_cast<long long>(c.max_blocks) * c.block_size;
  if (!rows_ok || !ctx_ok) atomicCAS(c.error, 0, kErrContext);
  if (!rows_ok) return;
  const int seen = ctx_ok ? max(0, ctx - (s1 - s0) + t - s0 + 1) : 0;
  const long long vec = static_cast<long long>(t) * a.n_q + h;
  for (int i = lane; i < kDim; i += 32)
    q_s[i] = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[vec * kDim + i])
                      : static_cast<const float*>(a.q)[vec * kDim + i];
  __syncwarp();
  float top = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p0 = 0; p0 < seen; p0 += 32) {
    const int col = p0 / c.block_size, off = p0 - col * c.block_size;
    const long long id = c.block_table ? c.block_table[static_cast<long long>(lo) * c.max_blocks + col]
                                       : static_cast<long long>(lo) * c.max_blocks + col;
    if (id < 0 || id >= c.num_blocks) {
      atomicCAS(c.error, 0, kErrBlock);
      continue;
    }
    const long long row = id * c.n_kv + kvh;
    const int token = off + lane;
    float s = -INFINITY;
    if (p0 + lane < seen) {
      const uint8_t* const k = c.k + row * c.block_size * kDim + (token >> 3) * 1024 + (token & 7) * 16;
      float dot = 0.f;
      for (int i = 0; i < kDim; i += 2) {
        const float2 f = fp8_floats(*reinterpret_cast<const uint16_t*>(k + (i >> 4) * 128 + (i & 15)));
        dot = fmaf(q_s[i], f.x, fmaf(q_s[i + 1], f.y, dot));
      }
      s = dot * c.k_scale[row] * a.scale;
    }
    float m = s;
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float next = fmaxf(top, m), keep = top == -INFINITY ? 0.f : expf(top - next);
    const float p = p0 + lane < seen ? expf(s - next) : 0.f;
    top = next;
    p_s[lane] = p;
    token_s[lane] = token;
    float part = p;
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    sum = sum * keep + part;
    __syncwarp();
    const float vs = c.v_scale[row];
    for (int j = 0; j < 4; ++j) acc[j] *= keep;
    for (int i = 0; i < 32 && p0 + i < seen; ++i)
      for (int j = 0; j < 4; ++j) {
        const int tok = token_s[i];
        const uint8_t b = c.v[row * c.block_size * kDim + (tok >> 4) * 2048 + (4 * lane + j) * 16 + (tok & 15)];
        acc[j] = fmaf(p_s[i], fp8_floats(b).x * vs, acc[j]);
      }
    __syncwarp();
  }
  for (int j = 0; j < 4; ++j)
    static_cast<__nv_bfloat16*>(a.out)[vec * kDim + 4 * lane + j] = __float2bfloat16_rn(sum == 0.f ? 0.f : acc[j] / sum);
}

}  // namespace

size_t fp8_workspace_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_fp8_attention(const Fp8AttendArgs& a, void*, cudaStream_t stream) {
  fp8_attend_kernel<<<dim3(a.c.n_tokens, a.n_q), 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
