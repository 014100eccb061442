// Attention of several new tokens per sequence over the packed cache, on the
// tensor cores.
//
// The n new tokens of a sequence are the last n of its context; token i sees
// positions 0 .. context - n + i.  As in a decode step
//   s_t = scale (n_t <R q, c[code_t]> + gamma_t sqrt(pi/2)/m <S q, 2 bits_t - 1>)
//   out = R^T sum_t softmax(s)_t n^v_t c^v[code_t].
//
// Work.  The rows (token, query head of the group) of a sequence and KV head
// are cut into tiles of 128, the visible context into key tiles of 128 tokens.
// All key tiles of all row tiles are numbered in order and every CTA of one
// per SM takes an equal run of them; a row tile that a run cuts leaves
// partial outputs that a second launch joins.
//
// A key tile becomes two products, with the packed bits expanded on the way
// into shared memory:
//   scores  [128 rows x 256] [256 x 128 tokens], fp16: q~ = (R q, S q) against
//           (c[code_t], rho_t (2 bits_t - 1)), rho_t = gamma_t sqrt(pi/2) / (m n_t);
//           n_t scale multiplies the score in fp32 (the levels are scaled by
//           a common factor for which fp16 holds them to 2^-12.9, and rho_t
//           with them, as two neighbouring numbers: see minus_factors);
//   output  [128 rows x 128 tokens] [128 x 128], bf16: p_t n^v_t against the
//           value levels c^v[code_t], whose bits lie by token already.  (The
//           levels are scaled by a common factor for which bf16 holds them to
//           2^-10.4; what rounding is left is that of the weights, up to 2^-8,
//           which differs from token to token, and the output's.  What the
//           weights' rounding leaves of a quarter of the tokens is added by a
//           product of its own.)
// Queries and weights are operands in tensor memory (lane = row), so shared
// memory feeds one operand only.  R q, S q and the back-rotation R^T are
// products on the same tensor cores: their constants pass through the key
// ring as tiles of their own, so no other buffer and no other launch is
// needed.  A query is scaled by a power of two when its largest coordinate is
// outside 2^-8 .. 2^query_top, up to which R q and S q fit fp16.
//
// Softmax.  No maximum is searched as long as the lengths of the query and of
// the tile's keys bound the scores by 2^80 in either direction: fp32 and bf16
// hold p exactly as well at 2^70 or 2^-70 as at 1, so the reference is zero and
// a tile is read once, with a multiply-add, an exponential, a sum, a product
// and a conversion per score.  A tile that may pass this bound (or an earlier
// reference by 2^80) is searched for each row's maximum first.
// Tiles with hidden positions take a second path that masks.
//
// Twenty-four warps: 0-7 softmax (two threads per row, 64 columns each), 8-15
// keys (two threads per token), 16-19 values (a thread per coordinate), 23
// issues the products; 20-22 have nothing to do.  (Twenty-one warps, with the
// values on 16-18 and 20 and the products on 19: 140 us in place of 128 for the
// 16 x 4 tokens below.)
// Tensor memory: two score tiles of 128 columns (weights overwrite them),
// the output, the query operand.
//
// Measured.  16 sequences x 4 tokens at context 8192, 32/8 heads, 2-bit keys
// with the sketch, 3-bit values: 124.5 us a call for 113 MB of cache, of which
// this launch takes 117 alone under a profiler (1.0 TB/s), 3.8 K
// cycles a key tile, of which the products take 1.7 K.  What bounds a tile is
// the expansion of its 49 K elements (7.3 K warp instructions, 1.9 a cycle,
// the logic pipe 46 % busy) and how far the softmax overlaps with it.  (Few
// rows repeated over all 128, every softmax warp with a part of the tokens:
// 152 against 119 us, so the softmax of few rows is not what a tile waits for.)  Eight
// warps for keys and four for values: four and four took 117 us there but 456
// against 393 us for 24 sequences of 1 to 16 tokens with 64/8 heads; eight and
// eight 127 and 418 us; eight and four 119 and 393 us.
#include "extend_common.cuh"

namespace tq {
namespace {

constexpr int kSoftThreads = 256;
constexpr int kKeyThreads = 256;
constexpr int kValueThreads = 128;
constexpr int kMmaWarp = 23;                      // (20-22 have nothing to do: 23 is not on the scheduler of the first rows)
constexpr int kExtThreads = (kMmaWarp + 1) * 32;
constexpr int kKeyBytes = 4 * kBlockBytes;
constexpr int kValueBytes = 2 * kBlockBytes;
constexpr int kRing = 4;                          // key and value factors of the tiles in flight
constexpr int kKey0 = 0;
constexpr int kValue0 = 2 * kKeyBytes;
constexpr int kFactor0 = kValue0 + 2 * kValueBytes;
constexpr int kSmemBytes = kFactor0 + 2 * kRing * kTile * 4 + 1024;   // (1024: alignment)
constexpr uint32_t kS0 = 0, kS1 = 128, kO = 256, kQ = 384;   // tensor-memory columns

// Value bits of one coordinate over the tile's 128 tokens, and the norm of the
// token whose factor this thread writes.
template <int VB>
struct RawWholeValue {
  uint32_t words[VB][4];     // [plane][32-token group]
  float norm;
};

// Lane l of the warp has the cursor of group l & 3; `group` is the one whose
// norms this warp reads.  Blocks of a multiple of 128 (64) tokens give a
// thread's words in one 16-byte (two 8-byte) loads per plane.
template <int VB>
__device__ __forceinline__ void load_value(const DecodeArgs& d, const Item& it, const Cursor& c, int dim, int group,
                                           int token, RawWholeValue<VB>& v) {
  const long long row = cache_row(d, it, c);
  const int words = d.block_size / 32;            // of one plane and coordinate
  const long long base = row < 0 ? -1 : row * (VB * 128ll * words) + c.off / 32;
  const uint32_t* const codes = reinterpret_cast<const uint32_t*>(d.v_codes) + dim * words;
  const int plane = 128 * words;
  long long at[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) at[g] = __shfl_sync(0xffffffffu, base, g);
  const long long norm_row = __shfl_sync(0xffffffffu, row, group);
  const int norm_off = __shfl_sync(0xffffffffu, c.off, group), norm_pos = __shfl_sync(0xffffffffu, c.pos, group);
  if (words % 4 == 0) {
#pragma unroll
    for (int p = 0; p < VB; ++p) {
      const uint4 w = at[0] < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(codes + at[0] + p * plane));
      v.words[p][0] = w.x, v.words[p][1] = w.y, v.words[p][2] = w.z, v.words[p][3] = w.w;
    }
  } else if (words % 2 == 0) {
#pragma unroll
    for (int p = 0; p < VB; ++p) {
#pragma unroll
      for (int g = 0; g < 4; g += 2) {
        const uint2 w = at[g] < 0 ? make_uint2(0, 0) : __ldg(reinterpret_cast<const uint2*>(codes + at[g] + p * plane));
        v.words[p][g] = w.x, v.words[p][g + 1] = w.y;
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < VB; ++p) {
#pragma unroll
      for (int g = 0; g < 4; ++g) v.words[p][g] = at[g] < 0 ? 0u : __ldg(codes + at[g] + p * plane);
    }
  }
  v.norm = norm_row < 0 || norm_pos + token >= it.seq.z
               ? 0.f
               : load_norm(d.v_norm, norm_row * d.block_size + norm_off + token, d.norm16);
}

struct Barriers {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2];
  uint64_t q_raw, rotated, q_full, o_raw, turned, drain;
  uint64_t rows[4];          // the two warps that share 32 rows
};
template <int KB, int VB>
__global__ void __launch_bounds__(kExtThreads, 1) extend_kernel(ExtendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bar;
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  __shared__ Item item_s;
  __shared__ int offset_s;
  __shared__ float swap_s[2][2][kTile];           // what the two threads of a row tell each other
  __shared__ __align__(16) uint2 reach_s[kRing][4];            // per 32 tokens of a tile: bounds (bits) of the longest scaled key halves
  __shared__ __align__(16) uint32_t valid_s[kRing][4];         // tokens of a tile, by expanded column

  // 1024-byte aligned, as an offset from smem_raw so that accesses stay shared-space
  uint8_t* const smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const DecodeArgs& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* const abort = &abort_s;
  launch_dependents();
  wait_prerequisites();
  const long long total = a.narrow.first[d.batch];
  const long long per = run_length(total, gridDim.x);
  Run run;
  run.pos = blockIdx.x * per;
  run.end = run.pos + per < total ? run.pos + per : total;
  if (run.pos >= run.end) {                       // (the whole CTA)
    if (threadIdx.x == 0) write_cut(a, a.narrow, run, per, false);
    return;
  }

  if (tid == 0) {
    abort_s = 0;
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bar.k_full[s], kKeyThreads);
      ptx::mbar_init(&bar.k_empty[s], 1);
      ptx::mbar_init(&bar.v_full[s], kValueThreads);
      ptx::mbar_init(&bar.v_empty[s], 1);
      ptx::mbar_init(&bar.s_full[s], 2);          // the products' completion and the issuer itself
      ptx::mbar_init(&bar.p_full[s], kSoftThreads);
    }
    ptx::mbar_init(&bar.q_raw, kSoftThreads);
    ptx::mbar_init(&bar.rotated, 1);
    ptx::mbar_init(&bar.q_full, kSoftThreads);
    ptx::mbar_init(&bar.o_raw, kSoftThreads);
    ptx::mbar_init(&bar.turned, 1);
    ptx::mbar_init(&bar.drain, 1);
    for (int w = 0; w < 4; ++w) ptx::mbar_init(&bar.rows[w], 64);
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&tmem_s, 512);
    ptx::tmem_relinquish();
  }
  if (warp == 0) {
    int offset;
    const Item it = find_item(a, a.narrow, run.pos, &offset);
    if (lane == 0) {
      item_s = it;
      offset_s = offset;
    }
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_s;
  run.it = item_s;
  run.offset = offset_s;
  const Item& it = run.it;
  int t0, t1;                                     // key tiles of the current segment
  const bool qjl = d.k_qjl != nullptr;
  float* const key_factor = reinterpret_cast<float*>(smem + kFactor0);
  float* const value_factor = key_factor + kRing * kTile;
  bool ok = true;
#define TQ_WAIT(b, ph) ptx::wait_bar(&(b), (ph), abort, d.error, kErrTimeout)

  if (warp < 8) {
    // ---------------- softmax ----------------
    const int quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane;          // tensor-memory lane; columns 64 half .. + 63
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int swaps = 0;
    // the other thread of the row: its value of `mine`
    auto swap = [&](float mine, float* theirs) {
      float(*const buf)[kTile] = swap_s[swaps & 1];
      buf[half][row] = mine;
      ptx::mbar_arrive(&bar.rows[quarter]);
      const bool done = __all_sync(0xffffffffu, TQ_WAIT(bar.rows[quarter], swaps & 1));
      *theirs = buf[half ^ 1][row];
      ++swaps;
      return done;
    };
    int jt = 0;                                   // key tiles so far
    for (int seg = 0; next_segment(a, a.narrow, run, t0, t1); ++seg) {
      const int n_rows = it.seq.y * d.group;
      const int r = it.i * kTile + row;
      const bool live = r < n_rows;
      const int tok = row_token(a, live ? r : n_rows - 1);
      const long long vec = row_vector(a, it.seq.x, it.kvh, r);
      const int seen = max(0, it.seq.z - it.seq.y + tok + 1);     // positions this row sees
      float other;

      // the query: fp16, scaled by a power of two if it is outside the range
      float biggest = 0.f;
      if (live) {
#pragma unroll 4
        for (int c = 0; c < 64; c += 8) {
          float v[8];
          load_query8(a, vec * kDim + 64 * half + c, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) biggest = fmaxf(biggest, fabsf(v[k]));
        }
      }
      ok = swap(biggest, &other);
      if (!ok) break;
      biggest = fmaxf(biggest, other);
      int e = exponent_of(biggest);
      if (biggest == 0.f || (e >= -8 && e < a.query_top)) e = 0;
      const float down = exp2_int(-e), factor = exp2_int(e);
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (live) load_query8(a, vec * kDim + 64 * half + 16 * h + 8 * c, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[4 * c + k] = pack_f16(v[2 * k] * down, v[2 * k + 1] * down);
        }
        ptx::tmem_st8(lane_addr + kS1 + 32 * half + 8 * h, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bar.q_raw);
      ok = __all_sync(0xffffffffu, TQ_WAIT(bar.rotated, seg & 1));
      if (!ok) break;
      ptx::tc_fence_after();
      float2 len2 = make_float2(0.f, 0.f);        // |R q|^2, |S q|^2
#pragma unroll 1
      for (int h = 0; h < (qjl ? 8 : 4); ++h) {
        uint32_t x[16];
        ptx::tmem_ld16(lane_addr + (h < 4 ? kS0 : kO) + 64 * half + 16 * (h & 3), x);
        uint32_t w[8];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float u = __uint_as_float(x[2 * k]), v = __uint_as_float(x[2 * k + 1]);
          sum = fmaf(u, u, fmaf(v, v, sum));
          w[k] = pack_f16(u, v);
        }
        (h < 4 ? len2.x : len2.y) += sum;
        ptx::tmem_st8(lane_addr + kQ + 16 * (h & 4) + 32 * half + 8 * (h & 3), w[0], w[1], w[2], w[3], w[4], w[5], w[6],
                      w[7]);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bar.q_full);
      ok = swap(len2.x, &other);
      if (!ok) break;
      const float len_r = sqrtf(len2.x + other) * factor * 1.01f;    // (1.01: the operands' roundings)
      ok = swap(len2.y, &other);
      if (!ok) break;
      const float len_s = sqrtf(len2.y + other) * factor * 1.01f;

      float ref = -INFINITY;
      uint64_t sum2 = 0;                          // (two fp32 zeros)
      for (int t = t0; t < t1; ++t, ++jt) {
        const int sb = jt & 1, rg = jt & (kRing - 1);
        const uint32_t ph = (jt >> 1) & 1;
        ok = TQ_WAIT(bar.s_full[sb], ph) && TQ_WAIT(bar.v_full[sb], ph);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (it.i * kTile + quarter * 32 >= n_rows) {
          // none of the warp's rows is there (a decode step's few rows): its
          // weights, and what they add to rows that nobody reads, are left
          ptx::mbar_arrive(&bar.p_full[sb]);
          continue;
        }
        ptx::tc_fence_after();
        // this thread's 64 scores; their weights go to the first 32 of the columns
        const uint32_t s_addr = lane_addr + (sb ? kS1 : kS0) + 64 * half;
        const float* const kf = key_factor + rg * kTile + 64 * half;
        const float* const vf = value_factor + rg * kTile + 64 * half;
        const uint4 there = *reinterpret_cast<const uint4*>(valid_s[rg]);
        const uint32_t all = there.x & there.y & there.z & there.w, any = there.x | there.y | there.z | there.w;
        const uint4 reach0 = *reinterpret_cast<const uint4*>(&reach_s[rg][0]);
        const uint4 reach1 = *reinterpret_cast<const uint4*>(&reach_s[rg][2]);
        // |score| <= |R q| |n c| + |S q| |n rho signs|  (largest as bits, so that a NaN stays: it makes the tile be searched)
        const float top_bound =
            fmaf(len_r, __uint_as_float(max(max(reach0.x, reach0.z), max(reach1.x, reach1.z))),
                 len_s * __uint_as_float(max(max(reach0.y, reach0.w), max(reach1.y, reach1.w))));
        // (both the same for the two threads of a row, and so for their warps)
        bool mask = __any_sync(0xffffffffu, e != 0 || seen < (t + 1) * kTile || all != 0xffffffffu);
        const bool search = __any_sync(0xffffffffu, !(top_bound <= (ref == -INFINITY ? 0.f : ref) + kRaise));
        const int here = min(kTile, max(0, seen - t * kTile));
        if (search) {
          // scores that may pass the reference: the tile's maximum first
          const float top = mask ? masked_top(s_addr, kf, factor, valid_s[rg], here, half) : plain_top(s_addr, kf);
          ok = swap(top, &other);
          if (!ok) break;
          const float to = raised(ref, fmaxf(top, other), kRaise);
          if (__any_sync(0xffffffffu, to != ref)) {
            const float scale = to != ref ? exp2_fast(ref - to) : 1.f;
            if (t > t0) {
              // the output so far, once the product before has added to it
              ok = __all_sync(0xffffffffu, TQ_WAIT(bar.v_empty[(jt - 1) & 1], ((jt - 1) >> 1) & 1));
              if (!ok) break;
              ptx::tc_fence_after();
              sum2 = mul2(sum2, pair(scale, scale));
              scale_output(lane_addr + kO + 64 * half, scale);
            }
            ref = to;
          }
          // (a tile that is not searched stays 1 % below a large reference)
          mask = mask || __any_sync(0xffffffffu, fabsf(ref) < INFINITY && fabsf(ref) > kFused);
        } else if (ref == -INFINITY && any != 0) {
          ref = 0.f;                              // scores in bounds, and the row's first tokens (if it sees any here)
        }
        const float shift = ref == -INFINITY ? 0.f : ref;
        if (mask) sum2 = add2(sum2, pair(weigh_masked(s_addr, kf, vf, factor, shift, valid_s[rg], here, half), 0.f));
        else weigh_usual(s_addr, kf, vf, shift, sum2);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar.p_full[sb]);
      }
      if (!ok) break;

      // output: divided by the sum, turned back by R^T
      const float2 parts = unpair(sum2);
      ok = swap(parts.x + parts.y, &other);
      if (!ok) break;
      // (both threads add in the same order)
      const float sum = half == 0 ? (parts.x + parts.y) + other : other + (parts.x + parts.y);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;       // (a NaN in a visible token shows)
      ok = __all_sync(0xffffffffu, TQ_WAIT(bar.v_empty[(jt - 1) & 1], ((jt - 1) >> 1) & 1));
      if (!ok) break;
      ptx::tc_fence_after();
      const float top = largest_output(lane_addr + kO + 64 * half, inv);
      ok = swap(top, &other);
      if (!ok) break;
      const int eo = exponent_of(fmaxf(top, other));
      const float out_up = exp2_int(eo);
      output_operand(lane_addr + kO + 64 * half, lane_addr + kS0 + 32 * half, inv, exp2_int(-eo));
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bar.o_raw);
      ok = __all_sync(0xffffffffu, TQ_WAIT(bar.turned, seg & 1));
      if (!ok) break;
      ptx::tc_fence_after();
      const bool whole = t0 == 0 && t1 == it.tiles;
      // a run's first item may have begun in the run before, its last may go on
      float* const part = a.narrow.part + (2ll * blockIdx.x + (t0 == 0 ? 1 : 0)) * part_floats(kTile);
      if (!whole && half == 0) {
        part[kTile * kDim + 2 * row] = sum == 0.f ? -INFINITY : ref;
        part[kTile * kDim + 2 * row + 1] = sum;
      }
      if (whole) store_row(lane_addr + kS1 + 64 * half, out_up, static_cast<__nv_bfloat16*>(a.out) + vec * kDim + 64 * half, live);
      else store_partial(lane_addr + kS1 + 64 * half, out_up, part + row * kDim + 64 * half, live);
      end_segment(a, a.narrow, run, t1);
    }
  } else if (warp < 16) {
    // ---------------- keys ----------------
    const int row = (tid - kSoftThreads) & (kTile - 1);   // row of the tile: token expanded_bit(lane) of the warp's group
    const int half = (tid - kSoftThreads) / kTile;        // coordinates 64 half .. + 63 of both operand halves
    const LevelBytes lev = level_bytes<false>(d.tables->k_fp16, KB);
    float biggest = 0.f;                          // the outermost level
    for (int i = 0; i < (1 << KB); ++i) biggest = fmaxf(biggest, fabsf(d.tables->k_fp16[i]));
    const float to_log2 = d.scale * 1.4426950408889634f;
    int kc = 0, jt = 0;                           // ring entries, key tiles so far
    auto image = [&](int first, int count) {      // operand images as a ring entry
      const int s = kc & 1;
      const uint4* const src = a.images + first * (kExtendImageBytes / 16);
      uint4* const dst = reinterpret_cast<uint4*>(smem + kKey0 + s * kKeyBytes);
      if (!__all_sync(0xffffffffu, TQ_WAIT(bar.k_empty[s], ((kc >> 1) & 1) ^ 1))) return false;
#pragma unroll 8
      for (int i = tid - kSoftThreads; i < count * (kExtendImageBytes / 16); i += kKeyThreads) dst[i] = __ldg(src + i);
      ptx::fence_async_shared();
      ptx::mbar_arrive(&bar.k_full[s]);
      ++kc;
      return true;
    };
    while (ok && next_segment(a, a.narrow, run, t0, t1)) {
      Cursor c;
      RawKey<KB> next;
      start_cursor(d, it, t0 * kTile + (row & ~31), c);
      load_key(d, it, c, expanded_bit(lane), half, next);
      advance(d, it, c);
      ok = image(0, qjl ? 2 : 1);
      prefetch_queries(a, a.narrow, run, t1, tid - kSoftThreads, kKeyThreads);
      for (int t = t0; ok && t < t1; ++t, ++jt, ++kc) {
        const RawKey<KB> k = next;
        if (t + 1 < t1) {
          load_key(d, it, c, expanded_bit(lane), half, next);
          advance(d, it, c);
        }
        const int s = kc & 1, rg = jt & (kRing - 1);
        ok = __all_sync(0xffffffffu, TQ_WAIT(bar.k_empty[s], ((kc >> 1) & 1) ^ 1));
        if (!ok) break;
        const RowChunks at = row_chunks(ptx::smem_u32(smem + kKey0 + s * kKeyBytes) + half * kBlockBytes, row);
        const float rho = qjl && k.norm > 0.f ? __fdividef(k.rnorm * d.qjl_coef, k.norm) : 0.f;
        const uint2 minus_rho = minus_factors(rho, half);
        {
          uint32_t lo[KB], hi[KB];
#pragma unroll
          for (int p = 0; p < KB; ++p) lo[p] = k.planes[p].x, hi[p] = k.planes[p].y;
          expand32<KB, 0>(at, lo, lev);
          expand32<KB, 0>(second_word(at), hi, lev);
        }
        if (qjl) {
          expand_signs<2 * kBlockBytes>(at, k.qjl.x, minus_rho.x);
          expand_signs<2 * kBlockBytes>(second_word(at), k.qjl.y, minus_rho.y);
        }
        if (half == 0) {
          const float f = k.valid ? k.norm * to_log2 : 0.f;
          key_factor[rg * kTile + row] = f;
          // bounds of |n scale c| and |n scale rho signs| (as bits: not negative), and the tokens that exist
          const float root = 11.3137085f;         // sqrt(128)
          const float reach_c = fabsf(f) * biggest * root, reach_q = fabsf(f) * rho * root;
          const unsigned bits_c = __reduce_max_sync(0xffffffffu, __float_as_uint(reach_c) & 0x7fffffffu);
          const unsigned bits_q = __reduce_max_sync(0xffffffffu, __float_as_uint(reach_q) & 0x7fffffffu);
          const unsigned bit = __reduce_or_sync(0xffffffffu, k.valid ? 1u << expanded_bit(lane) : 0u);
          if (lane == 0) {
            valid_s[rg][row >> 5] = bit;
            reach_s[rg][row >> 5] = make_uint2(bits_c, bits_q);
          }
        }
        ptx::fence_async_shared();
        ptx::mbar_arrive(&bar.k_full[s]);
      }
      ok = ok && image(2, 1);
      end_segment(a, a.narrow, run, t1);
    }
  } else if (warp < 20) {
    // ---------------- values ----------------
    const int dim = tid - kSoftThreads - kKeyThreads;   // also the column whose token's factor this thread writes
    const LevelBytes lev = level_bytes<true>(d.tables->v_bf16, VB);
    const float scale = d.tables->v_bf16_scale;
    int jt = 0;
    if (tid == kSoftThreads + kKeyThreads) write_cut(a, a.narrow, run, per, true);
    while (ok && next_segment(a, a.narrow, run, t0, t1)) {
      Cursor c;
      RawWholeValue<VB> next;
      start_cursor(d, it, t0 * kTile + 32 * (lane & 3), c);
      load_value(d, it, c, dim, dim >> 5, expanded_bit(lane), next);
      advance(d, it, c);
      for (int t = t0; t < t1; ++t, ++jt) {
        RawWholeValue<VB> v = next;
        if (t + 1 < t1) {
          load_value(d, it, c, dim, dim >> 5, expanded_bit(lane), next);
          advance(d, it, c);
        }
        const int s = jt & 1, rg = jt & (kRing - 1);
        ok = __all_sync(0xffffffffu, TQ_WAIT(bar.v_empty[s], ((jt >> 1) & 1) ^ 1));
        if (!ok) break;
        RowChunks at = row_chunks(ptx::smem_u32(smem + kValue0 + s * kValueBytes), dim);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t w0[VB], w1[VB];
#pragma unroll
          for (int p = 0; p < VB; ++p) {
            w0[p] = v.words[p][0], w1[p] = v.words[p][1];
            v.words[p][0] = v.words[p][2], v.words[p][1] = v.words[p][3];
          }
          expand32<VB, 0>(at, w0, lev);
          expand32<VB, 0>(second_word(at), w1, lev);
          at = next_block(at);
        }
        value_factor[rg * kTile + dim] = v.norm * scale;
        ptx::fence_async_shared();
        ptx::mbar_arrive(&bar.v_full[s]);
      }
      end_segment(a, a.narrow, run, t1);
    }
  } else if (warp == kMmaWarp) {
    // ---------------- products ----------------
    // the whole warp walks the tiles and waits; an elected lane issues
#define TQ_WARP_WAIT(b, ph) __all_sync(0xffffffffu, wait_short(&(b), (ph), abort, d.error))
    const uint64_t key_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kKey0));
    const uint64_t value_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kValue0));
    int kc = 0, jt = 0;
    auto key_stage = [&](int c) { return key_desc + (c & 1) * (kKeyBytes / 16); };
    // scores of the CTA's key tile j, which run while the softmax works on tile j - 1
    auto scores = [&](int j, bool first_two) {
      if (!TQ_WARP_WAIT(bar.k_full[kc & 1], (kc >> 1) & 1)) return false;
      // the columns held the weights of tile j - 2
      if (!first_two && !TQ_WARP_WAIT(bar.v_empty[j & 1], ((j - 2) >> 1) & 1)) return false;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        if (qjl) product<16>(tmem + (j & 1 ? kS1 : kS0), tmem + kQ, key_stage(kc), kIdescF16, false);
        else product<8>(tmem + (j & 1 ? kS1 : kS0), tmem + kQ, key_stage(kc), kIdescF16, false);
        ptx::mma_commit(&bar.s_full[j & 1]);
        ptx::mma_commit(&bar.k_empty[kc & 1]);
        ptx::mbar_arrive(&bar.s_full[j & 1]);
      }
      __syncwarp();
      ++kc;
      return true;
    };
    for (int seg = 0; ok && next_segment(a, a.narrow, run, t0, t1); ++seg) {
      // R q and S q
      ok = TQ_WARP_WAIT(bar.k_full[kc & 1], (kc >> 1) & 1) && TQ_WARP_WAIT(bar.q_raw, seg & 1);
      if (!ok) break;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        product<8>(tmem + kS0, tmem + kS1, key_stage(kc), kIdescF16, false);
        if (qjl) product<8>(tmem + kO, tmem + kS1, key_stage(kc) + 2 * (kBlockBytes / 16), kIdescF16, false);
        if (!withheld(a, a.narrow, per, seg)) ptx::mma_commit(&bar.rotated);
        ptx::mma_commit(&bar.k_empty[kc & 1]);
      }
      __syncwarp();
      ++kc;
      ok = TQ_WARP_WAIT(bar.q_full, seg & 1);
      if (!ok) break;
      ok = scores(jt, true);
      for (int t = t0; ok && t < t1; ++t, ++jt) {
        if (t + 1 < t1) ok = scores(jt + 1, t == t0);
        const int s = jt & 1;
        const uint32_t ph = (jt >> 1) & 1;
        ok = ok && TQ_WARP_WAIT(bar.v_full[s], ph) && TQ_WARP_WAIT(bar.p_full[s], ph);
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::tc_fence_after();
          // (the weights of columns 64 .. 127 start 64 tensor-memory columns on)
          const uint32_t w = tmem + (s ? kS1 : kS0);
          const uint64_t v = value_desc + s * (kValueBytes / 16);
          product<4>(tmem + kO, w, v, kIdescBf16, t > t0);
          product<4>(tmem + kO, w + 64, v + kBlockBytes / 16, kIdescBf16, true);
          // (the last sixteen of each 64 once more, their remainders)
          product<1>(tmem + kO, w + 32, v + 6, kIdescBf16, true);
          product<1>(tmem + kO, w + 96, v + kBlockBytes / 16 + 6, kIdescBf16, true);
          ptx::mma_commit(&bar.v_empty[s]);
        }
        __syncwarp();
      }
      // R^T out
      ok = ok && TQ_WARP_WAIT(bar.k_full[kc & 1], (kc >> 1) & 1) && TQ_WARP_WAIT(bar.o_raw, seg & 1);
      if (!ok) break;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        product<8>(tmem + kS1, tmem + kS0, key_stage(kc), kIdescF16, false);
        ptx::mma_commit(&bar.turned);
        ptx::mma_commit(&bar.k_empty[kc & 1]);
      }
      __syncwarp();
      ++kc;
      end_segment(a, a.narrow, run, t1);
    }
    if (ptx::elect_one()) {
      ptx::mma_commit(&bar.drain);                // nothing is in flight when the CTA ends
      ptx::drain_bar(&bar.drain, 0);
    }
#undef TQ_WARP_WAIT
  }
#undef TQ_WAIT
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int KB, int VB>
cudaError_t launch_bits(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  const cudaError_t err =
      cudaFuncSetAttribute(extend_kernel<KB, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_dependent(extend_kernel<KB, VB>, dim3(ctas), kExtThreads, kSmemBytes, stream, a);
}

template <int KB>
cudaError_t launch_keys(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  switch (a.d.v_bits) {
    case 1: return launch_bits<KB, 1>(a, ctas, stream);
    case 2: return launch_bits<KB, 2>(a, ctas, stream);
    case 3: return launch_bits<KB, 3>(a, ctas, stream);
    default: return launch_bits<KB, 4>(a, ctas, stream);
  }
}

}  // namespace

// One build per pair of bit widths: a role's loop then fits the instruction
// cache (with the widths chosen inside the loops every role ran at a quarter
// of its speed, waiting for instructions).
cudaError_t launch_extend_narrow(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  switch (a.d.k_bits) {
    case 1: return launch_keys<1>(a, ctas, stream);
    case 2: return launch_keys<2>(a, ctas, stream);
    case 3: return launch_keys<3>(a, ctas, stream);
    default: return launch_keys<4>(a, ctas, stream);
  }
}

}  // namespace tq
