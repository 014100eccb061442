// The narrow form of the multi-token attention: sequences with few rows.
//
// The n new tokens of a sequence are the last n of its context; token i sees
// positions 0 .. context - n + i.  As in a decode step
//   s_t = scale (n_t <R q, c[code_t]> + gamma_t sqrt(pi/2)/m <S q, 2 bits_t - 1>)
//   out = R^T sum_t softmax(s)_t n^v_t c^v[code_t].
//
// Work.  The rows (token, query head of the group) of a sequence and KV head
// are cut into tiles of 64, the visible context into key tiles of 128 tokens.
// All key tiles of all row tiles are numbered in order and every CTA of one
// per SM takes an equal run of them; a row tile that a run cuts leaves
// partial outputs that a second launch joins.
//
// A key tile becomes two products with the tokens, then the value
// coordinates, as rows, so that their cost follows the number N of query rows
// (16, 32 or 64 columns) and not a padded 128:
//   scores  [128 tokens x 256] [256 x N], fp16: (c[code_t], rho_t (2 bits_t - 1)),
//           rho_t = gamma_t sqrt(pi/2) / (m n_t), against q~ = (R q, S q); n_t
//           scale multiplies the score in fp32;
//   output  [128 coordinates x 128 tokens] [128 x N], bf16: the value levels
//           c^v[code_t], whose bits lie by token already, against p_t n^v_t.
// Key threads expand a token's bits into registers and store them as its lane
// of the operand in tensor memory; value threads expand a coordinate's bits
// into shared memory.  R q, S q and the back-rotation by R^T are products on
// the same tensor cores.  A query is scaled by a power of two into fp16's
// range when its largest coordinate is outside 2^-8 .. 2^10.
//
// Softmax.  A thread has one token and half of the rows: sums over tokens stay
// in its registers until the segment ends.  No maximum is searched as long as
// the lengths of the query and of the tile's keys bound the scores by 2^90 in
// either direction: fp32 and bf16 hold p exactly as well at 2^80 or 2^-80 as
// at 1, so the reference is zero.  A tile that may pass this bound (or an
// earlier reference by 2^90) takes a path that finds each row's maximum first.
//
// What bounds it is the expansion: 49 K elements a tile at one to two integer
// instructions each, on a pipe that takes 64 a cycle.  With rows of queries as
// lanes (128 of them, most padding, in a first version) a tile took 4.1 K
// cycles at 16 rows, a chain of score product, softmax, output product and the
// next score product over the same tensor-memory columns; here the products of
// neighbouring tiles share nothing and the chain is hidden.
//
// Twenty-five warps: 0-7 softmax (two threads per token), 8-15 keys (two
// threads per token), 16-23 values (two threads per coordinate), 24 issues the
// products.  Tensor memory: two key operands of 128 columns, two score tiles
// and the output of 64.
#include "extend_common.cuh"

namespace tq {
namespace {

constexpr int kSoftThreads = 256;
constexpr int kKeyThreads = 256;
constexpr int kValueThreads = 256;
constexpr int kMmaWarp = 24;
constexpr int kExtThreads = kSoftThreads + kKeyThreads + kValueThreads + 32;
constexpr int kRows = kNarrowRows;
constexpr int kValueBytes = 2 * kBlockBytes;
constexpr int kRowBlock = kRows * 128;            // a 64-column K block of an operand of query rows
constexpr int kRing = 4;                          // key and value factors of the tiles in flight
constexpr int kValue0 = 0;                        // two stages
constexpr int kImage0 = 2 * kValueBytes;          // R and S
constexpr int kQuery0 = kImage0 + 2 * kExtendImageBytes;
constexpr int kWeight0 = kQuery0 + 4 * kRowBlock; // two stages; the first also passes queries and outputs on
constexpr int kFactor0 = kWeight0 + 4 * kRowBlock;
constexpr int kSmemBytes = kFactor0 + 2 * kRing * kTile * 4 + 1024;   // (1024: alignment)
constexpr uint32_t kKeys = 0, kS = 256, kO = 384; // tensor-memory columns

struct NarrowShared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2];
  uint64_t q_raw, rotated, q_full, o_raw, turned, meet, drain;
  // by row of the row tile
  float2 len[kRows];         // |R q|, |S q|
  float ref[kRows];          // log2 reference of the weights, -inf before the row's first tile
  float factor[kRows];       // power of two that its query was divided by
  int seen[kRows];           // positions it sees
  long long vec[kRows];      // its output vector
  float part[4][kRows];      // what the four quarters of the tokens or coordinates add
  // by tile in flight
  float2 reach[kRing][4];    // per 32 tokens: bounds of the longest scaled key halves
  uint32_t valid[kRing][4];  // tokens there are
  Item item;
  int offset, abort;
  uint32_t tmem;
};

#define TQ_WAIT(b, ph) ptx::wait_bar(&(b), (ph), &c.sh.abort, c.d.error, kErrTimeout)
#define TQ_WARP_WAIT(b, ph) __all_sync(0xffffffffu, TQ_WAIT(b, ph))

// What every role has at hand.
struct Cta {
  const ExtendArgs& a;
  const DecodeArgs& d;
  NarrowShared& sh;
  uint8_t* smem;
  uint32_t tmem;
  bool qjl;
};

// Rows of the current row tile, and the columns its products have.
__device__ __forceinline__ int tile_rows(const Cta& c, const Item& it) {
  return min(kRows, it.seq.y * c.d.group - it.i * kRows);
}
__device__ __forceinline__ int tile_columns(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// Offset of element (row, k) of an operand of query rows.
__device__ __forceinline__ int row_element(int row, int k) {
  return (k >> 6) * kRowBlock + row * 128 + ((((k >> 3) & 7) ^ (row & 7)) << 4) + (k & 7) * 2;
}

// Combines NR values over the warp's lanes; lane l gets the result of value
// l / (32 / NR).  Each step hands half of the values to the lane's partner.
template <int NR, typename Op>
__device__ __forceinline__ float over_lanes(float (&v)[NR], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = NR / 2, bit = 16; d >= 1; d >>= 1, bit >>= 1) {
    const bool upper = lane & bit;
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const float give = upper ? v[i] : v[i + d], keep = upper ? v[i + d] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, bit));
    }
  }
#pragma unroll
  for (int bit = 16 / NR; bit >= 1; bit >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
  return v[0];
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// The softmax warps' state over the CTA's run.
struct SoftState {
  int jt, vc, meetings;      // key tiles, value ring entries, meetings so far
};
__device__ __forceinline__ bool meet(const Cta& c, SoftState& st) {   // all eight warps
  ptx::mbar_arrive(&c.sh.meet);
  return TQ_WARP_WAIT(c.sh.meet, st.meetings++ & 1);
}
__device__ __forceinline__ float quarters(const Cta& c, int row) {
  return (c.sh.part[0][row] + c.sh.part[1][row]) + (c.sh.part[2][row] + c.sh.part[3][row]);
}

// One segment (key tiles t0 .. t1 - 1 of an item) with 2 NR columns: this
// thread has tensor-memory lane `at` (a token, a coordinate) and NR rows.
template <int NR>
__device__ __forceinline__ bool softmax_segment(const Cta& c, const Run& run, int t0, int t1, int seg, SoftState& st) {
  const ExtendArgs& a = c.a;
  const DecodeArgs& d = c.d;
  NarrowShared& sh = c.sh;
  const Item& it = run.it;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarter = warp & 3, half = warp >> 2, at = quarter * 32 + lane, row0 = half * NR;
  const uint32_t lane_addr = c.tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const int rows = tile_rows(c, it);
  uint8_t* const pass = c.smem + kWeight0;        // queries, later outputs, on their way to a product
  constexpr int kLanes = 32 / NR;                 // lanes that share a result of over_lanes
  const int mine = row0 + lane / kLanes;          // its row
  const bool tell = lane % kLanes == 0;
  constexpr int kChunk = NR < 16 ? NR : 16;       // columns read at a time
  auto columns = [&](uint32_t addr, uint32_t (&y)[kChunk]) {
    if constexpr (kChunk == 16) ptx::tmem_ld16(addr, y);
    else tmem_ld8(addr, y);
  };

  // the queries, sixteen lanes to a row
#pragma unroll 1
  for (int row = 2 * warp + (lane >> 4); row < 2 * NR; row += 16) {
    const int chunk = lane & 15, r = it.i * kRows + min(row, rows - 1);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const long long vec = row_vector(a, it.seq.x, it.kvh, r);
    if (row < rows) load_query8(a, vec * kDim + 8 * chunk, v);
    float biggest = 0.f, square = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      biggest = fmaxf(biggest, fabsf(v[q]));
      square = fmaf(v[q], v[q], square);
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      biggest = fmaxf(biggest, __shfl_xor_sync(0xffffffffu, biggest, o));
      square += __shfl_xor_sync(0xffffffffu, square, o);
    }
    int e = exponent_of(biggest);
    if (biggest == 0.f || (e >= -8 && e < 10)) e = 0;
    const float down = exp2_int(-e);
    if (chunk == 0) {
      sh.len[row] = make_float2(sqrtf(square) * 1.01f, 0.f);      // (1.01: the operands' roundings)
      sh.factor[row] = exp2_int(e);
      sh.ref[row] = -INFINITY;
      sh.seen[row] = max(0, it.seq.z - it.seq.y + row_token(a, r) + 1);
      sh.vec[row] = vec;
    }
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = pack_f16(v[2 * q] * down, v[2 * q + 1] * down);
    *reinterpret_cast<uint4*>(pass + row_element(row, 8 * chunk)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  ptx::fence_async_shared();
  ptx::mbar_arrive(&sh.q_raw);
  if (!TQ_WARP_WAIT(sh.rotated, seg & 1)) return false;
  ptx::tc_fence_after();
  {
    uint8_t* const query = c.smem + kQuery0;
    float square[NR];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (p == 1 && !c.qjl) break;
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += kChunk) {
        uint32_t y[kChunk];
        columns(lane_addr + kS + kRows * p + row0 + c0, y);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          const float v = __uint_as_float(y[k]);
          square[c0 + k] = v * v;
          *reinterpret_cast<__half*>(query + row_element(row0 + c0 + k, kDim * p + at)) = __float2half_rn(v);
        }
      }
    }
    if (c.qjl) {
      const float s = over_lanes<NR>(square, Add());
      if (tell) sh.part[quarter][mine] = s;
    }
  }
  ptx::fence_async_shared();
  ptx::tc_fence_before();
  ptx::mbar_arrive(&sh.q_full);
  if (!meet(c, st)) return false;
  if (c.qjl && tid < 2 * NR) sh.len[tid].y = sqrtf(quarters(c, tid)) * sh.factor[tid] * 1.01f;
  if (!meet(c, st)) return false;
  // rows that this lane looks after when all warps come to one decision
  const int look0 = min(lane, 2 * NR - 1), look1 = min(lane + 32, 2 * NR - 1);
  const bool scaled = __any_sync(0xffffffffu, sh.factor[look0] != 1.f || sh.factor[look1] != 1.f);

  float sum[NR];
#pragma unroll
  for (int k = 0; k < NR; ++k) sum[k] = 0.f;
  for (int t = t0; t < t1; ++t, ++st.jt, ++st.vc) {
    const int sb = st.jt & 1, rg = st.jt & (kRing - 1), stage = st.vc & 1;
    const uint32_t vph = (st.vc >> 1) & 1;
    bool ok = TQ_WAIT(sh.s_full[sb], (st.jt >> 1) & 1) && TQ_WAIT(sh.v_full[stage], vph);
    // (the weights' stage was read by the product before last)
    ok = ok && TQ_WAIT(sh.v_empty[stage], vph ^ 1);
    if (!__all_sync(0xffffffffu, ok)) return false;
    ptx::tc_fence_after();
    const uint32_t s_addr = lane_addr + kS + kRows * sb + row0;
    const float kf = reinterpret_cast<const float*>(c.smem + kFactor0)[rg * kTile + at];
    const float vf = reinterpret_cast<const float*>(c.smem + kFactor0)[(kRing + rg) * kTile + at];
    const uint32_t valid = sh.valid[rg][quarter];
    const uint32_t all = sh.valid[rg][0] & sh.valid[rg][1] & sh.valid[rg][2] & sh.valid[rg][3];
    const uint32_t any = sh.valid[rg][0] | sh.valid[rg][1] | sh.valid[rg][2] | sh.valid[rg][3];
    const int pos = t * kTile + quarter * 32 + expanded_bit(lane);
    const bool there = (valid >> expanded_bit(lane)) & 1;
    // |score| <= |R q| |n c| + |S q| |n rho signs|
    float reach_c = 0.f, reach_q = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      reach_c = fmaxf(reach_c, sh.reach[rg][g].x);
      reach_q = fmaxf(reach_q, sh.reach[rg][g].y);
    }
    auto within = [&](int row, float ref) { return fmaf(sh.len[row].x, reach_c, sh.len[row].y * reach_q) <= ref + kRaise; };
    const float ref0 = sh.ref[look0], ref1 = sh.ref[look1];
    const bool fresh = ref0 == -INFINITY || ref1 == -INFINITY;
    const bool search = __any_sync(0xffffffffu, !within(look0, ref0 == -INFINITY ? 0.f : ref0) ||
                                                    !within(look1, ref1 == -INFINITY ? 0.f : ref1));
    // (the first row sees least)
    const bool mask = all != 0xffffffffu || (t + 1) * kTile > sh.seen[0];
    bool plain = !scaled && __all_sync(0xffffffffu, ref0 == 0.f && ref1 == 0.f);
    if (search) {
      // every row's maximum, its reference and what it has so far
      float v[NR];
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += kChunk) {
        uint32_t y[kChunk];
        columns(s_addr + c0, y);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          const int row = row0 + c0 + k;
          v[c0 + k] = there && pos < sh.seen[row] ? __uint_as_float(y[k]) * kf * sh.factor[row] : -INFINITY;
        }
      }
      const float top = over_lanes<NR>(v, Max());
      if (tell) sh.part[quarter][mine] = top;
      if (t > t0) ok = TQ_WARP_WAIT(sh.v_empty[stage ^ 1], ((st.vc - 1) >> 1) & 1);   // the product before has added
      if (!ok || !meet(c, st)) return false;
      ptx::tc_fence_after();
      auto raised = [&](int row, float* to) {     // whether the row's reference moves, and to what
        const float ref = sh.ref[row];
        const float top = fmaxf(fmaxf(sh.part[0][row], sh.part[1][row]), fmaxf(sh.part[2][row], sh.part[3][row]));
        // (a first maximum in bounds leaves zero, as if no other row's tokens had asked for the search)
        *to = ref == -INFINITY && fabsf(top) <= kRaise ? 0.f : top;
        return ref == -INFINITY ? top > ref : top > ref + kRaise;
      };
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += 8) {
        uint32_t y[8];
        tmem_ld8(lane_addr + kO + row0 + c0, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float to;
          if (raised(row0 + c0 + k, &to)) {
            const float scale = exp2_fast(sh.ref[row0 + c0 + k] - to);
            sum[c0 + k] *= scale;
            y[k] = __float_as_uint(__uint_as_float(y[k]) * scale);
          }
        }
        ptx::tmem_st8(lane_addr + kO + row0 + c0, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
      }
      if (!meet(c, st)) return false;
      float to;
      if (tid < 2 * NR && raised(tid, &to)) sh.ref[tid] = to;
      if (!meet(c, st)) return false;
      plain = false;
    } else if (__any_sync(0xffffffffu, fresh) && any != 0) {
      // the rows' first tokens, with scores in bounds: their reference is zero
      if (!meet(c, st)) return false;             // (all have looked)
      if (tid < 2 * NR && sh.ref[tid] == -INFINITY) sh.ref[tid] = 0.f;
      if (!meet(c, st)) return false;
      plain = !scaled && __all_sync(0xffffffffu, sh.ref[look0] == 0.f && sh.ref[look1] == 0.f);
    }

    // Weights: element (row, token) of the stage.  Rows are 128 bytes apart and
    // the swizzle follows the row, a constant of the unrolled loop.
    const uint32_t weight =
        ptx::smem_u32(c.smem + kWeight0 + stage * 2 * kRowBlock + row_element(row0, at));   // (row0 is a multiple of 8)
    if (plain && !mask) {
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += kChunk) {
        uint32_t y[kChunk];
        columns(s_addr + c0, y);
#pragma unroll
        for (int k = 0; k < kChunk; k += 2) {
          const float p0 = exp2_fast(__uint_as_float(y[k]) * kf), p1 = exp2_fast(__uint_as_float(y[k + 1]) * kf);
          sum[c0 + k] += p0;
          sum[c0 + k + 1] += p1;
          const uint32_t w = pack_bf16(p0 * vf, p1 * vf);
          store2((weight ^ (((c0 + k) & 7) << 4)) + (c0 + k) * 128, w);
          store2((weight ^ (((c0 + k + 1) & 7) << 4)) + (c0 + k + 1) * 128, w >> 16);
        }
      }
    } else {
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += 8) {
        uint32_t y[8];
        tmem_ld8(s_addr + c0, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = row0 + c0 + k;
          const float ref = sh.ref[row];
          const bool on = there && pos < sh.seen[row];
          const float s = __uint_as_float(y[k]) * kf * sh.factor[row] - (ref == -INFINITY ? 0.f : ref);
          const float p = on ? exp2_fast(s) : 0.f;
          sum[c0 + k] += p;
          store2((weight ^ (((c0 + k) & 7) << 4)) + (c0 + k) * 128, pack_bf16(on ? p * vf : 0.f, 0.f));
        }
      }
    }
    ptx::fence_async_shared();
    ptx::tc_fence_before();
    ptx::mbar_arrive(&sh.p_full[sb]);
  }

  // output: divided by the sum, turned back by R^T
  {
    const float s = over_lanes<NR>(sum, Add());
    if (tell) sh.part[quarter][mine] = s;
  }
  if (!TQ_WARP_WAIT(sh.v_empty[(st.vc - 1) & 1], ((st.vc - 1) >> 1) & 1) || !meet(c, st)) return false;
  ptx::tc_fence_after();
  const bool whole = t0 == 0 && t1 == it.tiles;
  // a run's first item may have begun in the run before, its last may go on
  float* const part = a.narrow.part + (2ll * blockIdx.x + (t0 == 0 ? 1 : 0)) * part_floats(kRows);
  // (a NaN in a visible token shows)
  float scale[NR], top[NR];
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const float s = quarters(c, row0 + k);
    scale[k] = s == 0.f ? 0.f : 1.f / s;
  }
  if (!whole && tid < rows) {
    const float s = quarters(c, tid);
    part[kRows * kDim + 2 * tid] = s == 0.f ? -INFINITY : sh.ref[tid];
    part[kRows * kDim + 2 * tid + 1] = s;
  }
#pragma unroll
  for (int c0 = 0; c0 < NR; c0 += 8) {
    uint32_t y[8];
    tmem_ld8(lane_addr + kO + row0 + c0, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) top[c0 + k] = fabsf(__uint_as_float(y[k]) * scale[c0 + k]);
  }
  const float largest = over_lanes<NR>(top, Max());
  if (!meet(c, st)) return false;                 // (the sums are read)
  if (tell) sh.part[quarter][mine] = largest;
  if (!meet(c, st)) return false;
  auto exponent = [&](int row) {
    return exponent_of(fmaxf(fmaxf(sh.part[0][row], sh.part[1][row]), fmaxf(sh.part[2][row], sh.part[3][row])));
  };
#pragma unroll
  for (int c0 = 0; c0 < NR; c0 += 8) {
    uint32_t y[8];
    tmem_ld8(lane_addr + kO + row0 + c0, y);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<__half*>(pass + row_element(row0 + c0 + k, at)) =
          __float2half_rn(__uint_as_float(y[k]) * scale[c0 + k] * exp2_int(-exponent(row0 + c0 + k)));
  }
  ptx::fence_async_shared();
  ptx::tc_fence_before();
  ptx::mbar_arrive(&sh.o_raw);
  if (!TQ_WARP_WAIT(sh.turned, seg & 1)) return false;
  ++st.vc;                                        // (R^T was a value ring entry)
  ptx::tc_fence_after();
#pragma unroll
  for (int c0 = 0; c0 < NR; c0 += 8) {
    uint32_t y[8];
    tmem_ld8(lane_addr + kS + row0 + c0, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = row0 + c0 + k;
      const float o = __uint_as_float(y[k]) * exp2_int(exponent(row));
      if (row < rows) {
        if (whole) static_cast<__nv_bfloat16*>(a.out)[sh.vec[row] * kDim + at] = __float2bfloat16_rn(o);
        else part[row * kDim + at] = o;
      }
    }
  }
  ptx::tc_fence_before();
  return meet(c, st);                             // (the rows' fields are read)
}

template <int KB, int VB>
__global__ void __launch_bounds__(kExtThreads, 1) extend_kernel(ExtendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ NarrowShared sh;
  // 1024-byte aligned, as an offset from smem_raw so that accesses stay shared-space
  uint8_t* const smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  const bool qjl = a.d.k_qjl != nullptr;
  {                                               // R and S (constants: before the launches this one follows are done)
    uint4* const dst = reinterpret_cast<uint4*>(smem + kImage0);
#pragma unroll 6
    for (int i = tid; i < (qjl ? 2 : 1) * (kExtendImageBytes / 16); i += kExtThreads) dst[i] = __ldg(a.images + i);
  }
  wait_prerequisites();
  const long long total = a.narrow.first[a.d.batch];
  const long long per = run_length(total, gridDim.x);
  Run run;
  run.pos = blockIdx.x * per;
  run.end = run.pos + per < total ? run.pos + per : total;
  if (run.pos >= run.end) {                       // (the whole CTA)
    if (threadIdx.x == 0) write_cut(a, a.narrow, run, per, false);
    return;
  }

  if (tid == 0) {
    sh.abort = 0;
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&sh.k_full[s], kKeyThreads);
      ptx::mbar_init(&sh.k_empty[s], 1);
      ptx::mbar_init(&sh.v_full[s], kValueThreads);
      ptx::mbar_init(&sh.v_empty[s], 1);
      ptx::mbar_init(&sh.s_full[s], 2);           // the products' completion and the issuer itself
      ptx::mbar_init(&sh.p_full[s], kSoftThreads);
    }
    ptx::mbar_init(&sh.q_raw, kSoftThreads);
    ptx::mbar_init(&sh.rotated, 1);
    ptx::mbar_init(&sh.q_full, kSoftThreads);
    ptx::mbar_init(&sh.o_raw, kSoftThreads);
    ptx::mbar_init(&sh.turned, 1);
    ptx::mbar_init(&sh.meet, kSoftThreads);
    ptx::mbar_init(&sh.drain, 1);
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&sh.tmem, 512);
    ptx::tmem_relinquish();
  }
  if (warp == 0) {
    int offset;
    const Item it = find_item(a, a.narrow, run.pos, &offset);
    if (lane == 0) {
      sh.item = it;
      sh.offset = offset;
    }
  }
  ptx::fence_async_shared();                      // (the images)
  __syncthreads();
  ptx::tc_fence_after();
  const Cta c{a, a.d, sh, smem, sh.tmem, qjl};
  const DecodeArgs& d = a.d;
  run.it = sh.item;
  run.offset = sh.offset;
  const Item& it = run.it;
  int t0, t1;                                     // key tiles of the current segment
  float* const key_factor = reinterpret_cast<float*>(smem + kFactor0);
  float* const value_factor = key_factor + kRing * kTile;
  bool ok = true;

  if (warp < 8) {
    // ---------------- softmax ----------------
    SoftState st{0, 0, 0};
    for (int seg = 0; ok && next_segment(a, a.narrow, run, t0, t1); ++seg) {
      const int columns = tile_columns(tile_rows(c, it));
      if (columns == 16) ok = softmax_segment<8>(c, run, t0, t1, seg, st);
      else if (columns == 32) ok = softmax_segment<16>(c, run, t0, t1, seg, st);
      else ok = softmax_segment<32>(c, run, t0, t1, seg, st);
      end_segment(a, a.narrow, run, t1);
    }
  } else if (warp < 16) {
    // ---------------- keys ----------------
    const int row = (tid - kSoftThreads) & (kTile - 1);   // lane of the operand: token expanded_bit(lane) of the warp's group
    const int half = (tid - kSoftThreads) / kTile;        // coordinates 64 half .. + 63 of both operand halves
    const LevelBytes lev = level_bytes<false>(d.tables->k_levels, KB);
    float biggest = 0.f;                          // the outermost level
    for (int i = 0; i < (1 << KB); ++i) biggest = fmaxf(biggest, fabsf(d.tables->k_levels[i]));
    const float to_log2 = d.scale * 1.4426950408889634f;
    const uint32_t lane_addr = c.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kKeys + 32 * half;
    int jt = 0;                                   // key tiles so far
    while (ok && next_segment(a, a.narrow, run, t0, t1)) {
      Cursor cur;
      RawKey<KB> next;
      start_cursor(d, it, t0 * kTile + (row & ~31), cur);
      load_key(d, it, cur, expanded_bit(lane), half, next);
      advance(d, it, cur);
      prefetch_queries(a, a.narrow, run, t1, tid - kSoftThreads, kKeyThreads);
      for (int t = t0; t < t1; ++t, ++jt) {
        const RawKey<KB> k = next;
        if (t + 1 < t1) {
          load_key(d, it, cur, expanded_bit(lane), half, next);
          advance(d, it, cur);
        }
        const int s = jt & 1, rg = jt & (kRing - 1);
        ok = TQ_WARP_WAIT(sh.k_empty[s], ((jt >> 1) & 1) ^ 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const float rho = qjl && k.norm > 0.f ? __fdividef(k.rnorm * d.qjl_coef, k.norm) : 0.f;
        const uint32_t minus_rho = __half_as_ushort(__float2half_rn(rho)) * 0x00010001u ^ 0x80008000u;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t planes[KB];
#pragma unroll
          for (int p = 0; p < KB; ++p) planes[p] = w ? k.planes[p].y : k.planes[p].x;
          store_levels<KB>(lane_addr + 128 * s + 16 * w, planes, lev);
          if (qjl) store_signs(lane_addr + 128 * s + 64 + 16 * w, w ? k.qjl.y : k.qjl.x, minus_rho);
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
            sh.valid[rg][row >> 5] = bit;
            sh.reach[rg][row >> 5] = make_float2(__uint_as_float(bits_c), __uint_as_float(bits_q));
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&sh.k_full[s]);
      }
      end_segment(a, a.narrow, run, t1);
    }
  } else if (warp < kMmaWarp) {
    // ---------------- values ----------------
    const int dim = (tid - kSoftThreads - kKeyThreads) & (kTile - 1);
    const int half = (tid - kSoftThreads - kKeyThreads) / kTile;   // 32-token groups 2 half and 2 half + 1
    // the first two warps of a half write its 64 factors, by expanded column
    const int mine = dim < 64 ? dim >> 5 : -1;
    const LevelBytes lev = level_bytes<true>(d.tables->v_levels, VB);
    int jt = 0, vc = 0;                           // key tiles, ring entries so far
    if (tid == kSoftThreads + kKeyThreads) write_cut(a, a.narrow, run, per, true);
    while (ok && next_segment(a, a.narrow, run, t0, t1)) {
      Cursor cur;
      RawValue<VB> next;
      start_cursor(d, it, t0 * kTile + 64 * half + 32 * (lane & 1), cur);
      load_value(d, it, cur, dim, mine, expanded_bit(lane), next);
      advance(d, it, cur);
      for (int t = t0; t < t1; ++t, ++jt, ++vc) {
        const RawValue<VB> v = next;
        if (t + 1 < t1) {
          load_value(d, it, cur, dim, mine, expanded_bit(lane), next);
          advance(d, it, cur);
        }
        const int s = vc & 1, rg = jt & (kRing - 1);
        ok = TQ_WARP_WAIT(sh.v_empty[s], ((vc >> 1) & 1) ^ 1);
        if (!ok) break;
        const RowChunks at = row_chunks(ptx::smem_u32(smem + kValue0 + s * kValueBytes) + half * kBlockBytes, dim);
        uint32_t lo[VB], hi[VB];
#pragma unroll
        for (int p = 0; p < VB; ++p) lo[p] = v.words[p][0], hi[p] = v.words[p][1];
        expand32<VB, 0>(at, lo, lev);
        expand32<VB, 0>(second_word(at), hi, lev);
        if (mine >= 0) value_factor[rg * kTile + 64 * half + dim] = v.norm;
        ptx::fence_async_shared();
        ptx::mbar_arrive(&sh.v_full[s]);
      }
      if (!ok) break;
      // R^T, for the output, as a ring entry
      const int s = vc & 1;
      ok = TQ_WARP_WAIT(sh.v_empty[s], ((vc >> 1) & 1) ^ 1);
      if (!ok) break;
      const uint4* const src = a.images + 2 * (kExtendImageBytes / 16);
      uint4* const dst = reinterpret_cast<uint4*>(smem + kValue0 + s * kValueBytes);
#pragma unroll
      for (int i = 0; i < kExtendImageBytes / 16 / kValueThreads; ++i) {
        const int k = i * kValueThreads + tid - kSoftThreads - kKeyThreads;
        dst[k] = __ldg(src + k);
      }
      ptx::fence_async_shared();
      ptx::mbar_arrive(&sh.v_full[s]);
      ++vc;
      end_segment(a, a.narrow, run, t1);
    }
  } else {
    // ---------------- products ----------------
    // the whole warp walks the tiles and waits; an elected lane issues
    const uint64_t value_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kValue0));
    const uint64_t image_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kImage0));
    const uint64_t query_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kQuery0));
    const uint64_t weight_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kWeight0));
    constexpr uint64_t kWide = kBlockBytes / 16, kSlim = kRowBlock / 16;   // K blocks in descriptor units
    int jt = 0, vc = 0;                           // key tiles, value ring entries so far
    for (int seg = 0; ok && next_segment(a, a.narrow, run, t0, t1); ++seg) {
      const uint32_t n = tile_columns(tile_rows(c, it));
      const uint32_t idesc_bf16 = ptx::idesc_bf16_f32(128, n), idesc_f16 = idesc_bf16 & ~((7u << 7) | (7u << 10));
      // (R q)^T and (S q)^T
      ok = TQ_WARP_WAIT(sh.q_raw, seg & 1);
      if (!ok) break;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        shared_product<8>(c.tmem + kS, image_desc, kWide, weight_desc, kSlim, idesc_f16, false);
        if (qjl)
          shared_product<8>(c.tmem + kS + kRows, image_desc + kExtendImageBytes / 16, kWide, weight_desc, kSlim, idesc_f16,
                            false);
        ptx::mma_commit(&sh.rotated);
      }
      __syncwarp();
      ok = TQ_WARP_WAIT(sh.q_full, seg & 1);
      if (!ok) break;
      // scores of the CTA's key tile j; the columns' last reader, the softmax of
      // tile j - 2, is done (its weights were waited for)
      auto scores = [&](int j) {
        if (!TQ_WARP_WAIT(sh.k_full[j & 1], (j >> 1) & 1)) return false;
        if (ptx::elect_one()) {
          ptx::tc_fence_after();
          const uint32_t keys = c.tmem + kKeys + 128 * (j & 1), to = c.tmem + kS + kRows * (j & 1);
#pragma unroll
          for (int ks = 0; ks < 16; ++ks)
            if (ks < 8 || qjl)
              ptx::mma_bf16_tmem_a(to, keys + 8 * ks, query_desc + (ks >> 2) * kSlim + (ks & 3) * 2, idesc_f16, ks > 0);
          ptx::mma_commit(&sh.s_full[j & 1]);
          ptx::mma_commit(&sh.k_empty[j & 1]);
          ptx::mbar_arrive(&sh.s_full[j & 1]);
        }
        __syncwarp();
        return true;
      };
      ok = scores(jt);
      for (int t = t0; ok && t < t1; ++t, ++jt, ++vc) {
        if (t + 1 < t1) ok = scores(jt + 1);
        const int s = vc & 1;
        ok = ok && TQ_WARP_WAIT(sh.v_full[s], (vc >> 1) & 1) && TQ_WARP_WAIT(sh.p_full[jt & 1], (jt >> 1) & 1);
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::tc_fence_after();
          shared_product<8>(c.tmem + kO, value_desc + s * (kValueBytes / 16), kWide, weight_desc + s * 2 * kSlim, kSlim,
                            idesc_bf16, t > t0);
          ptx::mma_commit(&sh.v_empty[s]);
        }
        __syncwarp();
      }
      // R^T out
      ok = ok && TQ_WARP_WAIT(sh.v_full[vc & 1], (vc >> 1) & 1) && TQ_WARP_WAIT(sh.o_raw, seg & 1);
      if (!ok) break;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        shared_product<8>(c.tmem + kS, value_desc + (vc & 1) * (kValueBytes / 16), kWide, weight_desc, kSlim, idesc_f16,
                          false);
        ptx::mma_commit(&sh.turned);
        ptx::mma_commit(&sh.v_empty[vc & 1]);
      }
      __syncwarp();
      ++vc;
      end_segment(a, a.narrow, run, t1);
    }
    if (ptx::elect_one()) {
      ptx::mma_commit(&sh.drain);                 // nothing is in flight when the CTA ends
      ptx::drain_bar(&sh.drain, 0);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(c.tmem, 512);
  }
}

#undef TQ_WARP_WAIT
#undef TQ_WAIT

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
