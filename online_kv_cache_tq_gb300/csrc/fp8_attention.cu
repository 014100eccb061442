// Attention over the 8-bit cache, few rows (new tokens x query heads of a
// group) per sequence: a decode step, the verification of drafted tokens.
//
//   s_tr = scale <q_r, c_t> 2^{e_k(t)},  o_r = sum_t p_tr c^v_t 2^{e_v(t)},  p = softmax(s)
//
// Both products run on the tensor cores on the codes as they lie in memory: a
// block's run of a KV head is a K-major operand without swizzle, so that a key
// or value tile (128 tokens) is four bulk copies of 32 tokens and no
// instruction touches its bytes.  Cached tokens are the lanes of the score
// product, coordinates those of the output product; rows are its columns:
//   scores [128 tokens x 2 RT or 4 RT] = keys x (two or four e4m3 pieces of each query)^T,
//   output [128 coordinates x 3 RT] = values^T x (three pieces of each weight)^T,
// each piece what those before leave, times a power of two.  Two pieces of four
// bits are a bf16 coordinate exactly, where it is 2^-12 of the query's largest or
// more, and hold it to 2^-21 of the largest below that; four hold a float32 one to
// 2^-16 of itself.  (bf16 with two | with four: 16 rows on 8192 tokens 58.5 | 60.3
// us, on 2000 99 | 105.)  Weights are held to 2^-11: rounded to fp16, then three
// pieces.  A thread owns a token for the softmax and a coordinate for the output,
// of eight rows; it keeps the output in registers and adds a tile's product to it,
// so nothing is rescaled in tensor memory.
//
// The bound is HBM: 256 bytes per token and KV head.  A tile of 32 KB takes an
// SM 1490 cycles at the copy rate; one chain of softmax on a tile (four warps:
// scores, a meeting over the tile's maximum, weights, the product before) takes
// 2400, so two CTAs an SM work side by side.  Measured: 64 sequences of 1 to 32 K
// tokens, 64/8 heads, 341 us (6.9 TB/s); 16 of 8192, 32/8 heads, 48.4 us, and one of
// 131072, 64/8, 48.6 us (5.5 TB/s): 2.5 us until the first copies, 3 us in which
// some CTAs are done and others not, 3 us for the join.  Sixteen rows a tile are
// issue bound: 53 us for 16 sequences of 8192 with 16 rows.
//
// Work is split as in extend.cu: an item is a row tile of a sequence and KV
// head, worth kItemCost units and one per key tile; every CTA takes an equal
// run of units, and row tiles that runs cut are joined by a second launch.
// Every CTA forms the sums over the batch itself, which costs less than a
// launch before it.  (An item cost of 1, 2, 3: the 64 sequences 353, 346, 345 us,
// 32 short ones of 16 rows 18.8, 18.9, 22.3 us.)
#include <algorithm>
#include <cstddef>

#include "dependent.cuh"
#include "fp8_common.cuh"
#include "tc_ptx.cuh"

namespace tq {
namespace {

#define TQ_WAIT(b, ph) ptx::wait_bar(&(b), (ph), abort, c.error, kErrTimeout)
#define TQ_WARP_WAIT(b, ph) __all_sync(0xffffffffu, TQ_WAIT(b, ph))

constexpr int kTile = 128;             // tokens of a key tile
constexpr int kSlotBytes = kTile * kDim;
constexpr int kGroupBytes = 32 * kDim; // keys or values of 32 tokens: one copy
constexpr int kRowsPerThread = 8;
constexpr int kMetaRing = 16;          // more tiles than can be on their way
constexpr int kItemCost = 2;
constexpr int kCtasPerSm = 2;
constexpr float kNothing = -3e38f;     // a row's reference before it sees a token
constexpr float kWeightScale = 256.f;  // weights are at most 1: times this in e4m3

// RT rows a tile, 8 or 16, with queries of QP pieces; two CTAs an SM.
template <int RT, int QP>
struct Shape {
  static constexpr int kSplit = RT / kRowsPerThread;        // threads per token
  static constexpr int kSoftWarps = 4 * kSplit;
  static constexpr int kThreads = 32 * (kSoftWarps + 2);
  static constexpr int kSlots = 5;                          // ring of key and value tiles in turn
  static constexpr float kPiece = QP == 2 ? 64.f : 16.f;    // a query's piece over the one before
  static constexpr int kQueryCols = QP * RT;
  static constexpr int kWeightCols = (3 * RT + 15) / 16 * 16;
  // (64 bytes more than the rows between sixteen tokens and the next, so that a
  // warp's byte stores to both meet different banks)
  static constexpr int kWeightStride = kWeightCols * 16 + 64;
  static constexpr int kQueryBytes = kQueryCols * kDim, kWeightBytes = kWeightStride * kTile / 16;
  static constexpr int kTmem = RT == 8 || QP == 2 ? 128 : 256;
  static constexpr int kSmem = kSlots * kSlotBytes + 2 * kQueryBytes + 2 * kWeightBytes + 128;   // (128: alignment)
  static_assert(2 * kQueryCols + kWeightCols <= kTmem, "two buffers of scores, one of outputs");
};

struct TileInfo {
  float k_scale[4], v_scale[4];   // by group of 32 tokens
  uint32_t groups;                // those that there are
};

// A sequence as the launch sees it.
struct Sequence {
  int row0, n, ctx;
  long long units;
  bool ok;
};
__device__ __forceinline__ int row_tiles(int rows, int rt) { return (rows + rt - 1) / rt; }
__device__ __forceinline__ int key_tiles(int ctx) { return max(1, (ctx + kTile - 1) / kTile); }
template <int RT>
__device__ __forceinline__ Sequence load_sequence(const Fp8AttendArgs& a, int b) {
  const Fp8Cache& c = a.c;
  Sequence s;
  if (a.seq != nullptr) {                         // (checked by the plan; the wide form's have no work here)
    const int4 q = a.seq[b];
    s.row0 = q.x;
    s.n = q.w >= 0 ? 0 : q.y;
    s.ctx = q.z;
    s.ok = true;
    s.units = s.n == 0 ? 0 : static_cast<long long>(c.n_kv) * row_tiles(s.n * a.group, RT) * (kItemCost + key_tiles(s.ctx));
    return s;
  }
  const int s0 = c.query_start[b], s1 = c.query_start[b + 1], ctx = c.context_lens[b];
  const bool rows_ok = s0 >= 0 && s0 <= s1 && s1 <= c.n_tokens;
  const bool ctx_ok = ctx >= 0 && ctx <= a.max_context && ctx <= static_cast<long long>(c.max_blocks) * c.block_size;
  s.row0 = rows_ok ? s0 : 0;
  s.n = rows_ok ? s1 - s0 : 0;
  s.ctx = ctx_ok ? ctx : 0;
  s.ok = rows_ok && ctx_ok;
  if (a.wide_from > 0 && s.n * a.group >= a.wide_from) s.n = 0;   // (the wide form's)
  s.units = s.n == 0 ? 0 : static_cast<long long>(c.n_kv) * row_tiles(s.n * a.group, RT) * (kItemCost + key_tiles(s.ctx));
  return s;
}

// Where a run of units begins: a sequence and the unit in it.
struct RunStart {
  long long total, rem;
  int b;
  Sequence s;
};

// A walk over a run's items: a sequence's row tiles, and in each its KV heads,
// so that the row tiles that read the same keys are worked on by different CTAs
// at about the same time and find them in L2.
template <int RT>
struct Walk {
  int b, kvh, rt;        // sequence, KV head, row tile
  int tile, tiles;       // the run's first key tile of the item, and how many the item has
  Sequence s;
  long long pos, end;    // unit of that tile, end of the run

  // At the run's first item; false when the run ends before a key tile.
  __device__ __forceinline__ bool start(const Fp8AttendArgs& a, const RunStart& at) {
    b = at.b;
    s = at.s;
    tiles = key_tiles(s.ctx);
    const long long item = at.rem / (kItemCost + tiles);
    const int offset = static_cast<int>(at.rem - item * (kItemCost + tiles));
    rt = static_cast<int>(item / a.c.n_kv);
    kvh = static_cast<int>(item - static_cast<long long>(rt) * a.c.n_kv);
    tile = max(0, offset - kItemCost);
    pos += max(0, kItemCost - offset);
    return pos < end;
  }
  // The run's key tiles of the item.
  __device__ __forceinline__ int span() const { return static_cast<int>(min(static_cast<long long>(tiles - tile), end - pos)); }
  // To the next item; false at the run's end.
  __device__ __forceinline__ bool next(const Fp8AttendArgs& a) {
    pos += (tiles - tile) + kItemCost;
    if (pos >= end) return false;
    if (++kvh >= a.c.n_kv) {
      kvh = 0;
      if (++rt >= row_tiles(s.n * a.group, RT)) {
        rt = 0;
        do {
          s = load_sequence<RT>(a, ++b);          // (units are left, so there is one with work)
        } while (s.units == 0);
        tiles = key_tiles(s.ctx);
      }
    }
    tile = 0;
    return true;
  }
};

// The run's start, by the whole CTA.
template <int RT, int kWarps>
__device__ __forceinline__ void find_run(const Fp8AttendArgs& a, RunStart* out, long long* warp_s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int batch = a.c.batch;
  // all units: in one round while the batch has no more sequences than the CTA threads
  long long mine = 0;
  Sequence s{};
  for (int b = tid; b < batch; b += blockDim.x) {
    s = load_sequence<RT>(a, b);
    if (!s.ok && blockIdx.x == 0) atomicCAS(a.c.error, 0, kErrContext);
    mine += s.units;
  }
  auto scan = [&](long long v, long long* total) {      // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += o;
    }
    if (lane == 31) warp_s[warp] = v;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_s[w];
      all += warp_s[w];
    }
    __syncthreads();
    *total = all;
    return v + before;
  };
  long long total;
  const long long upto = scan(mine, &total);
  const long long pos = blockIdx.x * ((total + gridDim.x - 1) / gridDim.x);
  if (tid == 0) out->total = total;
  auto look = [&](int b, long long end, const Sequence& seq) {
    if (seq.units > 0 && end - seq.units <= pos && pos < end) {
      out->b = b;
      out->rem = pos - (end - seq.units);
      out->s = seq;
    }
  };
  if (batch <= static_cast<int>(blockDim.x)) {
    look(tid, upto, s);
  } else {
    long long base = 0;
    for (int b0 = 0; b0 < batch; b0 += blockDim.x) {
      const int b = b0 + tid;
      Sequence one{};
      if (b < batch) one = load_sequence<RT>(a, b);
      long long all;
      const long long end = base + scan(one.units, &all);
      look(b, end, one);
      base += all;
    }
  }
  __syncthreads();
}

// Two halves as e4m3 codes, and back; a byte to shared memory.
__device__ __forceinline__ uint16_t fp8_pair_of_halves(__half2 h) {
  uint16_t p;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(p) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
  return p;
}
__device__ __forceinline__ __half2 halves_of_fp8_pair(uint16_t p) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(p));
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ void store_byte(uint32_t saddr, uint16_t b) {
  asm volatile("st.shared.b8 [%0], %1;" ::"r"(saddr), "h"(b) : "memory");
}
// All but the bytes whose bits are set (four of them).
__device__ __forceinline__ uint32_t bytes_without(uint32_t bits) {
  return ~(((bits & 1u) | (bits & 2u) << 7 | (bits & 4u) << 14 | (bits & 8u) << 21) * 255u);
}
// The warp's largest (NaN does not count).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void copy4_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
// An arrival when the thread's copies so far have landed.
__device__ __forceinline__ void arrive_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]),
                   "=r"(r[i + 7])
                 : "r"(taddr + i)
                 : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));   // (nothing that uses them goes before the wait)
}

template <int RT, int QP>
struct Barriers {
  uint64_t full[Shape<RT, QP>::kSlots], empty[Shape<RT, QP>::kSlots];
  uint64_t s_full[2], p_full[2], o_full[2];   // scores, weights and output product of a tile
  uint64_t q_full[2];                         // queries of a segment
  uint64_t maxima[Shape<RT, QP>::kSplit], sums;   // the softmax warps of a row split, and all of them
  uint64_t drain;
};

template <int RT, int QP>
struct Shared {
  Barriers<RT, QP> bar;
  TileInfo info[kMetaRing];
  __align__(16) float factor[2][RT];           // scale log2(e) over the query's piece scale
  int seen[2][RT];               // positions a row sees
  float4 top[2][Shape<RT, QP>::kSplit][4][2];   // largest scores of a tile, by warp: eight rows
  __align__(16) float sum[2][Shape<RT, QP>::kSoftWarps][kRowsPerThread];
  __align__(16) uint32_t poison[3][RT];        // rows that see a value that is NaN
  long long warp_s[Shape<RT, QP>::kThreads / 32];
  RunStart start;
  uint32_t tmem;
  int abort;
};

// Floats of a partial output: the rows' outputs, then their (reference, sum).
__host__ __device__ constexpr int part_floats(int rows) { return rows * (kDim + 2); }

// Vector (token x query head) of row r of a sequence and KV head.
__device__ __forceinline__ long long row_vector(const Fp8AttendArgs& a, int row0, int kvh, int r) {
  const int tok = r / a.group;
  return (static_cast<long long>(row0) + tok) * a.n_q + kvh * a.group + r - tok * a.group;
}

// Rows r0, r0 + step, .. (N of them) of the walk's item as operand rows of the
// score product, by a warp: four coordinates a lane, as e4m3 pieces of the
// query times a power of two.
template <int N, int RT, int QP>
__device__ __forceinline__ void prepare_rows(const Fp8AttendArgs& a, const Walk<RT>& walk, int r0, int step, uint8_t* operand,
                                             float* factor, int* seen) {
  const int lane = threadIdx.x & 31, rows = walk.s.n * a.group, first = walk.rt * RT;
  uint8_t* const dst = operand + (lane >> 2) * (Shape<RT, QP>::kQueryCols * 16) + (lane & 3) * 4;
  float v[N][4];
  int token[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = first + r0 + i * step;
    v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
    token[i] = row / a.group;
    if (row < rows) {
      const long long vec = (static_cast<long long>(walk.s.row0) + token[i]) * a.n_q + walk.kvh * a.group + row - token[i] * a.group;
      const long long at = vec * kDim + 4 * lane;
      if constexpr (QP == 2) {                    // (bf16)
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + at));
        v[i][0] = __uint_as_float(u.x << 16), v[i][1] = __uint_as_float(u.x & 0xffff0000u);
        v[i][2] = __uint_as_float(u.y << 16), v[i][3] = __uint_as_float(u.y & 0xffff0000u);
      } else {
        const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
        v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * step;
    const float most = fmaxf(fmaxf(fabsf(v[i][0]), fabsf(v[i][1])), fmaxf(fabsf(v[i][2]), fabsf(v[i][3])));
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    // 2^e <= most < 2^(e+1) goes to [64, 128); tiny queries stay tiny
    const int e = max(-100, static_cast<int>(bits >> 23) - 127);
    const float up = e > 127 ? __int_as_float(0x7fc00000) : fp8_power(6 - e);   // (infinite: the row is NaN)
    float4 y = make_float4(v[i][0] * up, v[i][1] * up, v[i][2] * up, v[i][3] * up);
#pragma unroll
    for (int p = 0; p < QP; ++p) {
      const uint32_t w = fp8_four(y.x, y.y, y.z, y.w);
      *reinterpret_cast<uint32_t*>(dst + (QP * r + p) * 16) = w;
      const float2 lo = fp8_floats(w), hi = fp8_floats(w >> 16);
      constexpr float up = Shape<RT, QP>::kPiece;
      y = make_float4((y.x - lo.x) * up, (y.y - lo.y) * up, (y.z - hi.x) * up, (y.w - hi.y) * up);
    }
    if (lane == 0) {
      const bool live = first + r < rows;
      factor[r] = live ? a.scale * 1.4426950408889634f * fp8_power(e - 6) : 0.f;
      seen[r] = live ? walk.s.ctx - walk.s.n + token[i] + 1 : walk.s.ctx;
    }
  }
  ptx::fence_async_shared();
  __syncwarp();
}

template <int RT, int QP>
__global__ void __launch_bounds__(Shape<RT, QP>::kThreads, kCtasPerSm) fp8_attend_kernel(Fp8AttendArgs a) {
  using P = Shape<RT, QP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<RT, QP> sh;
  using Sh = Shared<RT, QP>;
  static_assert(offsetof(Sh, top) % 16 == 0 && offsetof(Sh, factor) % 16 == 0 && offsetof(Sh, sum) % 16 == 0 &&
                    offsetof(Sh, poison) % 16 == 0 && alignof(Sh) >= 16, "16-byte stores");
  uint8_t* const smem = smem_raw + ((128u - (ptx::smem_u32(smem_raw) & 127u)) & 127u);
  uint8_t* const query_s = smem + P::kSlots * kSlotBytes;
  uint8_t* const weight_s = query_s + 2 * P::kQueryBytes;
  const Fp8Cache& c = a.c;
  Barriers<RT, QP>& bar = sh.bar;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* const abort = &sh.abort;
  launch_dependents();
  if (warp == P::kSoftWarps) {
    ptx::tmem_alloc(&sh.tmem, P::kTmem);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    sh.abort = 0;
    for (int s = 0; s < P::kSlots; ++s) {
      ptx::mbar_init(&bar.full[s], 5);            // the bytes, and four lanes
      ptx::mbar_init(&bar.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bar.s_full[s], 1);
      ptx::mbar_init(&bar.p_full[s], P::kSoftWarps);
      ptx::mbar_init(&bar.o_full[s], 1);
      ptx::mbar_init(&bar.q_full[s], P::kSoftWarps);
    }
    for (int s = 0; s < P::kSplit; ++s) ptx::mbar_init(&bar.maxima[s], 4);
    ptx::mbar_init(&bar.sums, P::kSoftWarps);
    ptx::mbar_init(&bar.drain, 1);
    ptx::fence_mbar_init();
  }
  for (int i = tid; i < 3 * RT; i += P::kThreads) (&sh.poison[0][0])[i] = 0;
  ptx::tc_fence_before();
  wait_prerequisites();                           // (for the plan, where there is one)
  find_run<RT, P::kThreads / 32>(a, &sh.start, sh.warp_s);
  ptx::tc_fence_after();
  const long long total = sh.start.total, per = (total + gridDim.x - 1) / gridDim.x;
  Walk<RT> walk;
  walk.pos = blockIdx.x * per;
  walk.end = min(walk.pos + per, total);
  bool more = walk.pos < walk.end && walk.start(a, sh.start);
  const uint32_t tmem = sh.tmem;
  const uint32_t scores_t = tmem, outputs_t = tmem + 2 * P::kQueryCols;
  bool ok = true;

  if (warp < P::kSoftWarps) {
    // ---------------- softmax and output ----------------
    const int quarter = warp & 3, split = warp >> 2, token = 32 * quarter + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t my_scores = scores_t + lanes + QP * kRowsPerThread * split;
    const uint32_t my_outputs = outputs_t + lanes + 3 * kRowsPerThread * split;
    const uint32_t my_weights =
        ptx::smem_u32(weight_s) + (token >> 4) * P::kWeightStride + 3 * kRowsPerThread * split * 16 + (token & 15);
    const __half2 weight_scale = __float2half2_rn(kWeightScale), sixteen = __float2half2_rn(16.f);
    int jt = 0, met = 0;                          // key tiles so far, and those that this split's warps met over
    int slot = 1, slot_phase = 0;                 // of the value tile
    auto prepare = [&](const Walk<RT>& w, int seg) {          // a segment's queries
      prepare_rows<RT / P::kSoftWarps, RT, QP>(a, w, warp, P::kSoftWarps, query_s + (seg & 1) * P::kQueryBytes, sh.factor[seg & 1],
                                           sh.seen[seg & 1]);
      if (lane == 0) ptx::mbar_arrive(&bar.q_full[seg & 1]);
    };
    if (more) prepare(walk, 0);
    for (int seg = 0; more; ++seg) {
      const int n = walk.s.n, ctx = walk.s.ctx, row0 = walk.s.row0, kvh = walk.kvh, rt = walk.rt;
      const int first = rt * RT + split * kRowsPerThread;     // my first row of the sequence
      const int tile0 = walk.tile, tiles = walk.tiles, reached = tile0 + walk.span();
      // (called after the last weights: the next queries, while the last product runs)
      auto move_on = [&]() {
        more = walk.next(a);
        if (more) prepare(walk, seg + 1);
      };
      if (first >= n * a.group) {
        // no such rows: only keep in step
        for (int t = tile0; ok && t < reached; ++t, ++jt) {
          ok = TQ_WARP_WAIT(bar.s_full[jt & 1], (jt >> 1) & 1);
          if (ok && lane == 0) ptx::mbar_arrive(&bar.p_full[jt & 1]);
          slot += 2;
          if (slot >= P::kSlots) slot -= P::kSlots, slot_phase ^= 1;
        }
        if (!ok) break;
        move_on();
        if (lane == 0) ptx::mbar_arrive(&bar.sums);
        ok = TQ_WARP_WAIT(bar.sums, seg & 1);
        if (!ok) break;
        continue;
      }
      ok = TQ_WARP_WAIT(bar.q_full[seg & 1], (seg >> 1) & 1);
      if (!ok) break;
      const float4* const factor4 = reinterpret_cast<const float4*>(sh.factor[seg & 1] + split * kRowsPerThread);
      const int* const seen = sh.seen[seg & 1] + split * kRowsPerThread;
      const int plain_tiles = sh.seen[seg & 1][0] / kTile;    // those before are seen by every row
      float acc[kRowsPerThread], sum[kRowsPerThread], ref[kRowsPerThread];
#pragma unroll
      for (int r = 0; r < kRowsPerThread; ++r) acc[r] = sum[r] = 0.f, ref[r] = kNothing;
      auto add_output = [&](int j) {              // tile j's product
        if (!TQ_WARP_WAIT(bar.o_full[j & 1], (j >> 1) & 1)) return false;
        ptx::tc_fence_after();
        uint32_t d[24];
        tmem_load(my_outputs, d);
        ptx::tc_fence_before();
        if (sh.info[j & (kMetaRing - 1)].groups == 0) return true;   // (nothing was multiplied)
#pragma unroll
        for (int r = 0; r < kRowsPerThread; ++r) {
          const float d0 = __uint_as_float(d[3 * r]), d1 = __uint_as_float(d[3 * r + 1]), d2 = __uint_as_float(d[3 * r + 2]);
          acc[r] = fmaf(fmaf(d2, 0.0625f, d1), 0.0625f, acc[r] + d0);
        }
        return true;
      };
      for (int t = tile0; t < reached; ++t, ++jt) {
        ok = TQ_WARP_WAIT(bar.s_full[jt & 1], (jt >> 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[QP * kRowsPerThread];
        tmem_load(my_scores + (jt & 1) * P::kQueryCols, s);
        ok = TQ_WARP_WAIT(bar.full[slot], slot_phase);
        if (!ok) break;
        const TileInfo& info = sh.info[jt & (kMetaRing - 1)];
        const uint32_t groups = info.groups;
        const float ks = info.k_scale[quarter];
        const int e = fp8_exponent(info.v_scale[quarter]);
        const float up = static_cast<float>(e), down = fp8_power(-e);
        const bool here = groups >> quarter & 1u;
        const int pos = t * kTile + token;
        float x[kRowsPerThread], top[kRowsPerThread];
        const float4 f0 = factor4[0], f1 = factor4[1];
        const float factor[kRowsPerThread] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int r = 0; r < kRowsPerThread; ++r) {
          float d = __uint_as_float(s[QP * r + QP - 1]);
#pragma unroll
          for (int p = QP - 2; p >= 0; --p) d = fmaf(d, 1.f / P::kPiece, __uint_as_float(s[QP * r + p]));
          // (with the value's scale: what the weight is of the block's codes)
          x[r] = fmaf(d * ks, factor[r], up);
        }
        if (groups != 15u || t >= plain_tiles) {
#pragma unroll
          for (int r = 0; r < kRowsPerThread; ++r) x[r] = here && pos < seen[r] ? x[r] : -INFINITY;
        }
        // the tile's largest, over the four warps
#pragma unroll
        for (int r = 0; r < kRowsPerThread; ++r) top[r] = warp_max(x[r]);
        float4(*const buf)[2] = sh.top[met & 1][split];
        if (lane == 0) {
          buf[quarter][0] = make_float4(top[0], top[1], top[2], top[3]);
          buf[quarter][1] = make_float4(top[4], top[5], top[6], top[7]);
          ptx::mbar_arrive(&bar.maxima[split]);
        }
        if (t > tile0) {                          // the tile before, while the warps meet
          ok = add_output(jt - 1);
          if (!ok) break;
        }
        ok = TQ_WARP_WAIT(bar.maxima[split], met & 1);
        if (!ok) break;
        ++met;
        bool raise = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 m0 = buf[0][h], m1 = buf[1][h], m2 = buf[2][h], m3 = buf[3][h];
          top[4 * h] = fmaxf(fmaxf(m0.x, m1.x), fmaxf(m2.x, m3.x));
          top[4 * h + 1] = fmaxf(fmaxf(m0.y, m1.y), fmaxf(m2.y, m3.y));
          top[4 * h + 2] = fmaxf(fmaxf(m0.z, m1.z), fmaxf(m2.z, m3.z));
          top[4 * h + 3] = fmaxf(fmaxf(m0.w, m1.w), fmaxf(m2.w, m3.w));
        }
#pragma unroll
        for (int r = 0; r < kRowsPerThread; ++r) raise = raise || top[r] > ref[r];
        if (raise) {                              // (the same for all four warps)
#pragma unroll
          for (int r = 0; r < kRowsPerThread; ++r) {
            const float to = fmaxf(ref[r], top[r]), keep = exp2_fast(ref[r] - to);
            sum[r] *= keep;
            acc[r] *= keep;
            ref[r] = to;
          }
        }
        // weights: at most 1, of the block's codes
        const uint32_t dst = my_weights + (jt & 1) * P::kWeightBytes;
#pragma unroll
        for (int r = 0; r < kRowsPerThread; r += 2) {
          const float w0 = exp2_fast(x[r] - ref[r]), w1 = exp2_fast(x[r + 1] - ref[r + 1]);
          sum[r] = fmaf(w0, down, sum[r]);
          sum[r + 1] = fmaf(w1, down, sum[r + 1]);
          // (fp16 holds 2^-12 of a weight too, and what pieces leave of it exactly)
          __half2 y = __hmul2(__floats2half2_rn(w0, w1), weight_scale);
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint16_t p = fp8_pair_of_halves(y);
            store_byte(dst + (3 * r + i) * 16, p);
            store_byte(dst + (3 * r + 3 + i) * 16, static_cast<uint16_t>(p >> 8));
            if (i < 2) y = __hmul2(__hsub2(y, halves_of_fp8_pair(p)), sixteen);
          }
        }
        if (split == 0 && here) {
          // values that no weight may meet: slots behind the context, whatever
          // they hold, and vectors that are NaN (whose rows are marked)
          uint8_t* const value = smem + slot * kSlotBytes + quarter * kGroupBytes;
          const bool nan = (value[(lane >> 4) * 2048 + (lane & 15)] & 0x7fu) == 0x7fu;
          const uint32_t gone = __ballot_sync(0xffffffffu, pos >= ctx || nan);
          if (gone != 0) {
            if (pos < ctx && nan)
              for (int r = 0; r < RT; ++r)
                if (pos < sh.seen[seg & 1][r]) sh.poison[seg % 3][r] = 1;
#pragma unroll 4
            for (int i = lane; i < 2 * kDim; i += 32) {       // sixteen tokens of a coordinate
              const uint32_t tokens = gone >> (i >= kDim ? 16 : 0);
              uint4* const p = reinterpret_cast<uint4*>(value + i * 16);
              uint4 u = *p;
              u.x &= bytes_without(tokens), u.y &= bytes_without(tokens >> 4);
              u.z &= bytes_without(tokens >> 8), u.w &= bytes_without(tokens >> 12);
              *p = u;
            }
          }
        }
        ptx::fence_async_shared();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar.p_full[jt & 1]);
        slot += 2;
        if (slot >= P::kSlots) slot -= P::kSlots, slot_phase ^= 1;
      }
      if (!ok) break;
      move_on();
      ok = add_output(jt - 1);
      if (!ok) break;
      // the rows' sums over the four warps: halves of the rows are exchanged until
      // a lane has one
#pragma unroll
      for (int o = 16, k = kRowsPerThread / 2; o >= 4; o >>= 1, k >>= 1)
#pragma unroll
        for (int r = 0; r < k; ++r) {
          const bool upper = lane & o;
          const float theirs = __shfl_xor_sync(0xffffffffu, upper ? sum[r] : sum[r + k], o);
          sum[r] = (upper ? sum[r + k] : sum[r]) + theirs;
        }
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
      if ((lane & 3) == 0) sh.sum[seg & 1][warp][(lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)] = sum[0];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bar.sums);
      ok = TQ_WARP_WAIT(bar.sums, seg & 1);
      if (!ok) break;
      if (tid < RT) sh.poison[(seg + 2) % 3][tid] = 0;        // (read by all before they came here)
      // (a run's first item may have begun in the run before, its last may go on)
      const bool whole = tile0 == 0 && reached == tiles;
      float* const part = a.part + (2ll * blockIdx.x + (tile0 == 0 ? 1 : 0)) * part_floats(RT);
      // a lane has a row's sum and vector (token x query head), and gives them to all
      const int mine = lane & (kRowsPerThread - 1);
      float all = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) all += sh.sum[seg & 1][4 * split + w][mine];
      if (sh.poison[seg % 3][split * kRowsPerThread + mine] != 0) all = __int_as_float(0x7fc00000);
      const int live = min(kRowsPerThread, n * a.group - first);
      if (whole) {
        const float inv = all == 0.f ? 0.f : __fdividef(1.f, kWeightScale * all);
        const int vec = static_cast<int>(row_vector(a, row0, kvh, first + mine));   // (n_tokens x n_q is an int)
#pragma unroll
        for (int r = 0; r < kRowsPerThread; ++r) {
          const float by = __shfl_sync(0xffffffffu, inv, r);
          const int to = __shfl_sync(0xffffffffu, vec, r);
          if (r < live) static_cast<__nv_bfloat16*>(a.out)[static_cast<long long>(to) * kDim + token] = __float2bfloat16_rn(acc[r] * by);
        }
      } else {
        float* const rows = part + split * kRowsPerThread * kDim + token;
        float2* const stats = reinterpret_cast<float2*>(part + RT * kDim) + split * kRowsPerThread;
#pragma unroll
        for (int r = 0; r < kRowsPerThread; ++r) {
          const float total = __shfl_sync(0xffffffffu, all, r);
          if (r < live) rows[r * kDim] = acc[r];
          if (r < live && token == 0) stats[r] = make_float2(ref[r], total);
        }
      }
    }
  } else if (warp == P::kSoftWarps) {
    // ---------------- products ----------------
    // the whole warp walks the tiles and waits; an elected lane issues
    const uint32_t ring = ptx::smem_u32(smem);
    const uint64_t key_desc = ptx::desc_k_plain(ring, 128, 1024), value_desc = ptx::desc_k_plain(ring, 2048, 128);
    const uint64_t query_desc = ptx::desc_k_plain(ptx::smem_u32(query_s), P::kQueryCols * 16, 128);
    const uint64_t weight_desc = ptx::desc_k_plain(ptx::smem_u32(weight_s), P::kWeightStride, 128);
    constexpr uint32_t kScores = ptx::idesc_e4m3_f32(kTile, P::kQueryCols), kOutput = ptx::idesc_e4m3_f32(kDim, P::kWeightCols);
    int seg = 0, left = more ? walk.span() : 0;   // of the next scores: segment, its tiles to come
    int k_slot = 0, k_phase = 0, v_slot = 1, v_phase = 0;
    bool fresh = true;                            // the segment's first scores
    auto scores = [&](int j) {
      if (fresh && !TQ_WARP_WAIT(bar.q_full[seg & 1], (seg >> 1) & 1)) return false;
      if (!TQ_WARP_WAIT(bar.full[k_slot], k_phase)) return false;
      fresh = --left == 0;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        const uint64_t k = key_desc + k_slot * (kSlotBytes / 16), q = query_desc + (seg & 1) * (P::kQueryBytes / 16);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          ptx::mma_e4m3(scores_t + (j & 1) * P::kQueryCols, k + ks * 16, q + ks * 2 * P::kQueryCols, kScores, ks > 0);
        // (a test of the bounded waits: the CTA with the first key tile)
        if (!(a.debug_withhold && blockIdx.x == kItemCost / per && j == 0)) ptx::mma_commit(&bar.s_full[j & 1]);
        ptx::mma_commit(&bar.empty[k_slot]);
      }
      __syncwarp();
      k_slot += 2;
      if (k_slot >= P::kSlots) k_slot -= P::kSlots, k_phase ^= 1;
      if (fresh) {
        ++seg;
        more = walk.next(a);
        if (more) left = walk.span();
      }
      return true;
    };
    ok = !more || scores(0);
    bool work = left > 0 || seg > 0;              // (a run without work has no tile)
    for (int j = 0; work && ok; ++j) {
      work = more;
      const bool later = fresh;                   // (a segment's queries come after the one before is done)
      if (work && !later) ok = scores(j + 1);
      ok = ok && TQ_WARP_WAIT(bar.full[v_slot], v_phase) && TQ_WARP_WAIT(bar.p_full[j & 1], (j >> 1) & 1);
      if (!ok) break;
      const uint32_t groups = sh.info[j & (kMetaRing - 1)].groups;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        const uint64_t v = value_desc + v_slot * (kSlotBytes / 16), w = weight_desc + (j & 1) * (P::kWeightBytes / 16);
        bool added = false;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (!(groups >> g & 1u)) continue;
          ptx::mma_e4m3(outputs_t, v + g * (kGroupBytes / 16), w + g * 2 * (P::kWeightStride / 16),
                        kOutput, added);
          added = true;
        }
        ptx::mma_commit(&bar.o_full[j & 1]);
        ptx::mma_commit(&bar.empty[v_slot]);
      }
      __syncwarp();
      v_slot += 2;
      if (v_slot >= P::kSlots) v_slot -= P::kSlots, v_phase ^= 1;
      if (work && later) ok = scores(j + 1);
    }
    if (ptx::elect_one()) {
      ptx::mma_commit(&bar.drain);                // nothing is in flight when the CTA ends
      ptx::drain_bar(&bar.drain, 0);
    }
  } else {
    // ---------------- copies ----------------
    // lane g < 4 has the tile's group g; its block id is read a tile ahead
    int slot = 0, phase = 1, issued = 0;
    int t = more ? walk.tile : 0, reached = more ? t + walk.span() : 0;
    struct Group {
      int off, id, kvh;
      bool here;
    };
    auto read_id = [&]() {                        // of tile t of the walk's item
      Group g{0, -1, walk.kvh, false};
      const int pos = t * kTile + 32 * lane;
      if (lane < 4 && pos < walk.s.ctx) {
        const int col = pos / c.block_size;
        g.off = pos - col * c.block_size;
        const long long at = static_cast<long long>(walk.b) * c.max_blocks + col;
        g.id = c.block_table ? __ldg(c.block_table + at) : static_cast<int>(at);
        g.here = true;
      }
      return g;
    };
    auto fill = [&](const uint8_t* src, uint32_t bytes) {   // the next slot; false when its wait ran out
      if (!TQ_WARP_WAIT(bar.empty[slot], phase)) return false;
      if (lane == 0) ptx::mbar_arrive_expect_tx(&bar.full[slot], bytes);
      __syncwarp();
      if (src != nullptr) ptx::bulk_load(smem + slot * kSlotBytes + lane * kGroupBytes, src, kGroupBytes, &bar.full[slot]);
      return true;
    };
    auto step = [&]() {
      ++issued;
      if (++slot == P::kSlots) slot = 0, phase ^= 1;
    };
    CutItem cut{0, 0, 0, 0, 0};
    auto begin = [&]() {                          // of an item
      // (the queries come from far memory, and a segment begins with them)
      const int rows = min(RT, walk.s.n * a.group - walk.rt * RT), lines = QP == 2 ? 2 : 4;   // of 128 bytes
      for (int k = lane; k < rows * lines; k += 32) {
        const long long vec = row_vector(a, walk.s.row0, walk.kvh, walk.rt * RT + k / lines);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.q) + (vec * lines + k % lines) * 128));
      }
      // what the run begins and does not end, for the join
      if (walk.tile == 0 && walk.span() < walk.tiles)
        cut = CutItem{walk.s.row0, walk.kvh, walk.rt, rows,
                      static_cast<int>((walk.pos + walk.tiles - 1) / per)};
    };
    Group now{};
    if (more) now = read_id(), begin();
    for (int j = 0; more; ++j) {
      if (++t == reached) {
        more = walk.next(a);
        if (more) begin();
        if (more) t = walk.tile, reached = t + walk.span();
      }
      Group ahead{};
      if (more) ahead = read_id();
      bool there = now.here;
      if (there && (now.id < 0 || now.id >= c.num_blocks)) {
        atomicCAS(c.error, 0, kErrBlock);
        there = false;
      }
      const long long vec = static_cast<long long>(now.id) * c.n_kv + now.kvh;
      const long long byte = (vec * c.block_size + now.off) * kDim;
      const uint32_t groups = __ballot_sync(0xffffffffu, there), bytes = __popc(groups) * kGroupBytes;
      // (the tile sixteen before is done: its slots have been filled again since)
      TileInfo& info = sh.info[j & (kMetaRing - 1)];
      ok = fill(there ? c.k + byte : nullptr, bytes);
      if (!ok) break;
      if (lane < 4) ptx::mbar_arrive(&bar.full[slot]);
      step();
      if (lane == 0) info.groups = groups;
      if (there) {
        copy4_async(&info.k_scale[lane], c.k_scale + vec);
        copy4_async(&info.v_scale[lane], c.v_scale + vec);
      }
      __syncwarp();
      ok = fill(there ? c.v + byte : nullptr, bytes);
      if (!ok) break;
      if (lane < 4) arrive_copies(&bar.full[slot]);
      step();
      now = ahead;
    }
    if (lane == 0) a.cuts[blockIdx.x] = cut;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (*abort && lane == 0)                      // copies in flight land before the CTA ends
      for (int i = max(0, issued - P::kSlots); i < issued; ++i) ptx::drain_bar(&bar.full[i % P::kSlots], (i / P::kSlots) & 1);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == P::kSoftWarps) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, P::kTmem);
  }
}

// Joins the partial outputs of a row tile: sum_s 2^{m_s - M} o_s over
// sum_s 2^{m_s - M} l_s.  Block (x, y) joins four rows, or one, of the item that
// run x begins and does not end: a warp a row, or four of which each takes every
// fourth part; four coordinates a lane.  (One warp, four warps: eight items of 38
// parts 51.3, 49.1 us; 24 sequences of drafted tokens, up to four parts each, 100.5,
// 103; one short context 7.8, 8.2.  Eight parts at once, which spill, in place of
// four: 49.0 us for 48.4, 99.8 for 99.0.)
constexpr int kJoinThreads = 128, kJoinAtOnce = 4;   // parts that a warp reads at a time
template <int kJoinWarps>
__global__ void __launch_bounds__(kJoinThreads, 8) fp8_join_kernel(Fp8AttendArgs a, int rt_rows) {
  constexpr int kJoinRows = kJoinThreads / 32 / kJoinWarps;
  __shared__ float4 acc_s[kJoinRows][kJoinWarps][32];
  __shared__ float sum_s[kJoinRows][kJoinWarps], top_s[kJoinRows][kJoinWarps];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % kJoinWarps, mine = (threadIdx.x >> 5) / kJoinWarps;
  const int row = blockIdx.y * kJoinRows + mine, c0 = blockIdx.x;
  wait_prerequisites();
  const CutItem cut = a.cuts[c0];
  if (static_cast<int>(blockIdx.y) * kJoinRows >= cut.rows) return;      // (the whole CTA)
  const bool live = row < cut.rows;
  // (the run that holds key tile 0 wrote its second slot, the others their first)
  auto part = [&](int s) { return a.part + (2ll * s + (s == c0 ? 1 : 0)) * part_floats(rt_rows); };
  const int stats = rt_rows * kDim + 2 * row;
  // one pass: four parts' reads at once, the reference raised as they come
  float top = kNothing, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = c0 + warp; live && s0 <= cut.last; s0 += kJoinAtOnce * kJoinWarps) {
    float2 ml[kJoinAtOnce];
    float4 o[kJoinAtOnce];
#pragma unroll
    for (int k = 0; k < kJoinAtOnce; ++k) {
      const int s = s0 + k * kJoinWarps;
      ml[k] = make_float2(kNothing, 0.f);
      o[k] = acc;
      if (s <= cut.last) {
        ml[k] = *reinterpret_cast<const float2*>(part(s) + stats);
        o[k] = reinterpret_cast<const float4*>(part(s) + row * kDim)[lane];
      }
    }
    float to = top;
#pragma unroll
    for (int k = 0; k < kJoinAtOnce; ++k) to = fmaxf(to, ml[k].x);
    const float keep = exp2_fast(top - to);
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep, sum *= keep;
    top = to;
#pragma unroll
    for (int k = 0; k < kJoinAtOnce; ++k) {
      if (ml[k].y == 0.f) continue;               // (a part that saw nothing)
      const float w = exp2_fast(ml[k].x - top);
      acc.x = fmaf(w, o[k].x, acc.x), acc.y = fmaf(w, o[k].y, acc.y), acc.z = fmaf(w, o[k].z, acc.z);
      acc.w = fmaf(w, o[k].w, acc.w);
      sum = fmaf(w, ml[k].y, sum);
    }
  }
  acc_s[mine][warp][lane] = acc;
  if (lane == 0) sum_s[mine][warp] = sum, top_s[mine][warp] = top;
  __syncthreads();
  if (warp != 0 || !live) return;
  float to = top;
  for (int w = 1; w < kJoinWarps; ++w) to = fmaxf(to, top_s[mine][w]);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float4 o = acc_s[mine][w][lane];
    const float f = exp2_fast(top_s[mine][w] - to);
    acc.x = fmaf(f, o.x, acc.x), acc.y = fmaf(f, o.y, acc.y), acc.z = fmaf(f, o.z, acc.z), acc.w = fmaf(f, o.w, acc.w);
    sum = fmaf(f, sum_s[mine][w], sum);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / (kWeightScale * sum);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  const long long vec = row_vector(a, cut.row0, cut.kvh, cut.i * rt_rows + row);
  reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + vec * kDim)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Rows of a row tile: 16 where the average sequence of the call has more than
// eight.  (16 sequences on 8192 tokens, 64/8 heads, 8 rows each: 52 us with
// eight a tile, 59 with 16; 16 rows: 91 and 58; 32 rows: 165 and 109.  With 32
// rows a tile and one CTA an SM 16 rows take 87 us and 32 rows 109; with four
// warps that turn the tiles into fp16 operands, which need no pieces, 105 and
// 135: then one chain of waits, exponentials and stores is all an SM has to do.)
int tile_rows(int n_tokens, int batch, int group) {
  return (static_cast<long long>(n_tokens) + batch - 1) / batch * group <= 8 ? 8 : 16;
}

// Rows from which a sequence takes the wide form (extend_wide.cu over tiles
// that fp8_wide.cu expands).  (Wide | few, us: 16 sequences on 8192 tokens, 64/8
// heads, 64 rows 381 | 184, 128 rows 385 | 344 (380 in float32), 256 rows 396 | 800; one on 32000,
// 128 rows 130 | 100; 8 on 2000, 32/8 heads, 128 rows 82 | 78.)
constexpr int kWideFrom = 144;
// Whether a call has the wide form's launches: if one sequence can have the rows,
// and if the call would lose more without them than they take, 9 us where there
// is no such sequence.  What it can lose goes with the products of tokens, query
// heads and context: this form does 0.3 to 0.4 million of them in a microsecond.
// A sequence has the rows if the others have a token each; or, as sequences
// may be empty, if it has all tokens.  A call that can have it only so is nearly
// always a decode step, whose contexts may be far shorter than max_context: such
// a call has the launches from 512 tokens on, and where they are 1 % of a decode
// step with contexts of max_context.
// (64/8 heads, us, with the launches | without.  A sequence of 2048 tokens on 16 K
// among 2048 854 | 7326, one of 256 on 8192 among 256 117 | 472, one of 64 on
// 8192 among 64 77 | 125.  Decode steps: 64 on 1 K to 32 K 321 | 312, 256 on 8192
// 630 | 621, 128 on 700 54 | 47.)
constexpr long long kWideWork = 1 << 22, kWideWorkIdle = 1 << 28;
constexpr int kWideTokensIdle = 512;
bool wide_possible(int n_tokens, int batch, int n_q, int n_kv, int max_context) {
  const long long context = max_context > 0 ? max_context : 1;
  auto gains = [&](long long most, long long work) { return most * (n_q / n_kv) >= kWideFrom && most * n_q >= work / context; };
  return gains(static_cast<long long>(n_tokens) - batch + 1, kWideWork) ||
         (n_tokens >= kWideTokensIdle && gains(n_tokens, kWideWorkIdle));
}

// `planned`: launches of the same call come before.
template <int RT, int QP>
cudaError_t attend(const Fp8AttendArgs& a, bool planned, cudaStream_t stream) {
  using P = Shape<RT, QP>;
  const cudaError_t err = cudaFuncSetAttribute(fp8_attend_kernel<RT, QP>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (err != cudaSuccess) return err;
  const int ctas = kCtasPerSm * a.num_sms;
  if (planned) return launch_dependent(fp8_attend_kernel<RT, QP>, dim3(ctas), P::kThreads, P::kSmem, stream, a);
  fp8_attend_kernel<RT, QP><<<ctas, P::kThreads, P::kSmem, stream>>>(a);
  return cudaGetLastError();
}

struct Layout {
  size_t part, wide, total;
};
Layout layout(int n_tokens, int batch, int n_q, int n_kv, int max_context, int num_sms) {
  const int rt = tile_rows(n_tokens, batch, n_q / n_kv), ctas = num_sms * kCtasPerSm;
  Layout l;
  l.part = align256(ctas * sizeof(CutItem));
  l.wide = l.part + align256(2ull * ctas * part_floats(rt) * sizeof(float));
  l.total = l.wide;
  if (wide_possible(n_tokens, batch, n_q, n_kv, max_context))
    l.total += extend_wide_workspace_bytes(n_tokens, batch, n_q, n_kv, max_context, num_sms, kWideFrom);
  return l;
}

}  // namespace

size_t fp8_workspace_bytes(int n_tokens, int batch, int n_q, int n_kv, int max_context, int num_sms) {
  return layout(n_tokens, batch, n_q, n_kv, max_context, num_sms).total;
}

cudaError_t launch_fp8_attention(const Fp8AttendArgs& args, void* workspace, cudaStream_t stream) {
  Fp8AttendArgs a = args;
  const Fp8Cache& c = a.c;
  char* const ws = static_cast<char*>(workspace);
  const Layout l = layout(c.n_tokens, c.batch, a.n_q, c.n_kv, a.max_context, a.num_sms);
  a.cuts = reinterpret_cast<CutItem*>(ws);
  a.part = reinterpret_cast<float*>(ws + l.part);
  const int rt = tile_rows(c.n_tokens, c.batch, a.group);
  auto few = [&](bool planned) { 
    if (a.q_bf16) return rt == 8 ? attend<8, 2>(a, planned, stream) : attend<16, 2>(a, planned, stream);
    return rt == 8 ? attend<8, 4>(a, planned, stream) : attend<16, 4>(a, planned, stream);
  };
  auto join = [&]() {
    // parts of an item: as many as it has CTAs on average, or key tiles
    const long long ctas = kCtasPerSm * a.num_sms, items = static_cast<long long>(c.batch) * c.n_kv;
    const bool one = std::min(ctas / items, static_cast<long long>(a.max_context / kTile)) < 2 * kJoinAtOnce;
    return one ? launch_dependent(fp8_join_kernel<1>, dim3(ctas, rt / 4), kJoinThreads, 0, stream, a, rt)
               : launch_dependent(fp8_join_kernel<4>, dim3(ctas, rt), kJoinThreads, 0, stream, a, rt);
  };
  cudaError_t err = cudaSuccess;
  if (l.total > l.wide) {
    // some sequence may have the rows for the wide form
    ExtendArgs e{};
    e.d.q = a.q;
    e.d.batch = c.batch;
    e.d.n_q = a.n_q;
    e.d.n_kv = c.n_kv;
    e.d.group = a.group;
    e.d.block_size = c.block_size;
    e.d.max_blocks = c.max_blocks;
    e.d.context_lens = c.context_lens;
    e.d.max_context = a.max_context;
    e.d.error = c.error;
    e.d.num_sms = a.num_sms;
    e.d.debug_withhold = a.debug_withhold;
    e.n_tokens = c.n_tokens;
    e.query_start = c.query_start;
    e.out = a.out;
    e.q_bf16 = a.q_bf16;
    e.query_top = 15;                             // coordinates below 2^15 are fp16 numbers as they are
    e.wide_from = kWideFrom;
    // Where the rows alone say which sequences those are, the others go first and
    // the plan runs beside them (24 sequences of 1 to 8 tokens: 109 us after it).
    const bool first = extend_wide_fits(c.n_tokens, c.batch, a.n_q, c.n_kv, a.max_context, a.num_sms, kWideFrom);
    if (first) {
      a.wide_from = kWideFrom;
      err = few(false);
    }
    if (err == cudaSuccess) err = launch_extend_wide_plan(e, ws + l.wide, first, stream);
    if (err == cudaSuccess) err = launch_fp8_expand(c, e, a.scale, stream);
    if (err == cudaSuccess) err = launch_extend_wide(e, false, a.num_sms, stream);
    if (err == cudaSuccess) err = launch_extend_wide_join(e, stream);
    if (err == cudaSuccess && !first) {
      a.seq = e.ws_seq;
      err = few(true);
    }
  } else {
    err = few(false);
  }
  return err == cudaSuccess ? join() : err;
}

}  // namespace tq
