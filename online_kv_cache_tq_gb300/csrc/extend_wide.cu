// The wide form of the multi-token attention: sequences with many rows.
//
// extend_expand_kernel turns every key tile (128 tokens of a KV head) of such
// a sequence into two operands, once: the keys back in the original space,
//   k_t = R^T c[code_t] + rho_t S^T (2 bits_t - 1)       (unit norm, fp16),
// products on the tensor cores of the expanded bits with R^T and S^T, joined by
// rho_t in fp32, and the
// value levels c^v[code_t] (rotated space, bf16).  They are stored in the
// swizzled layout the products read, 64 KB a tile, so that a tile is two bulk
// copies later.  Per token and KV head this costs 66 K operations and writes
// 520 bytes; it saves every row tile the expansion and half of the score
// product (128 columns in place of 256 with the sketch).
//
// extend_wide_kernel then works on row tiles of 256: two products of 128 rows
// take turns, so that the softmax of one runs under the products of the other.
//   scores  [128 x 128] = q k^T, fp16, queries in shared memory as they come
//           (scaled by a power of two outside 2^-8 .. 2^query_top);
//   output  [128 x 128] += p n^v c, bf16, weights in tensor memory over the scores;
// the last step turns the output back by R^T.  The softmax is that of the
// narrow form (extend_tc.cu: its reference, and when a tile may skip the
// search for its maximum).  The bound of the loop is the tensor cores: 2304
// cycles of products for 256 x 128 scores (256 of them for the remainders), plus twice the time from a
// product's end to the issue of the one that overwrites its operand.
//
// Measured.  2048 tokens on 14001, 64/8 heads: 750 us, 1.34 PFLOP/s, 3.6 K
// cycles for 256 x 128 scores, tensor pipe 64 % busy; expansion 31 us.  Short
// items cost 13 K cycles outside the loop (ragged prompts up to 4096 tokens,
// 32/8 heads: 249 us, 0.86 PFLOP/s; expansion 25 us).  Queries held in
// registers from one reading to the next spill into the loop (310 against 287
// us for those prompts, 852 against 753 us for the 2048 tokens).
//
// Eighteen warps: 0-7 and 8-15 the softmax of the two row tiles (two threads
// per row), 16 issues the products, 17 copies tiles.
#include "extend_common.cuh"

namespace tq {
namespace {

#define TQ_WAIT(b, ph) ptx::wait_bar(&(b), (ph), abort, d.error, kErrTimeout)
#define TQ_WARP_WAIT(b, ph) __all_sync(0xffffffffu, TQ_WAIT(b, ph))

// ---- expansion -----------------------------------------------------------------

// Two groups of 256 threads with a tile each, around one copy of R^T and S^T.
constexpr int kGroupThreads = 256;
constexpr int kExpandThreads = 2 * kGroupThreads;
constexpr int kExpandKey0 = 2 * kExtendImageBytes;
constexpr int kExpandSmem = kExpandKey0 + 2 * 4 * kBlockBytes + 1024; // (1024: alignment)

// Barrier of one group that also ORs a flag over it.
__device__ __forceinline__ bool group_sync(int group, bool flag) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(flag)), "r"(group + 1), "n"(kGroupThreads)
      : "memory");
  return r != 0;
}

// Bulk copy shared -> global, and the waits until its reads and its writes are done.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
               ::"l"(reinterpret_cast<uint64_t>(dst)), "r"(ptx::smem_u32(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// What a group's threads share about their tile.
struct ExpandShared {
  float factor[kTile], rho[kTile], norm[kTile], square[2][kTile], reach[4];
  uint32_t valid[4];
  uint64_t done, drain;
};

template <int KB, int VB>
__global__ void __launch_bounds__(kExpandThreads, 1) extend_expand_kernel(ExtendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExpandShared group_s[2];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  uint8_t* const smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const DecodeArgs& d = a.d;
  const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x % kGroupThreads;
  const int warp = tid >> 5, lane = tid & 31;     // of the group
  ExpandShared& sh = group_s[group];
  volatile int* const abort = &abort_s;
  launch_dependents();
  wait_prerequisites();
  const long long total = a.ws_expand[d.batch];
  if (2ll * blockIdx.x >= total) return;          // (the whole CTA)
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (ExpandShared& s : group_s) {
      ptx::mbar_init(&s.done, 1);
      ptx::mbar_init(&s.drain, 1);
    }
    ptx::fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    ptx::tmem_alloc(&tmem_s, 512);
    ptx::tmem_relinquish();
  }
  const bool qjl = d.k_qjl != nullptr;
  {                                               // R^T and S^T
    const uint4* const src = a.images + 3 * (kExtendImageBytes / 16);
    uint4* const dst = reinterpret_cast<uint4*>(smem);
#pragma unroll 8
    for (int i = threadIdx.x; i < 2 * (kExtendImageBytes / 16); i += kExpandThreads) dst[i] = __ldg(src + i);
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_s + 256 * group;           // R^T c, then S^T signs
  uint8_t* const keys_s = smem + kExpandKey0 + group * 4 * kBlockBytes;
  const int row = tid & (kTile - 1), half = tid / kTile;   // key row or value coordinate; half of the other side
  const LevelBytes key_levels = level_bytes<false>(d.tables->k_fp16, KB);
  const LevelBytes value_levels = level_bytes<true>(d.tables->v_bf16, VB);
  const float value_scale = d.tables->v_bf16_scale;
  const float to_log2 = d.scale * 1.4426950408889634f;
  // (the first two warps of a half read its 64 value norms, by expanded column)
  const int mine = row < 64 ? row >> 5 : -1;
  RawKey<KB> next_key;
  RawValue<VB> next_value;
  auto load_tile = [&](long long g) {             // the packed words of tile g
    int lo = 0, hi = d.batch;                     // the last sequence whose tiles start at or before g
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.ws_expand[mid] <= g) lo = mid;
      else hi = mid;
    }
    Item it{};
    it.b = lo;
    it.seq = a.ws_seq[lo];
    const int tiles = max(1, (it.seq.z + kTile - 1) / kTile), local = static_cast<int>(g - a.ws_expand[lo]);
    it.kvh = local / tiles;
    const int pos0 = (local - it.kvh * tiles) * kTile;
    Cursor kc, vc;
    start_cursor(d, it, pos0 + (row & ~31), kc);
    start_cursor(d, it, pos0 + 64 * half + 32 * (lane & 1), vc);
    load_key(d, it, kc, expanded_bit(lane), half, next_key);
    load_value(d, it, vc, row, mine, expanded_bit(lane), next_value);
  };
  const long long g0 = 2ll * blockIdx.x + group, step = 2ll * gridDim.x;
  if (g0 < total) load_tile(g0);
  uint32_t phase = 0;
  for (long long g = g0; g < total; g += step, phase ^= 1) {
    uint8_t* const out = a.ws_tiles + g * kTileImageBytes;
    TileMeta* const meta = a.ws_meta + g;
    const RawKey<KB> k = next_key;
    const RawValue<VB> v = next_value;
    if (g + step < total) load_tile(g + step);
    {
      const RowChunks at = row_chunks(ptx::smem_u32(keys_s) + half * kBlockBytes, row);
      uint32_t w0[KB], w1[KB];
#pragma unroll
      for (int p = 0; p < KB; ++p) w0[p] = k.planes[p].x, w1[p] = k.planes[p].y;
      expand32<KB, 0>(at, w0, key_levels);
      expand32<KB, 0>(second_word(at), w1, key_levels);
      if (qjl) {
        constexpr uint32_t kMinusOne = 0xbc00bc00u;
        if (half == 0) sh.rho[row] = k.norm > 0.f ? __fdividef(k.rnorm * d.qjl_coef, k.norm) : 0.f;
        expand_signs<2 * kBlockBytes>(at, k.qjl.x, kMinusOne);
        expand_signs<2 * kBlockBytes>(second_word(at), k.qjl.y, kMinusOne);
      }
    }
    if (half == 0) {
      const unsigned bit = __reduce_or_sync(0xffffffffu, k.valid ? 1u << expanded_bit(lane) : 0u);
      sh.factor[row] = k.valid ? k.norm * to_log2 : 0.f;
      if (lane == 0) sh.valid[warp] = bit;
    }
    if (mine >= 0) sh.norm[64 * half + row] = v.norm * value_scale;
    ptx::fence_async_shared();
    group_sync(group, false);
    if (warp == 0 && ptx::elect_one()) {
      ptx::tc_fence_after();
      const uint64_t keys = ptx::desc_k_sw128(ptx::smem_u32(keys_s));
      const uint64_t turn = ptx::desc_k_sw128(ptx::smem_u32(smem));
#pragma unroll
      for (int ks = 0; ks < 16; ++ks) {
        const uint64_t off = (ks >> 2) * (kBlockBytes / 16) + (ks & 3) * 2;
        if (ks < 8 || qjl) ptx::mma_bf16(tmem + (ks < 8 ? 0 : 128), keys + off, turn + off, kIdescF16, (ks & 7) > 0);
      }
      // (a test of the bounded waits: the first tile)
      if (!(d.debug_withhold && blockIdx.x == 0 && g == g0)) ptx::mma_commit(&sh.done);
    }
    __syncwarp();
    const bool ok = TQ_WAIT(sh.done, phase);
    if (group_sync(group, !ok)) break;
    // the product has read its operand: the tile's image takes its place
    {
      const RowChunks at = row_chunks(ptx::smem_u32(keys_s + kExtendImageBytes) + half * kBlockBytes, row);
      uint32_t w0[VB], w1[VB];
#pragma unroll
      for (int p = 0; p < VB; ++p) w0[p] = v.words[p][0], w1[p] = v.words[p][1];
      expand32<VB, 0>(at, w0, value_levels);
      expand32<VB, 0>(second_word(at), w1, value_levels);
    }
    ptx::tc_fence_after();
    {
      const int r = (warp & 3) * 32 + lane, h = warp >> 2;   // tensor-memory lane, columns 64 h .. + 63
      const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 64 * h;
      const float rho = qjl ? sh.rho[r] : 0.f;
      float square = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t y[16], z[16] = {}, w[8];
        ptx::tmem_ld16(at + 16 * c, y);
        if (qjl) ptx::tmem_ld16(at + 128 + 16 * c, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f0 = fmaf(rho, __uint_as_float(z[2 * e]), __uint_as_float(y[2 * e]));
          const float f1 = fmaf(rho, __uint_as_float(z[2 * e + 1]), __uint_as_float(y[2 * e + 1]));
          square = fmaf(f0, f0, fmaf(f1, f1, square));
          w[e] = pack_f16(f0, f1);
        }
        uint8_t* const dst = keys_s + h * kBlockBytes + r * 128;
        *reinterpret_cast<uint4*>(dst + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(dst + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
      }
      sh.square[h][r] = square;
    }
    ptx::tc_fence_before();
    ptx::fence_async_shared();
    group_sync(group, false);
    if (tid == 0) bulk_store(out, keys_s, kTileImageBytes);     // (in whole lines)
    if (tid < kTile) {
      const float f = sh.factor[tid];
      meta->key_factor[tid] = f;
      meta->value_factor[tid] = sh.norm[tid];
      const float reach = fabsf(f) * sqrtf(sh.square[0][tid] + sh.square[1][tid]);
      const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(reach) & 0x7fffffffu);   // (not negative)
      if (lane == 0) {
        sh.reach[warp] = __uint_as_float(bits);
        meta->valid[warp] = sh.valid[warp];
      }
    }
    group_sync(group, false);
    if (tid == 0) {
      // (a NaN has the largest bits, and takes the path that looks at every score)
      unsigned bits = 0;
      for (int w = 0; w < 4; ++w) bits = max(bits, __float_as_uint(sh.reach[w]));
      meta->reach = __uint_as_float(bits);
    }
    if (tid == 0) bulk_store_wait();
    group_sync(group, false);                     // (the next tile overwrites what was read)
  }
  if (tid == 0) bulk_store_done();                // nothing is in flight when the CTA ends, also after a wait ran out
  __syncwarp();
  if (warp == 0 && ptx::elect_one()) {
    ptx::mma_commit(&sh.drain);
    ptx::drain_bar(&sh.drain, 0);
  }
  __syncwarp();
  __syncthreads();
  if (threadIdx.x < 32) ptx::tmem_dealloc(tmem_s, 512);
}

// ---- attention -------------------------------------------------------------------

constexpr int kSoftThreads = 512;
constexpr int kMmaWarp = 16;
constexpr int kCopyWarp = 17;
constexpr int kWideThreads = kSoftThreads + 64;
constexpr int kImage = kExtendImageBytes;
constexpr int kQuery0 = 0;                        // two row tiles
constexpr int kKey0 = 2 * kImage;                 // two stages
constexpr int kValue0 = 4 * kImage;               // two stages
constexpr int kMeta0 = 6 * kImage;                // four
constexpr int kRing = 4;
constexpr int kWideSmem = kMeta0 + kRing * static_cast<int>(sizeof(TileMeta)) + 1024;   // (1024: alignment)
static_assert(sizeof(TileMeta) % 16 == 0, "bulk copies are multiples of 16 bytes");
constexpr uint32_t kS = 0, kO = 256;              // tensor-memory columns, 128 for each row tile

struct WideBarriers {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], added[2], o_raw[2], turned[2];   // by row tile
  uint64_t q_full, drain;
  uint64_t rows[8];          // the two warps that share 32 rows
};

__global__ void __launch_bounds__(kWideThreads, 1) extend_wide_kernel(ExtendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ WideBarriers bar;
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  __shared__ Item item_s;
  __shared__ int offset_s;
  __shared__ float swap_s[2][2][kWideRows];       // what the two threads of a row tell each other
  __shared__ float2 query_s[2][kWideRows];        // largest coordinate and squared length of half a row's query
  uint8_t* const smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const DecodeArgs& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* const abort = &abort_s;
  launch_dependents();
  wait_prerequisites();
  const long long total = a.wide.first[d.batch];
  const long long per = run_length(total, gridDim.x);
  Run run;
  run.pos = blockIdx.x * per;
  run.end = run.pos + per < total ? run.pos + per : total;
  if (run.pos >= run.end) {                       // (the whole CTA)
    if (threadIdx.x == 0) write_cut(a, a.wide, run, per, false);
    return;
  }

  if (tid == 0) {
    abort_s = 0;
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bar.k_full[s], 1);
      ptx::mbar_init(&bar.k_empty[s], 1);
      ptx::mbar_init(&bar.v_full[s], 1);
      ptx::mbar_init(&bar.v_empty[s], 1);
      ptx::mbar_init(&bar.s_full[s], 2);          // the product's completion and the issuer itself
      ptx::mbar_init(&bar.p_full[s], kSoftThreads / 2);
      ptx::mbar_init(&bar.added[s], 1);
      ptx::mbar_init(&bar.o_raw[s], kSoftThreads / 2);
      ptx::mbar_init(&bar.turned[s], 1);
    }
    ptx::mbar_init(&bar.q_full, kSoftThreads);
    ptx::mbar_init(&bar.drain, 1);
    for (int w = 0; w < 8; ++w) ptx::mbar_init(&bar.rows[w], 64);
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&tmem_s, 512);
    ptx::tmem_relinquish();
  }
  if (warp == 0) {
    int offset;
    const Item it = find_item(a, a.wide, run.pos, &offset);
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
  bool ok = true;

  if (warp < 16) {
    // ---------------- softmax ----------------
    const int x = warp >> 3, quarter = warp & 3, half = (warp >> 2) & 1;
    const int row = quarter * 32 + lane;          // of row tile x: tensor-memory lane; columns 64 half .. + 63
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_addr = lane_addr + kS + 128 * x + 64 * half, o_addr = lane_addr + kO + 128 * x + 64 * half;
    uint64_t* const pair_bar = &bar.rows[4 * x + quarter];
    int swaps = 0;
    auto meet = [&]() {                           // the row's two threads (their warps)
      ptx::mbar_arrive(pair_bar);
      return TQ_WARP_WAIT(*pair_bar, swaps++ & 1);
    };
    auto swap = [&](float mine, float* theirs) {  // the other thread of the row: its value of `mine`
      float(*const buf)[kWideRows] = swap_s[swaps & 1];
      buf[half][kTile * x + row] = mine;
      const bool done = meet();
      *theirs = buf[half ^ 1][kTile * x + row];
      return done;
    };
    // A warp copies queries and outputs between memory and shared memory for its
    // own rows and columns only, eight lanes to the 128 bytes of half a row: rows
    // copy_row, copy_row + 4, .. + 28, 16 bytes of each.
    const int copy_row = 32 * quarter + (lane >> 3), copy_chunk = lane & 7;
    uint8_t* const half_s = smem + kQuery0 + x * kImage + half * kBlockBytes;
    auto swizzled = [&](int qr, int chunk) { return reinterpret_cast<uint4*>(half_s + qr * 128 + (((chunk ^ qr) & 7) << 4)); };
    int jt = 0;                                   // key tiles so far
    for (int seg = 0; next_segment(a, a.wide, run, t0, t1); ++seg) {
      const int n_rows = it.seq.y * d.group;
      const int r = it.i * kWideRows + kTile * x + row;
      const bool live = r < n_rows;
      const int tok = row_token(a, live ? r : n_rows - 1);
      const int seen = max(0, it.seq.z - it.seq.y + tok + 1);     // positions this row sees
      // vector (token x query head) of row rr of the sequence and KV head (below 2^31)
      const uint32_t first_vec = it.seq.x * d.n_q + it.kvh * d.group, other_heads = d.n_q - d.group;
      auto vector_of = [&](int rr) { return static_cast<long long>(first_vec + row_token(a, rr) * other_heads + rr); };
      float other;
      // The queries: fp16, scaled by a power of two if outside the range,
      // swizzled.  bf16 rows are copied to their place first, in whole lines and
      // all in flight at once (a warp copies what it converts), then a thread
      // converts its half of a row where it lies.
      if (a.q_bf16) {
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const int qr = copy_row + 4 * k, rr = it.i * kWideRows + kTile * x + qr;
          const long long vec = vector_of(min(rr, n_rows - 1));
          copy16_async(swizzled(qr, copy_chunk),
                       static_cast<const __nv_bfloat16*>(d.q) + vec * kDim + 64 * half + copy_chunk * 8);
        }
        copies_wait();
        __syncwarp();
      }
      const long long query = vector_of(live ? r : n_rows - 1) * kDim + 64 * half;
      auto query8 = [&](int c, float (&v)[8]) {     // (rows that are not there convert another row's query)
        if (a.q_bf16) unpack_bf16(*swizzled(row, c), v);
        else load_query8(a, query + 8 * c, v);
      };
      float biggest = 0.f;
      uint64_t square2 = 0;                       // (two fp32 zeros)
#pragma unroll 2
      for (int c = 0; c < 8; ++c) {
        float v[8];
        query8(c, v);
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
          biggest = fmaxf(biggest, fmaxf(fabsf(v[q]), fabsf(v[q + 1])));
          square2 = fma2(pair(v[q], v[q + 1]), pair(v[q], v[q + 1]), square2);
        }
      }
      float2 square = unpair(square2);
      square.x += square.y;
      query_s[half][kTile * x + row] = make_float2(biggest, square.x);
      ok = meet();
      if (!ok) break;
      const float2 others = query_s[half ^ 1][kTile * x + row];
      biggest = fmaxf(biggest, others.x);
      const float len = sqrtf(square.x + others.y) * 1.01f;       // (1.01: the operands' roundings)
      int e = exponent_of(biggest);
      if (biggest == 0.f || (e >= -8 && e < a.query_top)) e = 0;
      const float down = exp2_int(-e), factor = exp2_int(e);
#pragma unroll 2
      for (int c = 0; c < 8; ++c) {
        float v[8];
        query8(c, v);
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = pack_f16(v[2 * q] * down, v[2 * q + 1] * down);
        *swizzled(row, c) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      ptx::fence_async_shared();
      ptx::mbar_arrive(&bar.q_full);

      float ref = -INFINITY;
      uint64_t sum2 = 0;                          // (two fp32 zeros)
      for (int t = t0; t < t1; ++t, ++jt) {
        ok = TQ_WARP_WAIT(bar.s_full[x], jt & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const TileMeta* const meta = reinterpret_cast<const TileMeta*>(smem + kMeta0) + (jt & (kRing - 1));
        const float *const kf = meta->key_factor + 64 * half, *const vf = meta->value_factor + 64 * half;
        const uint4 there = *reinterpret_cast<const uint4*>(meta->valid);
        const uint32_t all = there.x & there.y & there.z & there.w, any = there.x | there.y | there.z | there.w;
        // (both the same for the two threads of a row, and so for their warps)
        bool mask = __any_sync(0xffffffffu, e != 0 || seen < (t + 1) * kTile || all != 0xffffffffu);
        const bool search = __any_sync(0xffffffffu, !(len * meta->reach <= (ref == -INFINITY ? 0.f : ref) + kRaise));
        const int here = min(kTile, max(0, seen - t * kTile));
        if (search) {
          // scores that may pass the reference: the tile's maximum first
          const float top = mask ? masked_top(s_addr, kf, factor, meta->valid, here, half) : plain_top(s_addr, kf);
          ok = swap(top, &other);
          if (!ok) break;
          const float to = raised(ref, fmaxf(top, other));
          if (__any_sync(0xffffffffu, to != ref)) {
            const float scale = to != ref ? exp2_fast(ref - to) : 1.f;
            if (t > t0) {
              // the output so far, once the product before has added to it
              ok = TQ_WARP_WAIT(bar.added[x], (jt - 1) & 1);
              if (!ok) break;
              ptx::tc_fence_after();
              sum2 = mul2(sum2, pair(scale, scale));
              scale_output(o_addr, scale);
            }
            ref = to;
          }
          // (a tile that is not searched stays 1 % below a large reference)
          mask = mask || __any_sync(0xffffffffu, fabsf(ref) < INFINITY && fabsf(ref) > kFused);
        } else if (ref == -INFINITY && any != 0) {
          ref = 0.f;                              // scores in bounds, and the row's first tokens (if it sees any here)
        }
        const float shift = ref == -INFINITY ? 0.f : ref;
        if (mask) sum2 = add2(sum2, pair(weigh_masked(s_addr, kf, vf, factor, shift, meta->valid, here, half), 0.f));
        else weigh_usual(s_addr, kf, vf, shift, sum2);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar.p_full[x]);
      }
      if (!ok) break;

      // output: divided by the sum, turned back by R^T
      const float2 parts = unpair(sum2);
      ok = swap(parts.x + parts.y, &other);
      if (!ok) break;
      const float sum = (parts.x + parts.y) + other;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;       // (a NaN in a visible token shows)
      ok = TQ_WARP_WAIT(bar.added[x], (jt - 1) & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      const float top = largest_output(o_addr, inv);
      ok = swap(top, &other);
      if (!ok) break;
      const int eo = exponent_of(fmaxf(top, other));
      output_operand(o_addr, lane_addr + kS + 128 * x + 32 * half, inv, exp2_int(-eo));
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bar.o_raw[x]);
      ok = TQ_WARP_WAIT(bar.turned[x], seg & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      const bool whole = t0 == 0 && t1 == it.tiles;
      // a run's first item may have begun in the run before, its last may go on
      float* const part = a.wide.part + (2ll * blockIdx.x + (t0 == 0 ? 1 : 0)) * part_floats(kWideRows);
      const int part_row = kTile * x + row;
      if (!whole && half == 0) {
        part[kWideRows * kDim + 2 * part_row] = sum == 0.f ? -INFINITY : ref;
        part[kWideRows * kDim + 2 * part_row + 1] = sum;
      }
      if (!whole) {
        store_partial(o_addr, exp2_int(eo), part + part_row * kDim + 64 * half, live);
      } else {
        // bf16 rows through the queries' place in shared memory, to leave in whole lines
        output_rows(o_addr, exp2_int(eo), half_s + row * 128, row);
        __syncwarp();
#pragma unroll 2
        for (int k = 0; k < 8; ++k) {
          const int qr = copy_row + 4 * k, rr = it.i * kWideRows + kTile * x + qr;
          if (rr < n_rows)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + vector_of(rr) * kDim + 64 * half +
                                      copy_chunk * 8) = *swizzled(qr, copy_chunk);
        }
        __syncwarp();                             // (the next queries take their place)
      }
      ptx::tc_fence_before();
      end_segment(a, a.wide, run, t1);
    }
  } else if (warp == kMmaWarp) {
    // ---------------- products ----------------
    // the whole warp walks the tiles and waits; an elected lane issues
    const uint64_t query_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kQuery0));
    const uint64_t key_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kKey0));
    const uint64_t value_desc = ptx::desc_k_sw128(ptx::smem_u32(smem + kValue0));
    int kc = 0, jt = 0;                           // key ring entries, key tiles so far
    auto scores = [&](int x, bool last, bool silent = false) {   // of row tile x against the key ring's next entry
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        const uint64_t q = query_desc + x * (kImage / 16), k = key_desc + (kc & 1) * (kImage / 16);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t off = (ks >> 2) * (kBlockBytes / 16) + (ks & 3) * 2;
          ptx::mma_bf16(tmem + kS + 128 * x, q + off, k + off, kIdescF16, ks > 0);
        }
        if (!silent) ptx::mma_commit(&bar.s_full[x]);
        if (last) ptx::mma_commit(&bar.k_empty[kc & 1]);
        ptx::mbar_arrive(&bar.s_full[x]);
      }
      __syncwarp();
    };
    for (int seg = 0; ok && next_segment(a, a.wide, run, t0, t1); ++seg) {
      ok = TQ_WARP_WAIT(bar.q_full, seg & 1) && TQ_WARP_WAIT(bar.k_full[kc & 1], (kc >> 1) & 1);
      if (!ok) break;
      scores(0, false, withheld(a, a.wide, per, seg));
      scores(1, true);
      ++kc;
      for (int t = t0; ok && t < t1; ++t, ++jt) {
        ok = TQ_WARP_WAIT(bar.v_full[jt & 1], (jt >> 1) & 1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          ok = ok && TQ_WARP_WAIT(bar.p_full[x], jt & 1);
          if (!ok) break;
          if (ptx::elect_one()) {
            ptx::tc_fence_after();
            // (the weights of columns 64 .. 127 start 64 tensor-memory columns on)
            const uint32_t o = tmem + kO + 128 * x, w = tmem + kS + 128 * x;
            const uint64_t v = value_desc + (jt & 1) * (kImage / 16);
            product<4>(o, w, v, kIdescBf16, t > t0);
            product<4>(o, w + 64, v + kBlockBytes / 16, kIdescBf16, true);
            // (the last sixteen of each 64 once more, their remainders)
            product<1>(o, w + 32, v + 6, kIdescBf16, true);
            product<1>(o, w + 96, v + kBlockBytes / 16 + 6, kIdescBf16, true);
            ptx::mma_commit(&bar.added[x]);
            if (x == 1) ptx::mma_commit(&bar.v_empty[jt & 1]);
          }
          __syncwarp();
          if (t + 1 < t1) {
            // the next scores take the columns of the weights just read
            if (x == 0) ok = TQ_WARP_WAIT(bar.k_full[kc & 1], (kc >> 1) & 1);
            ok = ok && TQ_WARP_WAIT(bar.added[x], jt & 1);
            if (!ok) break;
            scores(x, x == 1);
            if (x == 1) ++kc;
          }
        }
      }
      // R^T out
      ok = ok && TQ_WARP_WAIT(bar.k_full[kc & 1], (kc >> 1) & 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        ok = ok && TQ_WARP_WAIT(bar.o_raw[x], seg & 1);
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::tc_fence_after();
          product<8>(tmem + kO + 128 * x, tmem + kS + 128 * x, key_desc + (kc & 1) * (kImage / 16), kIdescF16, false);
          ptx::mma_commit(&bar.turned[x]);
          if (x == 1) ptx::mma_commit(&bar.k_empty[kc & 1]);
        }
        __syncwarp();
      }
      if (!ok) break;
      ++kc;
      end_segment(a, a.wide, run, t1);
    }
    if (ptx::elect_one()) {
      ptx::mma_commit(&bar.drain);                // nothing is in flight when the CTA ends
      ptx::drain_bar(&bar.drain, 0);
    }
  } else {
    // ---------------- copies ----------------
    // the whole warp walks the segments and waits; lane 0 copies
    int kc = 0, jt = 0;
    if (lane == 1) write_cut(a, a.wide, run, per, true);
    while (ok && next_segment(a, a.wide, run, t0, t1)) {
      const long long first = it.seq.w + static_cast<long long>(it.kvh) * max(1, (it.seq.z + kTile - 1) / kTile);
      for (int t = t0; t < t1; ++t, ++jt, ++kc) {
        const uint8_t* const src = a.ws_tiles + (first + t) * kTileImageBytes;
        const int s = kc & 1, vs = jt & 1;
        ok = TQ_WARP_WAIT(bar.k_empty[s], ((kc >> 1) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&bar.k_full[s], kImage + sizeof(TileMeta));
          ptx::bulk_load(smem + kKey0 + s * kImage, src, kImage, &bar.k_full[s]);
          ptx::bulk_load(smem + kMeta0 + (jt & (kRing - 1)) * sizeof(TileMeta), a.ws_meta + first + t, sizeof(TileMeta),
                         &bar.k_full[s]);
        }
        ok = TQ_WARP_WAIT(bar.v_empty[vs], ((jt >> 1) & 1) ^ 1);
        if (!ok) {
          ++kc;
          break;
        }
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&bar.v_full[vs], kImage);
          ptx::bulk_load(smem + kValue0 + vs * kImage, src + kImage, kImage, &bar.v_full[vs]);
        }
        if (t == t0) prefetch_queries(a, a.wide, run, t1, lane, 32);
      }
      if (!ok) break;
      const int s = kc & 1;
      ok = TQ_WARP_WAIT(bar.k_empty[s], ((kc >> 1) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&bar.k_full[s], kImage);
        ptx::bulk_load(smem + kKey0 + s * kImage, a.images + 2 * (kImage / 16), kImage, &bar.k_full[s]);
      }
      ++kc;
      end_segment(a, a.wide, run, t1);
    }
    if (*abort && lane == 0) {                    // copies in flight land before the CTA ends
      for (int c = kc > 1 ? kc - 2 : 0; c < kc; ++c) ptx::drain_bar(&bar.k_full[c & 1], (c >> 1) & 1);
      for (int j = jt > 1 ? jt - 2 : 0; j < jt; ++j) ptx::drain_bar(&bar.v_full[j & 1], (j >> 1) & 1);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int KB, int VB>
cudaError_t expand_bits(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  const cudaError_t err =
      cudaFuncSetAttribute(extend_expand_kernel<KB, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(extend_expand_kernel<KB, VB>, dim3(ctas), kExpandThreads, kExpandSmem, stream, a);
}

template <int KB>
cudaError_t expand_keys(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  switch (a.d.v_bits) {
    case 1: return expand_bits<KB, 1>(a, ctas, stream);
    case 2: return expand_bits<KB, 2>(a, ctas, stream);
    case 3: return expand_bits<KB, 3>(a, ctas, stream);
    default: return expand_bits<KB, 4>(a, ctas, stream);
  }
}

cudaError_t expand(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  switch (a.d.k_bits) {
    case 1: return expand_keys<1>(a, ctas, stream);
    case 2: return expand_keys<2>(a, ctas, stream);
    case 3: return expand_keys<3>(a, ctas, stream);
    default: return expand_keys<4>(a, ctas, stream);
  }
}

}  // namespace

cudaError_t launch_extend_wide(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  cudaError_t err = expand(a, ctas, stream);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(extend_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(extend_wide_kernel, dim3(ctas), kWideThreads, kWideSmem, stream, a);
}

}  // namespace tq
