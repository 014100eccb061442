// Attention of several new tokens per sequence over the packed cache: the
// plan, the workspace, the two forms' launches and the join of split rows.
//
// A sequence takes one of two forms.  The narrow form (extend_tc.cu) expands
// packed key tiles on the way into its products and needs no other memory;
// its score product has 256 columns with the sketch, and every row tile of 128
// expands its key tiles again.  The wide form (extend_wide.cu) expands and
// turns back a sequence's keys and values once, into the workspace, for row
// tiles of 256 and score products of 128 columns.
#include "extend_common.cuh"

namespace tq {
namespace {

// Rows (new tokens x query heads of the group) from which a sequence takes the
// wide form, and most expanded tiles that a workspace holds (2 GiB).
// Sixteen sequences on 8192 (0) cached tokens, 32/8 heads, us, wide | narrow:
//                2-bit keys, sketch, 3-bit values     4-bit keys, 4-bit values
//    256 rows    338 | 249   (39 | 38)                318 | 321   (41 | 38)
//    384         447 | 358   (49 | 51)                427 | 462   (48 | 51)
//    512         449 | 468   (49 | 63)                429 | 607   (50 | 62)
//   1024         667 | 895   (78 | 113)               646 | 1185  (77 | 116)
// (Four-bit codes would cross lower, at 256 rows; one limit serves all widths.)
constexpr int kWideFrom = 512;
constexpr long long kTileCap = 1 << 15;

// One CTA checks the lengths, chooses the forms and forms the prefix sums of
// units of work and expanded tiles: a thread per sequence for what is read and
// written, a warp per sequence for the sums over its row tiles.
constexpr int kPlanThreads = 1024;

struct Sums {
  long long narrow, wide, expand;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.narrow + b.narrow, a.wide + b.wide, a.expand + b.expand};
}
__device__ __forceinline__ Sums shfl_up(const Sums& v, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, v.narrow, d), __shfl_up_sync(0xffffffffu, v.wide, d),
              __shfl_up_sync(0xffffffffu, v.expand, d)};
}

// Inclusive sums over the CTA's threads; *total: over all of them.
__device__ __forceinline__ Sums plan_scan(Sums v, Sums* warp_s, Sums* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x / 32;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(v, d);
    if (lane >= d) v = v + o;
  }
  if (lane == 31) warp_s[warp] = v;
  __syncthreads();
  Sums w = lane < warps ? warp_s[lane] : Sums{0, 0, 0};
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(w, d);
    if (lane >= d) w = w + o;
  }
  *total = Sums{__shfl_sync(0xffffffffu, w.narrow, 31), __shfl_sync(0xffffffffu, w.wide, 31),
                __shfl_sync(0xffffffffu, w.expand, 31)};
  const Sums before{__shfl_sync(0xffffffffu, w.narrow, warp - 1), __shfl_sync(0xffffffffu, w.wide, warp - 1),
                    __shfl_sync(0xffffffffu, w.expand, warp - 1)};
  __syncthreads();
  return warp > 0 ? v + before : v;
}

__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(ExtendArgs a) {
  __shared__ long long narrow_s[kPlanThreads], wide_s[kPlanThreads];
  __shared__ int2 seq_s[kPlanThreads];
  __shared__ Sums warp_s[32];
  launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  const int group = a.d.group;
  Sums base{0, 0, 0};
  long long asked = 0;                            // expanded tiles of the sequences that could be wide
  for (int b0 = 0; b0 < a.d.batch; b0 += threads) {
    const int nb = min(threads, a.d.batch - b0), b = b0 + tid;
    const bool here = tid < nb;
    int4 seq = make_int4(0, 0, 0, 0);
    if (here) {
      const int s0 = a.query_start[b], s1 = a.query_start[b + 1], ctx = a.d.context_lens[b];
      const bool rows_ok = s0 >= 0 && s0 <= s1 && s1 <= a.n_tokens;
      const bool ctx_ok = ctx >= 0 && ctx <= a.d.max_context &&
                          ctx <= static_cast<long long>(a.d.max_blocks) * a.d.block_size;
      if (!rows_ok || !ctx_ok) atomicCAS(a.d.error, 0, kErrContext);
      seq = make_int4(rows_ok ? s0 : 0, rows_ok ? s1 - s0 : 0, ctx_ok ? ctx : 0, 0);
      seq_s[tid] = make_int2(seq.y, seq.z);
    }
    const bool eligible = a.tile_cap > 0 && static_cast<long long>(seq.y) * group >= kWideFrom;
    __syncthreads();
    for (int k = warp; k < nb; k += threads / 32) {
      const int n = seq_s[k].x, ctx = seq_s[k].y;
      long long narrow = 0, wide = 0;
      for (int i = lane; i < row_tiles(kNarrowRows, n, group); i += 32)
        narrow += kNarrowCost + key_tiles(a, i, kNarrowRows, n, ctx);
      if (a.tile_cap > 0)
        for (int i = lane; i < row_tiles(kWideRows, n, group); i += 32)
          wide += kWideCost + key_tiles(a, i, kWideRows, n, ctx);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        narrow += __shfl_xor_sync(0xffffffffu, narrow, d);
        wide += __shfl_xor_sync(0xffffffffu, wide, d);
      }
      if (lane == 0) {
        narrow_s[k] = narrow * a.d.n_kv;
        wide_s[k] = wide * a.d.n_kv;
      }
    }
    __syncthreads();
    bool wide = false;
    long long want = 0;
    if (a.tile_cap > 0) {
      // a sequence that could be wide is, if its tiles fit behind those of the
      // ones before (at least one tile: rows that see nothing are given one)
      want = eligible ? static_cast<long long>(max(1, (seq.z + kTile - 1) / kTile)) * a.d.n_kv : 0;
      Sums total;
      const Sums upto = plan_scan(Sums{want, 0, 0}, warp_s, &total);
      wide = want > 0 && asked + upto.narrow <= a.tile_cap;
      asked += total.narrow;
    }
    const Sums own{here && !wide ? narrow_s[tid] : 0, wide ? wide_s[tid] : 0, wide ? want : 0};
    Sums total;
    const Sums upto = base + plan_scan(own, warp_s, &total);
    if (here) {
      a.narrow.first[b] = upto.narrow - own.narrow;
      a.wide.first[b] = upto.wide - own.wide;
      a.ws_expand[b] = upto.expand - own.expand;
      seq.w = wide ? static_cast<int>(upto.expand - own.expand) : -1;
      a.ws_seq[b] = seq;
    }
    base = base + total;
  }
  if (tid == 0) {
    a.narrow.first[a.d.batch] = base.narrow;
    a.wide.first[a.d.batch] = base.wide;
    a.ws_expand[a.d.batch] = base.expand;
  }
}

// Joins the partial outputs of a split row tile: sum_s l_s 2^{m_s - M} o_s / sum_s l_s 2^{m_s - M}.
// Block x joins the item that run x begins and does not end.  A warp per row,
// four coordinates a lane.
constexpr int kJoinWarps = 8;
constexpr int kJoinSplit = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) extend_join_kernel(ExtendArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ExtendForm f = blockIdx.z == 0 ? a.narrow : a.wide;
  wait_prerequisites();
  const CutItem cut = f.cuts[blockIdx.x];
  const int c0 = blockIdx.x;
  // (the run that holds key tile 0 wrote its second slot, the others their first)
  auto part = [&](int c) { return f.part + (2ll * c + (c == c0 ? 1 : 0)) * part_floats(f.rows); };
  for (int row = blockIdx.y * kJoinWarps + warp; row < cut.rows; row += kJoinSplit * kJoinWarps) {
    const int stats = f.rows * kDim + 2 * row;
    float top = -INFINITY;
    for (int c = c0 + lane; c <= cut.last; c += 32) top = fmaxf(top, part(c)[stats]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float weight = 0.f;
#pragma unroll 4
    for (int c = c0; c <= cut.last; ++c) {
      const float* const p = part(c);
      const float2 ml = *reinterpret_cast<const float2*>(p + stats);
      const float4 o = reinterpret_cast<const float4*>(p + row * kDim)[lane];
      const float w = ml.y == 0.f ? 0.f : ml.y * exp2_fast(ml.x - top);
      if (w == 0.f) continue;                     // (a run that saw nothing left no output)
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
      weight += w;
    }
    const float inv = weight == 0.f ? 0.f : 1.f / weight;
    const long long vec = row_vector(a, cut.row0, cut.kvh, cut.i * f.rows + row);
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + vec * kDim)[lane] =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t first, wide_first, expand, seq, cuts, part, wide_part, meta, tiles, total;
  int tile_cap;
};

// The wide form's regions are there only if some sequence can have the rows
// for it; then as many expanded tiles as that many sequences can need.
Layout layout(int n_tokens, int batch, int group, int n_kv, int max_context, int num_sms) {
  Layout l;
  const long long wide = static_cast<long long>(n_tokens) * group / kWideFrom;
  const long long sequences = wide < batch ? wide : batch;
  const long long context_tiles = max_context > kTile ? (static_cast<long long>(max_context) + kTile - 1) / kTile : 1;
  long long cap = context_tiles > kTileCap / n_kv ? (sequences > 0 ? kTileCap : 0) : sequences * context_tiles * n_kv;
  if (cap > kTileCap) cap = kTileCap;
  l.tile_cap = static_cast<int>(cap);
  const size_t sums = align256((static_cast<size_t>(batch) + 1) * sizeof(long long));
  l.first = 0;
  l.wide_first = sums;
  l.expand = 2 * sums;
  l.seq = 3 * sums;
  l.cuts = l.seq + align256(static_cast<size_t>(batch) * sizeof(int4));
  l.part = l.cuts + align256(2 * static_cast<size_t>(num_sms) * sizeof(CutItem));
  l.wide_part = l.part + align256(2 * static_cast<size_t>(num_sms) * part_floats(kNarrowRows) * sizeof(float));
  l.meta = l.wide_part +
           (cap > 0 ? align256(2 * static_cast<size_t>(num_sms) * part_floats(kWideRows) * sizeof(float)) : 0);
  l.tiles = l.meta + align256(static_cast<size_t>(cap) * sizeof(TileMeta));
  l.total = l.tiles + static_cast<size_t>(cap) * kTileImageBytes;
  return l;
}

}  // namespace

size_t extend_workspace_bytes(int n_tokens, int batch, int n_q, int n_kv, int max_context, int num_sms) {
  return layout(n_tokens, batch, n_q / n_kv, n_kv, max_context, num_sms).total;
}

cudaError_t launch_extend(const ExtendArgs& args, void* workspace, cudaStream_t stream) {
  ExtendArgs a = args;
  char* const ws = static_cast<char*>(workspace);
  const int ctas = a.d.num_sms;
  const Layout l = layout(a.n_tokens, a.d.batch, a.d.group, a.d.n_kv, a.d.max_context, ctas);
  a.narrow = ExtendForm{kNarrowRows, kNarrowCost, reinterpret_cast<long long*>(ws + l.first),
                        reinterpret_cast<float*>(ws + l.part), reinterpret_cast<CutItem*>(ws + l.cuts)};
  a.wide = ExtendForm{kWideRows, kWideCost, reinterpret_cast<long long*>(ws + l.wide_first),
                      reinterpret_cast<float*>(ws + l.wide_part), reinterpret_cast<CutItem*>(ws + l.cuts) + ctas};
  a.ws_expand = reinterpret_cast<long long*>(ws + l.expand);
  a.ws_seq = reinterpret_cast<int4*>(ws + l.seq);
  a.ws_meta = reinterpret_cast<TileMeta*>(ws + l.meta);
  a.ws_tiles = reinterpret_cast<uint8_t*>(ws + l.tiles);
  a.tile_cap = l.tile_cap;
  a.group_shift = 0;
  while ((1 << a.group_shift) < a.d.group) ++a.group_shift;
  a.group_mul = static_cast<uint32_t>(((1ull << (31 + a.group_shift)) + a.d.group - 1) / a.d.group);
  const int plan_threads = a.d.batch >= kPlanThreads ? kPlanThreads : (a.d.batch + 255) / 256 * 256;
  extend_plan_kernel<<<1, plan_threads, 0, stream>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess && a.tile_cap > 0) err = launch_extend_wide(a, ctas, stream);
  if (err == cudaSuccess) err = launch_extend_narrow(a, ctas, stream);
  if (err != cudaSuccess || ctas < 2) return err;
  return launch_dependent(extend_join_kernel, dim3(ctas, kJoinSplit, a.tile_cap > 0 ? 2 : 1), 32 * kJoinWarps, 0, stream, a);
}

}  // namespace tq
