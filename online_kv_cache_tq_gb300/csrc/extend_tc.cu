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
//           n_t scale multiplies the score in fp32;
//   output  [128 rows x 128 tokens] [128 x 128], bf16: p_t n^v_t against the
//           value levels c^v[code_t], whose bits lie by token already.
// Queries and weights are operands in tensor memory (lane = row), so shared
// memory feeds one operand only.  R q, S q and the back-rotation R^T are
// products on the same tensor cores: their constants pass through the key
// ring as tiles of their own, so no other buffer and no other launch is
// needed.  A query is scaled by a power of two into fp16's range when its
// largest coordinate is outside 2^-8 .. 2^10.
//
// Softmax.  Scores are kept against a reference that is the maximum of the
// row's first visible tile and moves only when a later score may pass it by
// 2^90: fp32 and bf16 hold p exactly as well at 2^80 as at 1.  Whether it may
// is known without looking at the scores, from the length of the query and
// the largest key of the tile, so the usual tile is read once and pays a
// multiply-add, an exponential, a sum, a product and a conversion per score.
// Tiles with hidden positions take a second path that masks.
//
// Twenty-five warps: 0-7 softmax (two threads per row, 64 columns each), 8-15
// keys (two threads per token), 16-23 values (two threads per coordinate), 24
// issues the products.  With half as many, each role's chain of dependent
// instructions was longer than the products it feeds.
// Tensor memory: two score tiles of 128 columns (weights overwrite them),
// the output, the query operand.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "tc_ptx.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;                        // rows of a row tile, tokens of a key tile
constexpr int kSoftThreads = 256;
constexpr int kKeyThreads = 256;
constexpr int kValueThreads = 256;
constexpr int kMmaWarp = 24;
constexpr int kExtThreads = kSoftThreads + kKeyThreads + kValueThreads + 32;
constexpr int kBlockBytes = kTile * 128;          // a 64-column K block of a 128-row operand
constexpr int kKeyBytes = 4 * kBlockBytes;
constexpr int kValueBytes = 2 * kBlockBytes;
constexpr int kRing = 4;                          // key and value factors of the tiles in flight
constexpr int kKey0 = 0;
constexpr int kValue0 = 2 * kKeyBytes;
constexpr int kFactor0 = kValue0 + 2 * kValueBytes;
constexpr int kSmemBytes = kFactor0 + 2 * kRing * kTile * 4 + 1024;   // (1024: alignment)
constexpr uint32_t kS0 = 0, kS1 = 128, kO = 256, kQ = 384;   // tensor-memory columns
constexpr float kRaise = 90.f;                    // log2 by which scores may pass the reference
constexpr int kExtPart = kTile * (kDim + 2);      // floats of a partial: outputs, then (reference, sum)

// kind::f16 with fp16 or bf16 operands, fp32 accumulators, 128 x 128.
constexpr uint32_t kIdescBf16 = ptx::idesc_bf16_f32(128, 128);
constexpr uint32_t kIdescF16 = kIdescBf16 & ~((7u << 7) | (7u << 10));

// ---- work items ------------------------------------------------------------

// Key tiles of row tile i of a sequence: those its last token sees, at least
// one (rows that see nothing still need their zero output).
__device__ __forceinline__ int key_tiles(int i, int n_new, int ctx, int group) {
  const int last = min(n_new - 1, (kTile * (i + 1) - 1) / group);
  const int seen = ctx - n_new + last + 1;
  return seen <= kTile ? 1 : (seen + kTile - 1) / kTile;
}
__device__ __forceinline__ int row_tiles(int n_new, int group) {
  return static_cast<int>((static_cast<long long>(n_new) * group + kTile - 1) / kTile);
}

// One CTA checks the lengths and forms the prefix sums of the key tiles.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(ExtendArgs a) {
  __shared__ long long tiles_s[kPlanThreads];
  __shared__ long long warp_s[kPlanThreads / 32];
  __shared__ long long carry_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) carry_s = 0;
  for (int b0 = 0; b0 < a.d.batch; b0 += kPlanThreads) {
    const int nb = min(kPlanThreads, a.d.batch - b0);
    for (int k = warp; k < nb; k += kPlanThreads / 32) {
      const int b = b0 + k;
      int s0 = a.query_start[b], s1 = a.query_start[b + 1], ctx = a.d.context_lens[b];
      const bool rows_ok = s0 >= 0 && s0 <= s1 && s1 <= a.n_tokens;
      const bool ctx_ok = ctx >= 0 && ctx <= a.d.max_context &&
                          ctx <= static_cast<long long>(a.d.max_blocks) * a.d.block_size;
      if (lane == 0 && (!rows_ok || !ctx_ok)) atomicCAS(a.d.error, 0, kErrContext);
      if (!rows_ok) s0 = s1 = 0;
      if (!ctx_ok) ctx = 0;
      const int mt = row_tiles(s1 - s0, a.d.group);
      long long sum = 0;
      for (int i = lane; i < mt; i += 32) sum += key_tiles(i, s1 - s0, ctx, a.d.group);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) {
        tiles_s[k] = sum * a.d.n_kv;
        a.ws_seq[b] = make_int4(s0, s1 - s0, ctx, 0);
      }
    }
    __syncthreads();
    long long own = tid < nb ? tiles_s[tid] : 0, sum = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 31) warp_s[warp] = sum;
    __syncthreads();
    long long before = carry_s;
    for (int w = 0; w < warp; ++w) before += warp_s[w];
    if (tid < nb) a.ws_first[b0 + tid] = before + sum - own;
    __syncthreads();
    if (tid == kPlanThreads - 1) carry_s = before + sum;
    __syncthreads();
  }
  if (tid == 0) a.ws_first[a.d.batch] = carry_s;
}

// A work item: a row tile of a sequence and KV head, and a key tile in it.
struct Item {
  int b, kvh, i;       // sequence, KV head, row tile
  int tile, tiles;     // current key tile, key tiles of the item
  int4 seq;            // first row, new tokens, context
};

// The item that holds key tile `pos` (found by a whole warp).
__device__ __forceinline__ Item find_item(const ExtendArgs& a, long long pos) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.d.batch;                     // the last sequence that starts at or before pos
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.ws_first[mid] <= pos) lo = mid;
    else hi = mid;
  }
  Item it;
  it.b = lo;
  it.seq = a.ws_seq[lo];
  const long long per_head = (a.ws_first[lo + 1] - a.ws_first[lo]) / a.d.n_kv;
  long long rem = pos - a.ws_first[lo];
  it.kvh = static_cast<int>(rem / per_head);
  rem -= it.kvh * per_head;
  const int mt = row_tiles(it.seq.y, a.d.group);
  it.i = 0;
  it.tile = it.tiles = 0;
  for (int i0 = 0; i0 < mt; i0 += 32) {
    const int nt = i0 + lane < mt ? key_tiles(i0 + lane, it.seq.y, it.seq.z, a.d.group) : 0;
    long long upto = nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const unsigned past = __ballot_sync(0xffffffffu, upto > rem);
    if (past != 0) {
      const int src = __ffs(past) - 1;
      it.i = i0 + src;
      it.tiles = __shfl_sync(0xffffffffu, nt, src);
      it.tile = static_cast<int>(rem - __shfl_sync(0xffffffffu, upto - nt, src));
      break;
    }
    rem -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return it;
}

__device__ __forceinline__ void next_item(const ExtendArgs& a, Item& it) {
  it.tile = 0;
  if (++it.i >= row_tiles(it.seq.y, a.d.group)) {
    it.i = 0;
    if (++it.kvh >= a.d.n_kv) {
      it.kvh = 0;
      do {
        it.seq = a.ws_seq[++it.b];
      } while (it.seq.y == 0);
    }
  }
  it.tiles = key_tiles(it.i, it.seq.y, it.seq.z, a.d.group);
}

// Key tiles of every CTA's run.
__device__ __forceinline__ long long run_length(long long total, int ctas) { return (total + ctas - 1) / ctas; }

// ---- expansion of packed bits ------------------------------------------------

template <int OFFSET>
__device__ __forceinline__ void store16(uint32_t saddr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0 + %5], {%1, %2, %3, %4};"
               ::"r"(saddr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "n"(OFFSET)
               : "memory");
}
__device__ __forceinline__ float4 load16(uint32_t saddr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(saddr));
  return v;
}

// The 16-bit patterns of a codebook's levels as byte tables: low and high
// bytes of levels 0..7 (for 16 levels, of the eight positive ones; the sign is
// set from the top bit of the code).
struct LevelBytes {
  uint32_t lo[2], hi[2];
};
template <bool BF16>
__device__ __forceinline__ LevelBytes level_bytes(const float* levels, int bits) {
  LevelBytes t;
  const int base = bits == 4 ? 8 : 0;
  uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = levels[base + i];
    const uint32_t h = BF16 ? static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v)))
                            : static_cast<uint32_t>(__half_as_ushort(__float2half_rn(v)));
    lo[i >> 2] |= (h & 255u) << (8 * (i & 3));
    hi[i >> 2] |= (h >> 8) << (8 * (i & 3));
  }
  t.lo[0] = lo[0], t.lo[1] = lo[1], t.hi[0] = hi[0], t.hi[1] = hi[1];
  return t;
}

// The bits i, i + 4, .., i + 28 of a plane word, each moved to bit `to` of its nibble.
__device__ __forceinline__ uint32_t every_fourth(uint32_t w, int i, int to) {
  return (i >= to ? w >> (i - to) : w << (to - i)) & (0x11111111u << to);
}

// Chunk i (bits i, i + 4, .., i + 28) of one plane word per code bit, as eight
// 16-bit levels.  A code of up to three bits selects bytes from the tables
// directly; with four the magnitude is the low three bits, inverted when the
// top bit is clear, and a clear top bit sets the sign.
template <int BITS>
__device__ __forceinline__ uint4 expand8(const uint32_t (&w)[BITS], int i, const LevelBytes& t) {
  constexpr int kMag = BITS == 4 ? 3 : BITS;
  uint32_t sel = every_fourth(w[0], i, 0);
  if constexpr (kMag > 1) sel |= every_fourth(w[1], i, 1);
  if constexpr (kMag > 2) sel |= every_fourth(w[2], i, 2);
  uint32_t top = 0;
  if constexpr (BITS == 4) top = every_fourth(w[3], i, 0);
  uint32_t out[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __byte_perm(t.lo[0], t.lo[1], h ? sel >> 16 : sel);
    uint32_t hi = __byte_perm(t.hi[0], t.hi[1], h ? sel >> 16 : sel);
    if constexpr (BITS == 4) hi ^= __byte_perm(0x00000080u, 0u, h ? top >> 16 : top);
    out[2 * h] = __byte_perm(lo, hi, 0x5140);
    out[2 * h + 1] = __byte_perm(lo, hi, 0x7362);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Shared addresses of chunks 0..3 of a row's first K block (swizzled); the
// row's other chunks follow: ^ 64 bytes for chunks 4..7.
struct RowChunks {
  uint32_t at[4];
};
__device__ __forceinline__ RowChunks row_chunks(uint32_t operand, int row) {
  RowChunks r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.at[i] = operand + row * 128 + ((i ^ (row & 7)) << 4);
  return r;
}
__device__ __forceinline__ RowChunks second_word(const RowChunks& r) {   // chunks 4..7
  return RowChunks{{r.at[0] ^ 64, r.at[1] ^ 64, r.at[2] ^ 64, r.at[3] ^ 64}};
}

// One word per plane (32 coordinates or tokens) into four chunks of a row.
template <int BITS, int OFFSET>
__device__ __forceinline__ void expand32(const RowChunks& r, uint32_t (&w)[BITS], const LevelBytes& t) {
  if constexpr (BITS == 4) {
#pragma unroll
    for (int p = 0; p < 3; ++p) w[p] = w[p] ^ ~w[3];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) store16<OFFSET>(r.at[i], expand8<BITS>(w, i, t));
}

// A word of sketch signs: a set bit clears the sign of -rho.
template <int OFFSET>
__device__ __forceinline__ void expand_signs(const RowChunks& r, uint32_t bits, uint32_t minus_rho) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t out[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) out[h] = ((bits << (15 - 4 * i - h)) & 0x80008000u) ^ minus_rho;
    store16<OFFSET>(r.at[i], make_uint4(out[0], out[1], out[2], out[3]));
  }
}

// ---- products ----------------------------------------------------------------

// D (+)= A B^T over STEPS K steps of 16, issued by one lane: A in tensor
// memory (8 columns a step), B in shared memory K blocks of 64 columns (a step
// is 32 bytes, a block 16 KB: 2 and 1024 in the descriptor's units).
template <int STEPS>
__device__ __forceinline__ void product(uint32_t d, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks)
    ptx::mma_bf16_tmem_a(d, a_tmem + 8 * ks, b_desc + (ks >> 2) * (kBlockBytes / 16) + (ks & 3) * 2, idesc,
                         accumulate || ks > 0);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Two fp32 lanes of one 64-bit register.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
// ptx::tmem_ld16 in two steps, so that a load runs while the columns before it are worked on.
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
}

// 2^e for a normal exponent.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) {   // clamped so that 2^-e is a normal number
  const int e = static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127;
  return e < -100 ? -100 : (e > 100 ? 100 : e);
}

__device__ __forceinline__ void load_query8(const ExtendArgs& a, long long at, float (&v)[8]) {
  if (a.q_bf16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.d.q) + at);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.d.q) + at);
    const float4 x = p[0], y = p[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
}

// Walks the cache blocks under 32-token groups of a sequence, 128 tokens at a
// time (a block holds whole groups), with the block table entry read one step
// ahead.
struct Cursor {
  int pos, col, off;         // of the group that `id` belongs to
  int id;
};
__device__ __forceinline__ int table_entry(const DecodeArgs& d, const Item& it, int pos, int col) {
  if (pos >= it.seq.z) return -1;
  return d.block_table ? __ldg(d.block_table + static_cast<long long>(it.b) * d.max_blocks + col)
                       : it.b * d.max_blocks + col;
}
__device__ __forceinline__ void start_cursor(const DecodeArgs& d, const Item& it, int pos, Cursor& c) {
  c.pos = pos;
  c.col = pos / d.block_size;
  c.off = pos - c.col * d.block_size;
  c.id = table_entry(d, it, c.pos, c.col);
}
__device__ __forceinline__ void advance(const DecodeArgs& d, const Item& it, Cursor& c) {
  c.pos += kTile;
  c.off += kTile;
  while (c.off >= d.block_size) {
    c.off -= d.block_size;
    ++c.col;
  }
  c.id = table_entry(d, it, c.pos, c.col);
}
// Row of (block, KV head) in the cache, -1 behind the context and (recorded)
// for an entry outside the cache.
__device__ __forceinline__ long long cache_row(const DecodeArgs& d, const Item& it, const Cursor& c) {
  if (c.pos >= it.seq.z) return -1;
  if (c.id >= 0 && c.id < d.num_blocks) return static_cast<long long>(c.id) * d.n_kv + it.kvh;
  atomicCAS(d.error, 0, kErrBlock);
  return -1;
}

struct Barriers {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2];
  uint64_t q_raw, rotated, q_full, o_raw, turned, drain;
  uint64_t rows[4];          // the two warps that share 32 rows
};

// Half of a packed key (64 coordinates) on its way into the ring.
template <int KB>
struct RawKey {
  uint2 planes[KB], qjl;
  float norm, rnorm;
  bool valid;
};

// Token `token` (0..31) of the group under the cursor.
template <int KB>
__device__ __forceinline__ void load_key(const DecodeArgs& d, const Item& it, const Cursor& c, int token, int half,
                                         RawKey<KB>& k) {
  k.valid = false;
  k.norm = k.rnorm = 0.f;
  const long long blk = cache_row(d, it, c);
  if (blk < 0 || c.pos + token >= it.seq.z) return;
  const long long row = blk * d.block_size + c.off + token;
  const uint2* const codes = reinterpret_cast<const uint2*>(d.k_codes + row * (KB * 16)) + half;
#pragma unroll
  for (int p = 0; p < KB; ++p) k.planes[p] = __ldg(codes + 2 * p);
  k.norm = load_norm(d.k_norm, row, d.norm16);
  if (d.k_qjl != nullptr) {
    k.qjl = __ldg(reinterpret_cast<const uint2*>(d.k_qjl + row * 16) + half);
    k.rnorm = load_norm(d.k_rnorm, row, d.norm16);
  }
  k.valid = true;
}

// Value bits of one coordinate over two of the tile's 32-token groups, and the
// norm of the token whose factor this thread writes.
template <int VB>
struct RawValue {
  uint32_t words[VB][2];     // [plane][group]
  float norm;
};

// Lane l of the warp has the cursor of the first or second of the thread's two
// groups (l & 1); `mine` is the one whose norms this warp reads (-1: neither).
// Blocks of a multiple of 64 tokens give both words of a plane in one load.
template <int VB>
__device__ __forceinline__ void load_value(const DecodeArgs& d, const Item& it, const Cursor& c, int dim, int mine,
                                           int token, RawValue<VB>& v) {
  const long long row = cache_row(d, it, c);
  const int words = d.block_size / 32;            // of one plane and coordinate
  const long long base = row < 0 ? -1 : row * (VB * 128ll * words) + c.off / 32;
  const uint32_t* const codes = reinterpret_cast<const uint32_t*>(d.v_codes) + dim * words;
  const int plane = 128 * words;
  const long long at0 = __shfl_sync(0xffffffffu, base, 0), at1 = __shfl_sync(0xffffffffu, base, 1);
  if (words % 2 == 0) {
#pragma unroll
    for (int p = 0; p < VB; ++p) {
      const uint2 w = at0 < 0 ? make_uint2(0, 0) : __ldg(reinterpret_cast<const uint2*>(codes + at0 + p * plane));
      v.words[p][0] = w.x, v.words[p][1] = w.y;
    }
  } else {
#pragma unroll
    for (int p = 0; p < VB; ++p) {
      v.words[p][0] = at0 < 0 ? 0u : __ldg(codes + at0 + p * plane);
      v.words[p][1] = at1 < 0 ? 0u : __ldg(codes + at1 + p * plane);
    }
  }
  v.norm = 0.f;
  if (mine >= 0) {
    const long long norm_row = __shfl_sync(0xffffffffu, row, mine);
    const int norm_off = __shfl_sync(0xffffffffu, c.off, mine), norm_pos = __shfl_sync(0xffffffffu, c.pos, mine);
    if (norm_row >= 0 && norm_pos + token < it.seq.z)
      v.norm = load_norm(d.v_norm, norm_row * d.block_size + norm_off + token, d.norm16);
  }
}

template <int KB, int VB>
__global__ void __launch_bounds__(kExtThreads, 1) extend_kernel(ExtendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bar;
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  __shared__ Item item_s;
  __shared__ float swap_s[2][2][kTile];           // what the two threads of a row tell each other
  __shared__ float2 reach_s[kRing][4];            // per 32 tokens of a tile: bounds of the longest scaled key halves
  __shared__ uint32_t valid_s[kRing][4];          // tokens of a tile, by expanded column

  // 1024-byte aligned, as an offset from smem_raw so that accesses stay shared-space
  uint8_t* const smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const DecodeArgs& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* const abort = &abort_s;
  const long long total = a.ws_first[d.batch];
  const long long per = run_length(total, gridDim.x);
  const long long begin = blockIdx.x * per, end = begin + per < total ? begin + per : total;
  if (begin >= end) return;                       // (the whole CTA)

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
    const Item it = find_item(a, begin);
    if (lane == 0) item_s = it;
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_s;
  Item it = item_s;
  const bool qjl = d.k_qjl != nullptr;
  float* const key_factor = reinterpret_cast<float*>(smem + kFactor0);
  float* const value_factor = key_factor + kRing * kTile;
  long long pos = begin;
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
    for (int seg = 0; pos < end; ++seg) {
      const int t0 = it.tile, t1 = static_cast<int>(min(static_cast<long long>(it.tiles), t0 + (end - pos)));
      const int n_rows = it.seq.y * d.group;
      const int r = it.i * kTile + row;
      const bool live = r < n_rows;
      const int tok = (live ? r : n_rows - 1) / d.group;
      const long long vec = (static_cast<long long>(it.seq.x) + tok) * d.n_q + it.kvh * d.group + r - tok * d.group;
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
      if (biggest == 0.f || (e >= -8 && e < 10)) e = 0;
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
        ptx::tc_fence_after();
        // this thread's 64 scores; their weights go to the first 32 of the columns
        const uint32_t s_addr = lane_addr + (sb ? kS1 : kS0) + 64 * half;
        const uint32_t kf = ptx::smem_u32(key_factor + rg * kTile + 64 * half);
        const uint32_t vf = ptx::smem_u32(value_factor + rg * kTile + 64 * half);
        const uint32_t all = valid_s[rg][0] & valid_s[rg][1] & valid_s[rg][2] & valid_s[rg][3];
        float top_bound = 0.f;                    // |score| <= |R q| |n c| + |S q| |n rho signs|
#pragma unroll
        for (int g = 0; g < 4; ++g)
          top_bound = fmaxf(top_bound, fmaf(len_r, reach_s[rg][g].x, len_s * reach_s[rg][g].y));
        // (the same for both threads of a row)
        const bool usual = t > t0 && e == 0 && seen >= (t + 1) * kTile && all == 0xffffffffu && top_bound <= ref + kRaise;
        if (__all_sync(0xffffffffu, usual)) {
          const uint64_t minus = pair(-ref, -ref);
          uint32_t x[2][16];
          tmem_ld16_start(s_addr, x[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld16_wait(x[c & 1]);
            if (c < 3) tmem_ld16_start(s_addr + 16 * (c + 1), x[(c + 1) & 1]);
            const uint32_t(&y)[16] = x[c & 1];
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 f = load16(kf + 64 * c + 16 * k);
              const float4 g = load16(vf + 64 * c + 16 * k);
              const float2 z0 = unpair(fma2(pair(__uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1])),
                                            pair(f.x, f.y), minus));
              const float2 z1 = unpair(fma2(pair(__uint_as_float(y[4 * k + 2]), __uint_as_float(y[4 * k + 3])),
                                            pair(f.z, f.w), minus));
              const uint64_t p0 = pair(exp2_fast(z0.x), exp2_fast(z0.y)), p1 = pair(exp2_fast(z1.x), exp2_fast(z1.y));
              sum2 = add2(sum2, add2(p0, p1));
              const float2 w0 = unpair(mul2(p0, pair(g.x, g.y))), w1 = unpair(mul2(p1, pair(g.z, g.w)));
              w[2 * k] = pack_bf16(w0.x, w0.y);
              w[2 * k + 1] = pack_bf16(w1.x, w1.y);
            }
            ptx::tmem_st8(s_addr + 8 * c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
          }
        } else {
          // hidden positions, a scaled query, or scores that may pass the
          // reference: the tile's maximum first
          const int here = min(kTile, max(0, seen - t * kTile));
          auto mask_of = [&](int g) {             // visible tokens of group g
            const int n = min(32, max(0, here - 32 * g));
            return (n == 32 ? 0xffffffffu : (1u << n) - 1u) & valid_s[rg][g];
          };
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            const uint32_t mask = mask_of(2 * half + c);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t y[16];
              ptx::tmem_ld16(s_addr + 32 * c + 16 * h, y);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float4 f = load16(kf + 128 * c + 64 * h + 16 * k);
                const float fk[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float s = __uint_as_float(y[4 * k + q]) * fk[q] * factor;
                  top = mask & (1u << expanded_bit(16 * h + 4 * k + q)) ? fmaxf(top, s) : top;
                }
              }
            }
          }
          ok = swap(top, &other);
          if (!ok) break;
          top = fmaxf(top, other);
          const bool raise = top > ref + kRaise || (ref == -INFINITY && top > ref);
          if (__any_sync(0xffffffffu, raise)) {
            const float scale = raise ? exp2_fast(ref - top) : 1.f;
            if (raise) ref = top;
            if (t > t0) {
              // the output so far, once the product before has added to it
              ok = __all_sync(0xffffffffu, TQ_WAIT(bar.v_empty[(jt - 1) & 1], ((jt - 1) >> 1) & 1));
              if (!ok) break;
              ptx::tc_fence_after();
              sum2 = mul2(sum2, pair(scale, scale));
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                const uint32_t at = lane_addr + kO + 64 * half + 8 * c;
                uint32_t y[8];
                tmem_ld8(at, y);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * scale);
                ptx::tmem_st8(at, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
              }
            }
          }
          const float shift = ref == -INFINITY ? 0.f : ref;
          float sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            const uint32_t mask = mask_of(2 * half + c);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t y[16], w[8];
              ptx::tmem_ld16(s_addr + 32 * c + 16 * h, y);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float4 f = load16(kf + 128 * c + 64 * h + 16 * k);
                const float4 g = load16(vf + 128 * c + 64 * h + 16 * k);
                const float fk[4] = {f.x, f.y, f.z, f.w}, gk[4] = {g.x, g.y, g.z, g.w};
                float p[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const bool on = mask & (1u << expanded_bit(16 * h + 4 * k + q));
                  p[q] = on ? exp2_fast(__uint_as_float(y[4 * k + q]) * fk[q] * factor - shift) : 0.f;
                  sum += p[q];
                  p[q] = on ? p[q] * gk[q] : 0.f;
                }
                w[2 * k] = pack_bf16(p[0], p[1]);
                w[2 * k + 1] = pack_bf16(p[2], p[3]);
              }
              ptx::tmem_st8(s_addr + 16 * c + 8 * h, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
            }
          }
          sum2 = add2(sum2, pair(sum, 0.f));
        }
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
      float top = 0.f;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t y[16];
        ptx::tmem_ld16(lane_addr + kO + 64 * half + 16 * c, y);
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(__uint_as_float(y[k]) * inv));
      }
      ok = swap(top, &other);
      if (!ok) break;
      const int eo = exponent_of(fmaxf(top, other));
      const float out_down = inv * exp2_int(-eo), out_up = exp2_int(eo);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t y[16], w[8];
        ptx::tmem_ld16(lane_addr + kO + 64 * half + 16 * c, y);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          w[k] = pack_f16(__uint_as_float(y[2 * k]) * out_down, __uint_as_float(y[2 * k + 1]) * out_down);
        ptx::tmem_st8(lane_addr + kS0 + 32 * half + 8 * c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bar.o_raw);
      ok = __all_sync(0xffffffffu, TQ_WAIT(bar.turned, seg & 1));
      if (!ok) break;
      ptx::tc_fence_after();
      const bool whole = t0 == 0 && t1 == it.tiles;
      // a run's first item may have begun in the run before, its last may go on
      float* const part = a.ws_part + (2ll * blockIdx.x + (t0 == 0 ? 1 : 0)) * kExtPart;
      if (!whole && half == 0) {
        part[kTile * kDim + 2 * row] = sum == 0.f ? -INFINITY : ref;
        part[kTile * kDim + 2 * row + 1] = sum;
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t y[16];
        ptx::tmem_ld16(lane_addr + kS1 + 64 * half + 16 * c, y);
        if (live && whole) {
          uint4* const dst =
              reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + vec * kDim + 64 * half + 16 * c);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = pack_bf16(__uint_as_float(y[8 * k + 2 * q]) * out_up, __uint_as_float(y[8 * k + 2 * q + 1]) * out_up);
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (live) {
          float4* const dst = reinterpret_cast<float4*>(part + row * kDim + 64 * half + 16 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_float4(__uint_as_float(y[4 * k]) * out_up, __uint_as_float(y[4 * k + 1]) * out_up,
                                 __uint_as_float(y[4 * k + 2]) * out_up, __uint_as_float(y[4 * k + 3]) * out_up);
        }
      }
      pos += t1 - t0;
      if (pos < end) next_item(a, it);
    }
  } else if (warp < 16) {
    // ---------------- keys ----------------
    const int row = (tid - kSoftThreads) & (kTile - 1);   // row of the tile: token expanded_bit(lane) of the warp's group
    const int half = (tid - kSoftThreads) / kTile;        // coordinates 64 half .. + 63 of both operand halves
    const LevelBytes lev = level_bytes<false>(d.tables->k_levels, KB);
    float biggest = 0.f;                          // the outermost level
    for (int i = 0; i < (1 << KB); ++i) biggest = fmaxf(biggest, fabsf(d.tables->k_levels[i]));
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
    while (ok && pos < end) {
      const int t0 = it.tile, t1 = static_cast<int>(min(static_cast<long long>(it.tiles), t0 + (end - pos)));
      Cursor c;
      RawKey<KB> next;
      start_cursor(d, it, t0 * kTile + (row & ~31), c);
      load_key(d, it, c, expanded_bit(lane), half, next);
      advance(d, it, c);
      ok = image(0, qjl ? 2 : 1);
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
        const uint32_t minus_rho = __half_as_ushort(__float2half_rn(rho)) * 0x00010001u ^ 0x80008000u;
        {
          uint32_t lo[KB], hi[KB];
#pragma unroll
          for (int p = 0; p < KB; ++p) lo[p] = k.planes[p].x, hi[p] = k.planes[p].y;
          expand32<KB, 0>(at, lo, lev);
          expand32<KB, 0>(second_word(at), hi, lev);
        }
        if (qjl) {
          expand_signs<2 * kBlockBytes>(at, k.qjl.x, minus_rho);
          expand_signs<2 * kBlockBytes>(second_word(at), k.qjl.y, minus_rho);
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
            reach_s[rg][row >> 5] = make_float2(__uint_as_float(bits_c), __uint_as_float(bits_q));
          }
        }
        ptx::fence_async_shared();
        ptx::mbar_arrive(&bar.k_full[s]);
      }
      ok = ok && image(2, 1);
      pos += t1 - t0;
      if (pos < end) next_item(a, it);
    }
  } else if (warp < kMmaWarp) {
    // ---------------- values ----------------
    const int dim = (tid - kSoftThreads - kKeyThreads) & (kTile - 1);
    const int half = (tid - kSoftThreads - kKeyThreads) / kTile;   // 32-token groups 2 half and 2 half + 1
    // the first two warps of a half write its 64 factors, by expanded column
    const int mine = dim < 64 ? dim >> 5 : -1;
    const LevelBytes lev = level_bytes<true>(d.tables->v_levels, VB);
    int jt = 0;
    while (ok && pos < end) {
      const int t0 = it.tile, t1 = static_cast<int>(min(static_cast<long long>(it.tiles), t0 + (end - pos)));
      Cursor c;
      RawValue<VB> next;
      start_cursor(d, it, t0 * kTile + 64 * half + 32 * (lane & 1), c);
      load_value(d, it, c, dim, mine, expanded_bit(lane), next);
      advance(d, it, c);
      for (int t = t0; t < t1; ++t, ++jt) {
        const RawValue<VB> v = next;
        if (t + 1 < t1) {
          load_value(d, it, c, dim, mine, expanded_bit(lane), next);
          advance(d, it, c);
        }
        const int s = jt & 1, rg = jt & (kRing - 1);
        ok = __all_sync(0xffffffffu, TQ_WAIT(bar.v_empty[s], ((jt >> 1) & 1) ^ 1));
        if (!ok) break;
        const RowChunks at = row_chunks(ptx::smem_u32(smem + kValue0 + s * kValueBytes) + half * kBlockBytes, dim);
        uint32_t lo[VB], hi[VB];
#pragma unroll
        for (int p = 0; p < VB; ++p) lo[p] = v.words[p][0], hi[p] = v.words[p][1];
        expand32<VB, 0>(at, lo, lev);
        expand32<VB, 0>(second_word(at), hi, lev);
        if (mine >= 0) value_factor[rg * kTile + 64 * half + dim] = v.norm;
        ptx::fence_async_shared();
        ptx::mbar_arrive(&bar.v_full[s]);
      }
      pos += t1 - t0;
      if (pos < end) next_item(a, it);
    }
  } else {
    // ---------------- products ----------------
    // the whole warp walks the tiles and waits; an elected lane issues
#define TQ_WARP_WAIT(b, ph) __all_sync(0xffffffffu, TQ_WAIT(b, ph))
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
    for (int seg = 0; ok && pos < end; ++seg) {
      const int t0 = it.tile, t1 = static_cast<int>(min(static_cast<long long>(it.tiles), t0 + (end - pos)));
      // R q and S q
      ok = TQ_WARP_WAIT(bar.k_full[kc & 1], (kc >> 1) & 1) && TQ_WARP_WAIT(bar.q_raw, seg & 1);
      if (!ok) break;
      if (ptx::elect_one()) {
        ptx::tc_fence_after();
        product<8>(tmem + kS0, tmem + kS1, key_stage(kc), kIdescF16, false);
        if (qjl) product<8>(tmem + kO, tmem + kS1, key_stage(kc) + 2 * (kBlockBytes / 16), kIdescF16, false);
        ptx::mma_commit(&bar.rotated);
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
      pos += t1 - t0;
      if (pos < end) next_item(a, it);
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

// Joins the partial outputs of a split row tile: sum_s l_s 2^{m_s - M} o_s / sum_s l_s 2^{m_s - M}.
// blockIdx.x + 1 is a run's number; the block works if that run's beginning is
// the first cut inside its item.  A warp per row, four coordinates a lane.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) extend_join_kernel(ExtendArgs a, int ctas) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long total = a.ws_first[a.d.batch];
  const long long per = run_length(total, ctas);
  const long long cut = (blockIdx.x + 1) * per;
  if (cut >= total) return;
  const Item it = find_item(a, cut);
  const long long start = cut - it.tile;          // the item's first key tile
  if (it.tile == 0 || start < cut - per) return;  // no cut here, or an earlier one inside the item
  const int c0 = static_cast<int>(start / per);   // runs c0 .. c1 hold it
  const int c1 = static_cast<int>((start + it.tiles - 1) / per);
  const int n_rows = it.seq.y * a.d.group;
  const int row = blockIdx.y * kJoinWarps + warp, r = it.i * kTile + row;
  if (r >= n_rows) return;
  // (the run that holds key tile 0 wrote its second slot, the others their first)
  auto part = [&](int c) { return a.ws_part + (2ll * c + (c == c0 ? 1 : 0)) * kExtPart; };
  float top = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, part(c)[kTile * kDim + 2 * row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float weight = 0.f;
  for (int c = c0; c <= c1; ++c) {
    const float* const p = part(c);
    const float l = p[kTile * kDim + 2 * row + 1];
    if (l == 0.f) continue;
    const float w = l * exp2_fast(p[kTile * kDim + 2 * row] - top);
    const float4 o = reinterpret_cast<const float4*>(p + row * kDim)[lane];
    acc.x = fmaf(w, o.x, acc.x);
    acc.y = fmaf(w, o.y, acc.y);
    acc.z = fmaf(w, o.z, acc.z);
    acc.w = fmaf(w, o.w, acc.w);
    weight += w;
  }
  const float inv = weight == 0.f ? 0.f : 1.f / weight;
  const int tok = r / a.d.group;
  const long long vec = (static_cast<long long>(it.seq.x) + tok) * a.d.n_q + it.kvh * a.d.group + r - tok * a.d.group;
  reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + vec * kDim)[lane] =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

template <int KB, int VB>
cudaError_t launch_bits(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  const cudaError_t err =
      cudaFuncSetAttribute(extend_kernel<KB, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (err != cudaSuccess) return err;
  extend_kernel<KB, VB><<<ctas, kExtThreads, kSmemBytes, stream>>>(a);
  return cudaGetLastError();
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

// One build per pair of bit widths: a role's loop then fits the instruction
// cache (with the widths chosen inside the loops every role ran at a quarter
// of its speed, waiting for instructions).
cudaError_t launch_main(const ExtendArgs& a, int ctas, cudaStream_t stream) {
  switch (a.d.k_bits) {
    case 1: return launch_keys<1>(a, ctas, stream);
    case 2: return launch_keys<2>(a, ctas, stream);
    case 3: return launch_keys<3>(a, ctas, stream);
    default: return launch_keys<4>(a, ctas, stream);
  }
}

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t extend_workspace_bytes(int batch, int num_sms) {
  return align256((static_cast<size_t>(batch) + 1) * sizeof(long long)) +
         align256(static_cast<size_t>(batch) * sizeof(int4)) + 2 * static_cast<size_t>(num_sms) * kExtPart * sizeof(float);
}

cudaError_t launch_extend(const ExtendArgs& args, void* workspace, cudaStream_t stream) {
  ExtendArgs a = args;
  char* const ws = static_cast<char*>(workspace);
  a.ws_first = reinterpret_cast<long long*>(ws);
  a.ws_seq = reinterpret_cast<int4*>(ws + align256((static_cast<size_t>(a.d.batch) + 1) * sizeof(long long)));
  a.ws_part = reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws_seq) +
                                       align256(static_cast<size_t>(a.d.batch) * sizeof(int4)));
  const int ctas = a.d.num_sms;
  extend_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  const cudaError_t err = launch_main(a, ctas, stream);
  if (err != cudaSuccess) return err;
  if (ctas > 1) extend_join_kernel<<<dim3(ctas - 1, kTile / kJoinWarps), 32 * kJoinWarps, 0, stream>>>(a, ctas);
  return cudaGetLastError();
}

}  // namespace tq
