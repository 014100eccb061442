// Device code shared by the two forms of the multi-token attention
// (extend_tc.cu, extend_wide.cu): work items, the expansion of packed bits,
// the softmax of a score tile in tensor memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dependent.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;                        // rows of a product, tokens of a key tile
constexpr int kBlockBytes = kTile * 128;          // a 64-column K block of a 128-row operand
// log2 by which scores may pass the reference (zero at first), or lie below it
// while it is zero: 2^80 leaves fp32 sums and bf16 weights room for 2^20 tokens
// with values of 2^27, and weights of values of 2^-40 are normal numbers.
// (16 sequences x 4 tokens at context 8192, whose keys' channels spread by a
// factor of two, have bounds up to 2^75: 123 us; with 2^72 some tiles are
// searched, 133 us; with a limit per tile from its largest value, 127 us.)
constexpr float kRaise = 80.f;
// log2 by which a row's largest score may lie below a reference of zero for the
// 8-bit cache, whose weights take their value's scale (2^-40 to 2^14) in the
// exponent before they are summed: tokens down to 2^-30 of the largest weight stay
// normal numbers, 56 + 40 + 30 = 126.  A row's first tile decides it.
constexpr float kBelowScaled = 56.f;
// References up to which a score may keep its product's low bits while the
// reference, a rounded product, does not: they differ by 2^-24 of it, 1/16 here.
// Beyond, both are rounded alike (else 2^32 could leave an exponent of 256).
constexpr float kFused = 1048576.f;

// kind::f16 with fp16 or bf16 operands, fp32 accumulators, 128 x 128.
constexpr uint32_t kIdescBf16 = ptx::idesc_bf16_f32(128, 128);
constexpr uint32_t kIdescF16 = kIdescBf16 & ~((7u << 7) | (7u << 10));

// ptx::wait_bar without its suspension hint: a waiting warp sleeps for the
// hardware's own short time, which wakes it sooner than the hint does; the
// clock and the abort flag are looked at once in 64 tries.
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity, volatile int* abort, int* error) {
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    const uint64_t now = ptx::global_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > ptx::kWaitLimitNs) {
      *abort = 1;
      atomicCAS(error, 0, kErrTimeout);
      return false;
    }
  }
}

// ---- work items ------------------------------------------------------------

// Token of row r of a sequence and KV head: r / group.
__device__ __forceinline__ int row_token(const ExtendArgs& a, int r) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(r)) * a.group_mul) >> (31 + a.group_shift));
}

// Key tiles of row tile i (`rows` rows) of a sequence: those its last token
// sees, at least one (rows that see nothing still need their zero output).
__device__ __forceinline__ int key_tiles(const ExtendArgs& a, int i, int rows, int n_new, int ctx) {
  const int last = min(n_new - 1, row_token(a, rows * (i + 1) - 1));
  const int seen = ctx - n_new + last + 1;
  return seen <= kTile ? 1 : (seen + kTile - 1) / kTile;
}
__device__ __forceinline__ int row_tiles(int rows, int n_new, int group) {
  return static_cast<int>((static_cast<long long>(n_new) * group + rows - 1) / rows);
}

// A work item: a row tile of a sequence and KV head.
struct Item {
  int b, kvh, i;       // sequence, KV head, row tile
  int tiles;           // its key tiles
  int4 seq;            // first row, new tokens, context, first expanded tile
};

// A CTA's run of work.  Work is counted in units: an item has f.cost units for
// its beginning and end, then one per key tile, so that many short items weigh
// what they take.  Every CTA has an equal run of units; what it works on is
// the key tiles among them.
struct Run {
  long long pos, end;  // units
  int offset;          // of pos in the item
  Item it;
};
__device__ __forceinline__ long long run_length(long long total, int ctas) { return (total + ctas - 1) / ctas; }

// The item of form `f` that holds unit `pos`, and the offset in it (found by a whole warp).
__device__ __forceinline__ Item find_item(const ExtendArgs& a, const ExtendForm& f, long long pos, int* offset) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.d.batch;                     // the last sequence that starts at or before pos
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (f.first[mid] <= pos) lo = mid;
    else hi = mid;
  }
  Item it;
  it.b = lo;
  it.seq = a.ws_seq[lo];
  const long long per_head = (f.first[lo + 1] - f.first[lo]) / a.d.n_kv;
  long long rem = pos - f.first[lo];
  it.kvh = static_cast<int>(rem / per_head);
  rem -= it.kvh * per_head;
  const int mt = row_tiles(f.rows, it.seq.y, a.d.group);
  it.i = 0;
  it.tiles = 0;
  *offset = 0;
  for (int i0 = 0; i0 < mt; i0 += 32) {
    const int nt = i0 + lane < mt ? key_tiles(a, i0 + lane, f.rows, it.seq.y, it.seq.z) : 0;
    const long long units = i0 + lane < mt ? nt + f.cost : 0;
    long long upto = units;
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
      *offset = static_cast<int>(rem - __shfl_sync(0xffffffffu, upto - units, src));
      break;
    }
    rem -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return it;
}

__device__ __forceinline__ void next_item(const ExtendArgs& a, const ExtendForm& f, Item& it) {
  if (++it.i >= row_tiles(f.rows, it.seq.y, a.d.group)) {
    it.i = 0;
    if (++it.kvh >= a.d.n_kv) {
      it.kvh = 0;
      do {
        ++it.b;
      } while (f.first[it.b + 1] == f.first[it.b]);
      it.seq = a.ws_seq[it.b];
    }
  }
  it.tiles = key_tiles(a, it.i, f.rows, it.seq.y, it.seq.z);
}

// The run's next segment: key tiles t0 .. t1 - 1 of r.it.  `end_segment` moves behind it.
__device__ __forceinline__ bool next_segment(const ExtendArgs& a, const ExtendForm& f, Run& r, int& t0, int& t1) {
  while (r.pos < r.end) {
    const long long left = r.end - r.pos;
    const int units = f.cost + r.it.tiles;
    const int upto = left < units - r.offset ? r.offset + static_cast<int>(left) : units;
    t0 = max(0, r.offset - f.cost);
    t1 = max(0, upto - f.cost);
    if (t0 < t1) return true;
    r.pos += upto - r.offset;                     // (the run ends before the item's first key tile)
  }
  return false;
}
__device__ __forceinline__ void end_segment(const ExtendArgs& a, const ExtendForm& f, Run& r, int t1) {
  r.pos += f.cost + t1 - r.offset;
  r.offset = 0;
  if (r.pos < r.end) next_item(a, f, r.it);
}

// A test of the bounded waits: the run with the form's first key tile withholds
// its first product's completion.
__device__ __forceinline__ bool withheld(const ExtendArgs& a, const ExtendForm& f, long long per, int seg) {
  return a.d.debug_withhold && seg == 0 && blockIdx.x == f.cost / per;
}

// What run blockIdx.x leaves for the join: the item it begins and does not
// end, if any (one thread, before the run is walked; `any`: the run has work).
__device__ __forceinline__ void write_cut(const ExtendArgs& a, const ExtendForm& f, Run r, long long per, bool any) {
  CutItem cut{0, 0, 0, 0, 0};
  int t0, t1;
  while (any && next_segment(a, f, r, t0, t1)) {
    if (t0 == 0 && t1 < r.it.tiles) {
      const long long first = r.pos - r.offset + f.cost;        // unit of its first key tile
      cut.row0 = r.it.seq.x;
      cut.kvh = r.it.kvh;
      cut.i = r.it.i;
      cut.rows = min(f.rows, r.it.seq.y * a.d.group - r.it.i * f.rows);
      cut.last = static_cast<int>((first + r.it.tiles - 1) / per);
    }
    end_segment(a, f, r, t1);
  }
  f.cuts[blockIdx.x] = cut;
}

// Floats of a partial output: the rows' outputs, then their (reference, sum).
__host__ __device__ constexpr int part_floats(int rows) { return rows * (kDim + 2); }

// ---- expansion of packed bits ------------------------------------------------

template <int OFFSET>
__device__ __forceinline__ void store16(uint32_t saddr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0 + %5], {%1, %2, %3, %4};"
               ::"r"(saddr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "n"(OFFSET)
               : "memory");
}
__device__ __forceinline__ float4 load16(const float* p) { return *reinterpret_cast<const float4*>(p); }

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

__device__ __forceinline__ RowChunks next_block(const RowChunks& r) {
  return RowChunks{{r.at[0] + kBlockBytes, r.at[1] + kBlockBytes, r.at[2] + kBlockBytes, r.at[3] + kBlockBytes}};
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

// The sketch's factor as fp16 numbers for four groups of sixteen coordinates
// of a half (`half`), as the two packed words that expand_signs takes.  One
// rounding for all 128 coordinates would be off by up to 2^-11 of the whole
// sketch; instead as many of the eight groups take the number above rho as make
// the mean right to 2^-14.5, and what is left differs in sign from coordinate
// to coordinate.  (24 sequences of 1 to 16 tokens: 389 us in place of 384; two
// sketch scores of 60 differ by 0.007 in the rms where one rounding left 0.023.)
__device__ __forceinline__ uint2 minus_factors(float rho, int half) {
  const uint32_t below = __half_as_ushort(__float2half_rd(rho));
  const float lo = __half2float(__ushort_as_half(below)), hi = __half2float(__ushort_as_half(below + 1));
  const float above = __fdividef(rho - lo, hi - lo) * 8.f;      // groups, of eight (0, 4, 2, 6 | 1, 5, 3, 7 in order)
  const float first = above - 0.5f - half;
  const uint32_t x = (first > 0.f ? 1u : 0u) + (first > 4.f ? 0x10000u : 0u);
  const uint32_t y = (first > 2.f ? 1u : 0u) + (first > 6.f ? 0x10000u : 0u);
  const uint32_t both = below * 0x00010001u;
  return make_uint2((both + x) ^ 0x80008000u, (both + y) ^ 0x80008000u);
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
// What is left of (lo, hi) beside the bf16 pair `w`, as another one.
__device__ __forceinline__ uint32_t remainder_bf16(float lo, float hi, uint32_t w) {
  return pack_bf16(lo - __uint_as_float(w << 16), hi - __uint_as_float(w & 0xffff0000u));
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
__device__ __forceinline__ int exponent_of(float x) {   // clamped so that 2^e and 2^-e are normal numbers
  const int e = static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127;
  return e < -126 ? -126 : (e > 126 ? 126 : e);
}

__device__ __forceinline__ void unpack_bf16(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_query8(const ExtendArgs& a, long long at, float (&v)[8]) {
  if (a.q_bf16) {
    unpack_bf16(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.d.q) + at), v);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.d.q) + at);
    const float4 x = p[0], y = p[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
}

// A thread's own 16-byte copies global -> shared, and the wait for them.
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Vector (token x query head) of row r of an item's sequence and KV head.
__device__ __forceinline__ long long row_vector(const ExtendArgs& a, int row0, int kvh, int r) {
  const int tok = row_token(a, r);
  return (static_cast<long long>(row0) + tok) * a.d.n_q + kvh * a.d.group + r - tok * a.d.group;
}

// Brings the query rows of the run's next item to L2 while a segment that ends
// with key tile t1 is worked on: they come from far memory, and a segment
// begins with them.
__device__ __forceinline__ void prefetch_queries(const ExtendArgs& a, const ExtendForm& f, const Run& r, int t1, int t,
                                                 int threads) {
  if (r.pos + f.cost + t1 - r.offset >= r.end) return;
  Item it = r.it;
  next_item(a, f, it);
  const int lines = a.q_bf16 ? 2 : 4;             // of 128 bytes
  const int rows = min(f.rows, it.seq.y * a.d.group - it.i * f.rows);
  for (int k = t; k < rows * lines; k += threads) {
    const long long vec = row_vector(a, it.seq.x, it.kvh, it.i * f.rows + k / lines);
    const char* const p = static_cast<const char*>(a.d.q) + (vec * lines + k % lines) * 128;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
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
// ---- softmax of a score tile ---------------------------------------------------
//
// A thread has 64 scores of its row at tensor-memory columns s .. s + 63 and
// leaves its weights (bf16 pairs) in the first 32 of them, and what the
// rounding left of the last sixteen in the next 8 (another step of the output
// product).  kf, vf: the columns' key and value factors in shared memory.
//
// The weights' rounding is as large as the output's own (1.7e-3 of it each in
// the rms); every other rounding brings the sum to 1.5 times the latter.  A
// quarter of the remainders makes it 1.4.

// The row's reference after a search found `top` (-inf: nothing visible).  A
// first maximum in bounds leaves zero, as it would be without the search, so
// that what other rows see does not change a row's bits.  below: how far it may
// lie below that (kRaise or kBelowScaled).
__device__ __forceinline__ float raised(float ref, float top, float below) {
  if (ref == -INFINITY) return top >= -below && top <= kRaise ? 0.f : top;
  return top > ref + kRaise ? top : ref;
}

// No score hidden, none that may pass the reference by 2^kRaise.
__device__ __forceinline__ void weigh_usual(uint32_t s, const float* kf, const float* vf, float ref, uint64_t& sum2) {
  const uint64_t minus = pair(-ref, -ref);
  uint32_t x[2][16], rest[8];
  tmem_ld16_start(s, x[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tmem_ld16_wait(x[c & 1]);
    if (c < 3) tmem_ld16_start(s + 16 * (c + 1), x[(c + 1) & 1]);
    const uint32_t(&y)[16] = x[c & 1];
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 f = load16(kf + 16 * c + 4 * k);
      const float2 z0 = unpair(fma2(pair(__uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1])), pair(f.x, f.y), minus));
      const float2 z1 =
          unpair(fma2(pair(__uint_as_float(y[4 * k + 2]), __uint_as_float(y[4 * k + 3])), pair(f.z, f.w), minus));
      const uint64_t p0 = pair(exp2_fast(z0.x), exp2_fast(z0.y)), p1 = pair(exp2_fast(z1.x), exp2_fast(z1.y));
      sum2 = add2(sum2, add2(p0, p1));
      const float4 g = load16(vf + 16 * c + 4 * k);
      const float2 w0 = unpair(mul2(p0, pair(g.x, g.y))), w1 = unpair(mul2(p1, pair(g.z, g.w)));
      w[2 * k] = pack_bf16(w0.x, w0.y);
      w[2 * k + 1] = pack_bf16(w1.x, w1.y);
      if (c == 3) {
        rest[2 * k] = remainder_bf16(w0.x, w0.y, w[2 * k]);
        rest[2 * k + 1] = remainder_bf16(w1.x, w1.y, w[2 * k + 1]);
      }
    }
    ptx::tmem_st8(s + 8 * c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  }
  ptx::tmem_st8(s + 32, rest[0], rest[1], rest[2], rest[3], rest[4], rest[5], rest[6], rest[7]);
}

// As weigh_usual where a group's 32 columns have one key factor and one power of
// two 2^e as value factor (the 8-bit cache): the exponent takes it, the sum gives
// it back once a group.  (A row's largest weight is 2^-kBelowScaled or more.)
__device__ __forceinline__ void weigh_grouped(uint32_t s, const float* kf, const float* vf, float ref, uint64_t& sum2) {
  uint32_t x[2][16], rest[8];
  tmem_ld16_start(s, x[0]);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float f = kf[32 * g];
    const int e = exponent_of(vf[32 * g]);
    const uint64_t factor = pair(f, f), shift = pair(e - ref, e - ref);
    uint64_t part = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 2 * g + h;
      tmem_ld16_wait(x[c & 1]);
      if (c < 3) tmem_ld16_start(s + 16 * (c + 1), x[(c + 1) & 1]);
      const uint32_t(&y)[16] = x[c & 1];
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 z = unpair(fma2(pair(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), factor, shift));
        const float p0 = exp2_fast(z.x), p1 = exp2_fast(z.y);
        part = add2(part, pair(p0, p1));
        w[k] = pack_bf16(p0, p1);
        if (c == 3) rest[k] = remainder_bf16(p0, p1, w[k]);
      }
      ptx::tmem_st8(s + 8 * c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    }
    sum2 = fma2(part, pair(exp2_int(-e), exp2_int(-e)), sum2);
  }
  ptx::tmem_st8(s + 32, rest[0], rest[1], rest[2], rest[3], rest[4], rest[5], rest[6], rest[7]);
}
// As plain_top for such columns (their key factors are not negative).
__device__ __forceinline__ float grouped_top(uint32_t s, const float* kf) {
  float top[2] = {-INFINITY, -INFINITY};
  uint32_t x[2][16];
  tmem_ld16_start(s, x[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tmem_ld16_wait(x[c & 1]);
    if (c < 3) tmem_ld16_start(s + 16 * (c + 1), x[(c + 1) & 1]);
    const uint32_t(&y)[16] = x[c & 1];
#pragma unroll
    for (int k = 0; k < 16; ++k) top[c >> 1] = fmaxf(top[c >> 1], __uint_as_float(y[k]));
  }
  return fmaxf(top[0] * kf[0], top[1] * kf[32]);
}

// Visible tokens of group g (32 bits by token) when `here` of the tile's are
// behind the row's position limit.
__device__ __forceinline__ uint32_t visible(const uint32_t* valid, int here, int g) {
  const int n = min(32, max(0, here - 32 * g));
  return (n == 32 ? 0xffffffffu : (1u << n) - 1u) & valid[g];
}

// The largest of the thread's scores.
__device__ __forceinline__ float plain_top(uint32_t s, const float* kf) {
  float top = -INFINITY;
  uint32_t x[2][16];
  tmem_ld16_start(s, x[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tmem_ld16_wait(x[c & 1]);
    if (c < 3) tmem_ld16_start(s + 16 * (c + 1), x[(c + 1) & 1]);
    const uint32_t(&y)[16] = x[c & 1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 f = load16(kf + 16 * c + 4 * k);
      top = fmaxf(fmaxf(top, __uint_as_float(y[4 * k]) * f.x), __uint_as_float(y[4 * k + 1]) * f.y);
      top = fmaxf(fmaxf(top, __uint_as_float(y[4 * k + 2]) * f.z), __uint_as_float(y[4 * k + 3]) * f.w);
    }
  }
  return top;
}

// The same of the visible scores, or of a scaled query.
__device__ __forceinline__ float masked_top(uint32_t s, const float* kf, float factor, const uint32_t* valid, int here,
                                            int half) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const uint32_t mask = visible(valid, here, 2 * half + c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t y[16];
      ptx::tmem_ld16(s + 32 * c + 16 * h, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 f = load16(kf + 32 * c + 16 * h + 4 * k);
        const float fk[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = __uint_as_float(y[4 * k + q]) * fk[q] * factor;
          top = mask & (1u << expanded_bit(16 * h + 4 * k + q)) ? fmaxf(top, v) : top;
        }
      }
    }
  }
  return top;
}

__device__ __forceinline__ float weigh_masked(uint32_t s, const float* kf, const float* vf, float factor, float shift,
                                              const uint32_t* valid, int here, int half) {
  float sum = 0.f;
  uint32_t rest[8];                               // (of the last sixteen)
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const uint32_t mask = visible(valid, here, 2 * half + c);
    if (!__any_sync(0xffffffffu, mask != 0)) {    // no row of the warp sees them
#pragma unroll
      for (int h = 0; h < 2; ++h) ptx::tmem_st8(s + 16 * c + 8 * h, 0, 0, 0, 0, 0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) rest[k] = 0;
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t y[16], w[8];
      ptx::tmem_ld16(s + 32 * c + 16 * h, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 f = load16(kf + 32 * c + 16 * h + 4 * k);
        const float4 g = load16(vf + 32 * c + 16 * h + 4 * k);
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
        rest[2 * k] = remainder_bf16(p[0], p[1], w[2 * k]);
        rest[2 * k + 1] = remainder_bf16(p[2], p[3], w[2 * k + 1]);
      }
      ptx::tmem_st8(s + 16 * c + 8 * h, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    }
  }
  ptx::tmem_st8(s + 32, rest[0], rest[1], rest[2], rest[3], rest[4], rest[5], rest[6], rest[7]);
  return sum;
}

// 64 columns of the output so far, scaled.
__device__ __forceinline__ void scale_output(uint32_t o, float scale) {
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint32_t y[8];
    tmem_ld8(o + 8 * c, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * scale);
    ptx::tmem_st8(o + 8 * c, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
  }
}

// The largest of 64 columns of the output.  (A bound from the values' norms
// would save this pass, but a huge value that a row does not see would push
// the row's output out of fp16's range.)
__device__ __forceinline__ float largest_output(uint32_t o, float inv) {
  float top = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t y[16];
    ptx::tmem_ld16(o + 16 * c, y);
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(__uint_as_float(y[k]) * inv));
  }
  return top;
}

// 64 columns of the output, divided by the row's sum and by a power of two, as
// an fp16 operand at `dst` (32 columns).  (One after the other: the two factors'
// product can pass fp32's range, and zero times infinity is no zero.)
__device__ __forceinline__ void output_operand(uint32_t o, uint32_t dst, float inv, float down) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t y[16], w[8];
    ptx::tmem_ld16(o + 16 * c, y);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[k] = pack_f16(__uint_as_float(y[2 * k]) * inv * down, __uint_as_float(y[2 * k + 1]) * inv * down);
    ptx::tmem_st8(dst + 8 * c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  }
}

// The turned output's 64 columns, as fp32 to a partial.
__device__ __forceinline__ void store_partial(uint32_t o, float scale, float* part, bool live) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t y[16];
    ptx::tmem_ld16(o + 16 * c, y);
    if (live) {
      float4* const dst = reinterpret_cast<float4*>(part + 16 * c);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        dst[k] = make_float4(__uint_as_float(y[4 * k]) * scale, __uint_as_float(y[4 * k + 1]) * scale,
                             __uint_as_float(y[4 * k + 2]) * scale, __uint_as_float(y[4 * k + 3]) * scale);
    }
  }
}

// The same as bf16 to the output row.
__device__ __forceinline__ void store_row(uint32_t o, float scale, __nv_bfloat16* out, bool live) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t y[16];
    ptx::tmem_ld16(o + 16 * c, y);
    if (live) {
      uint4* const dst = reinterpret_cast<uint4*>(out + 16 * c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] = pack_bf16(__uint_as_float(y[8 * k + 2 * q]) * scale, __uint_as_float(y[8 * k + 2 * q + 1]) * scale);
        dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// The same as bf16 into eight swizzled 16-byte chunks of a row in shared memory.
__device__ __forceinline__ void output_rows(uint32_t o, float scale, uint8_t* dst, int row) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t y[16], w[8];
    ptx::tmem_ld16(o + 16 * c, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16(__uint_as_float(y[2 * k]) * scale, __uint_as_float(y[2 * k + 1]) * scale);
    *reinterpret_cast<uint4*>(dst + (((2 * c) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(dst + (((2 * c + 1) ^ (row & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

}  // namespace
}  // namespace tq
