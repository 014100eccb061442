// Token map of one step: context lengths, query starts, positions, slots and
// freshly taken cache blocks, from the sequences' lengths, on the device.
//
//   context[b]  = past[b] + fresh[b]
//   start[b]    = sum of fresh over the sequences before b
//   taken       = ceil(context / block) - ceil(past / block) blocks per
//                 sequence, handed out from the free list in sequence order
//   token t of b: position past[b] + t - start[b], slot from the block table
//
// Everything follows from two prefix sums over the batch (tokens and blocks),
// which are a few KB: every CTA forms both in shared memory instead of waiting
// for another launch, then takes 1024 tokens (a binary search in the starts
// finds a token's sequence) and every gridDim-th group of sequences of the
// block table.  A token in a fresh block reads its block id from the free
// list itself, so no CTA reads a table entry that another one writes.
// The bytes are a few MB at most and the call is bound by its launch and one
// chain of dependent loads (lengths, then table or free list): 6 us for a
// decode step of 64 sequences, 8 us for 250 mixed ones, 9 us for 500 prompts of
// up to 4000 tokens (2.8 MB, 0.4 us at the copy rate).
#include "kernels.h"

namespace tq {
namespace {

constexpr int kMapThreads = 256;
constexpr int kMapTokens = 1024;      // tokens per CTA

__device__ __forceinline__ int saturate(long long x) { return x > 0x7fffffffll ? 0x7fffffff : static_cast<int>(x); }

struct Pair {
  long long tokens, blocks;
};

// Lengths of sequence b; out-of-range lengths count as an empty sequence.
__device__ __forceinline__ bool sequence_lengths(const TokenMapArgs& a, int b, int* past, int* fresh) {
  const long long p = a.past_lens[b], n = a.new_lens[b];
  const bool ok = p >= 0 && n >= 0 && p + n <= static_cast<long long>(a.max_blocks) * a.block_size;
  *past = ok ? static_cast<int>(p) : 0;
  *fresh = ok ? static_cast<int>(n) : 0;
  return ok;
}

__device__ __forceinline__ int blocks_of(int tokens, int block_size) {
  return tokens / block_size + (tokens % block_size != 0);
}

// The i-th block of the free list, or -1 (recorded) when the list is too
// short or holds an id outside the cache.
__device__ __forceinline__ int free_block(const TokenMapArgs& a, long long i) {
  if (i >= a.n_free) {
    atomicCAS(a.error, 0, kErrNoBlock);
    return -1;
  }
  const int id = a.free_blocks[i];
  if (id < 0 || id >= a.num_blocks) {
    atomicCAS(a.error, 0, kErrBlock);
    return -1;
  }
  return id;
}

__global__ void __launch_bounds__(kMapThreads) token_map_kernel(TokenMapArgs a) {
  extern __shared__ int map_s[];
  int* const start_s = map_s;                     // [batch + 1]
  int* const first_s = map_s + a.batch + 1;       // [batch]: taken blocks before the sequence's first
  __shared__ Pair warp_sum[kMapThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  Pair carry{0, 0};
  for (int b0 = 0; b0 < a.batch; b0 += kMapThreads) {
    const int b = b0 + tid;
    int past = 0, fresh = 0;
    if (b < a.batch) {
      const bool ok = sequence_lengths(a, b, &past, &fresh);
      if (blockIdx.x == 0) {
        a.context_lens[b] = past + fresh;
        if (!ok) atomicCAS(a.error, 0, kErrContext);
      }
    }
    const Pair own{fresh, blocks_of(past + fresh, a.block_size) - blocks_of(past, a.block_size)};
    Pair sum = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, sum.tokens, d);
      const long long k = __shfl_up_sync(0xffffffffu, sum.blocks, d);
      if (lane >= d) {
        sum.tokens += t;
        sum.blocks += k;
      }
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    Pair total = carry;
#pragma unroll
    for (int w = 0; w < kMapThreads / 32; ++w) {
      if (w == warp) {
        sum.tokens += total.tokens;
        sum.blocks += total.blocks;
      }
      total.tokens += warp_sum[w].tokens;
      total.blocks += warp_sum[w].blocks;
    }
    if (b < a.batch) {
      start_s[b] = saturate(sum.tokens - own.tokens);
      first_s[b] = saturate(sum.blocks - own.blocks);
      if (blockIdx.x == 0) a.query_start[b] = start_s[b];
    }
    carry = total;
    __syncthreads();
  }
  if (tid == 0) {
    start_s[a.batch] = saturate(carry.tokens);
    if (blockIdx.x == 0) {
      a.query_start[a.batch] = saturate(carry.tokens);
      *a.blocks_taken = saturate(carry.blocks);
      if (carry.tokens > a.n_tokens) atomicCAS(a.error, 0, kErrTokens);
    }
  }
  __syncthreads();

  // fresh block table entries: one warp per sequence, lanes over its blocks
  for (int b = blockIdx.x * (kMapThreads / 32) + warp; b < a.batch; b += gridDim.x * (kMapThreads / 32)) {
    int past, fresh;
    sequence_lengths(a, b, &past, &fresh);
    const int before = blocks_of(past, a.block_size), after = blocks_of(past + fresh, a.block_size);
    for (int c = before + lane; c < after; c += 32)
      a.block_table[static_cast<long long>(b) * a.max_blocks + c] =
          free_block(a, static_cast<long long>(first_s[b]) + c - before);
  }

  // tokens
  const int total = start_s[a.batch];
  const long long t_end = min(static_cast<long long>(a.n_tokens), (blockIdx.x + 1ll) * kMapTokens);
  for (long long t = static_cast<long long>(blockIdx.x) * kMapTokens + tid; t < t_end; t += kMapThreads) {
    int pos = -1;
    long long slot = -1;
    if (t < total) {
      int lo = 0, hi = a.batch;                   // the last sequence that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start_s[mid] <= t) lo = mid;
        else hi = mid;
      }
      int past, fresh;
      sequence_lengths(a, lo, &past, &fresh);
      pos = past + static_cast<int>(t - start_s[lo]);
      const int before = blocks_of(past, a.block_size), col = pos / a.block_size;
      int id;
      if (col >= before) {
        id = free_block(a, static_cast<long long>(first_s[lo]) + col - before);
      } else {
        id = a.block_table[static_cast<long long>(lo) * a.max_blocks + col];
        if (id < 0 || id >= a.num_blocks) {
          atomicCAS(a.error, 0, kErrBlock);
          id = -1;
        }
      }
      if (id >= 0) slot = static_cast<long long>(id) * a.block_size + pos % a.block_size;
    }
    a.positions[t] = pos;
    a.slot_mapping[t] = slot;
  }
}

}  // namespace

cudaError_t launch_token_map(const TokenMapArgs& a, cudaStream_t stream) {
  constexpr size_t kMost = (2 * kMapMaxBatch + 1) * sizeof(int);
  static_assert(kMost <= 100 * 1024, "the starts of a batch fit in shared memory");
  const size_t smem = (2 * static_cast<size_t>(a.batch) + 1) * sizeof(int);
  if (smem > 40 * 1024) {
    // (the limit is the process's: calls of other threads must not lower it, so it is the largest batch's)
    const cudaError_t err = cudaFuncSetAttribute(token_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (err != cudaSuccess) return err;
  }
  // enough CTAs for the tokens, and for eight sequences of the table per warp
  const int by_tokens = a.n_tokens / kMapTokens + (a.n_tokens % kMapTokens != 0);
  const int by_table = (a.batch + 63) / 64;
  const int grid = by_tokens > by_table ? by_tokens : by_table;
  token_map_kernel<<<grid > 0 ? grid : 1, kMapThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
