// kv4.cuh -- layout and batch arithmetic of the 4-bit paged cache (include/pnmix.h), shared
// by its kernels.
#pragma once

#include "common.cuh"

namespace pnmix {
namespace kv4 {

constexpr int kBlock = 16;           // tokens of a block, the unit of the layout
constexpr int kMaxBatch = 2048;
constexpr float kLimit = 61440.0f;   // magnitudes are stored up to this

// A validated configuration and cache, by value to the kernels.
struct Geo {
  int Hq, Hkv, G, D;
  int page_shift;         // log2 page_tokens
  int n_pages;
  float scale;
  uint8_t* pages;
  uint32_t* error;
  uint32_t wait_limit;    // try_wait rounds before a wait for staged pages gives up
  int skip_seq;           // test hook: the sequence whose pages are never staged (-1: none)
};

// A validated batch.
struct Batch {
  int B, n_tokens, max_pages, max_q;
  int uniform;            // rows of every sequence when there is no q_start
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
};

__host__ __device__ __forceinline__ int block_bytes(int D) { return 20 * D; }

struct Rows {
  const uint16_t* p;
  long long ts, hs;
};

// Rows [start, start + n) of sequence b; false if q_start is not ascending within
// [0, n_tokens] there, or the sequence has more than max_q rows.
__device__ __forceinline__ bool seq_rows(const Batch& bt, int b, int& start, int& n) {
  if (!bt.q_start) {
    start = b * bt.uniform;
    n = bt.uniform;
    return true;
  }
  start = bt.q_start[b];
  n = bt.q_start[b + 1] - start;
  return start >= 0 && n >= 0 && start <= bt.n_tokens - n && n <= bt.max_q;
}

// Tokens sequence b holds, clamped to what its page table can hold.
__device__ __forceinline__ int seq_len(const Batch& bt, int page_shift, int b, bool& bad) {
  const int raw = bt.kv_len[b], cap = bt.max_pages << page_shift;
  const int n = min(max(raw, 0), cap);
  bad |= raw != n;
  return n;
}

// Sets bits of the device error word.
__device__ __forceinline__ void raise(uint32_t* error, uint32_t bits) {
  atomicOr(error, bits);
}

// Where piece w of token t's value row lies (see the layout): 8-byte pieces are crossed in
// every other token pair, so the lanes of a warp that read four tokens' pieces at once meet
// in no shared-memory bank.
template <int D>
__device__ __forceinline__ int value_place(int t, int w) {
  return D == 128 ? w ^ (((t >> 1) & 1) << 2) : w;
}

}  // namespace kv4
}  // namespace pnmix
