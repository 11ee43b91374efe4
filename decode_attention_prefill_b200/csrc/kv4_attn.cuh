// kv4_attn.cuh -- work partition and partial results of the attention over the 4-bit paged
// cache.
//
// A UNIT is a tile of RT query rows of one (sequence b, KV head h): row r of the T * G rows is
// token j = r / G of the sequence's new tokens, query head h * G + r % G.  A unit counts
// `lead` items for its fixed cost and one item per ITEM tokens of the sequence.  Units are
// numbered b-major, then h, then tile; their items are numbered in that order, X in total,
// and CTA i of N takes [floor(i X / N), floor((i + 1) X / N)).  Every CTA works the numbers
// out from q_start and kv_len itself (a block-wide prefix sum), so any mix of lengths is
// balanced and the host needs to know none.  A piece of a unit that does not cover it whole
// leaves a partial (m, l, O) per row in slot i + unit (the slots of a unit are contiguous and
// disjoint from other units'), which the combine kernel merges; a CTA that has a unit to
// itself writes its rows at once.
#pragma once

#include "decode_frag.cuh"
#include "kv4.cuh"

namespace pnmix {
namespace kv4 {

struct UnitInfo {     // of a unit that several CTAs share; first < 0: nothing to merge
  int first, last;    // CTAs
  int b, h, tile, pad[3];
};

struct Work {
  float* part;        // [slots][RT][D + 4]: m, l, -, -, O
  UnitInfo* info;     // [units], each written by the CTA that holds the unit's first item
  int* count;         // units
};

__host__ __device__ __forceinline__ int part_stride(int D) { return D + 4; }

// Host bound of the number of units: sum over b of Hkv * ceil(G T_b / RT).
__host__ __forceinline__ long long max_units(const Geo& g, const Batch& bt, int rt) {
  return static_cast<long long>(g.Hkv) * (bt.B + static_cast<long long>(bt.n_tokens) * g.G / rt);
}

struct Piece {
  int b, h, tile, unit;
  int lo, hi;             // items of the unit past its lead, [lo, hi)
  int first, last;        // CTAs that share the unit
  int start, T, len;      // rows and tokens of the sequence
};

__device__ __forceinline__ int cta_of_item(long long x, long long X, int N) {
  return static_cast<int>(((x + 1) * N - 1) / X);
}

// Shared-memory bytes of the prefix sums.
__host__ __device__ __forceinline__ size_t plan_bytes(int B) { return (static_cast<size_t>(B) + 1) * 12 + 4; }

// Prefix sums over the sequences: items[b] and units[b] before sequence b.  All threads of
// the CTA call it.  Row ranges that are out of order or out of the tensors could name more
// rows than the workspace is made for, so with any of those there is no work at all.
template <int THREADS>
__device__ __forceinline__ void build_plan(const Geo& g, const Batch& bt, int RT, int item, int lead,
                                           long long* items, int* units, long long* tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = THREADS / 32;
  long long carry_i = 0;
  int carry_u = 0;
  bool bad = false, bad_len = false;
  for (int base = 0; base < bt.B; base += THREADS) {
    const int b = base + tid;
    long long it = 0;
    int un = 0;
    if (b < bt.B) {
      int start, T;
      if (!seq_rows(bt, b, start, T)) {
        bad = true;
        T = 0;
      }
      const int len = seq_len(bt, g.page_shift, b, bad_len);
      un = g.Hkv * ((T * g.G + RT - 1) / RT);
      it = static_cast<long long>(un) * (lead + (len + item - 1) / item);
    }
    long long si = it;
    int su = un;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long vi = __shfl_up_sync(0xffffffffu, si, o);
      const int vu = __shfl_up_sync(0xffffffffu, su, o);
      if (lane >= o) {
        si += vi;
        su += vu;
      }
    }
    if (lane == 31) {
      tmp[2 * warp] = si;
      tmp[2 * warp + 1] = su;
    }
    __syncthreads();
    long long off_i = carry_i;
    int off_u = carry_u;
    for (int w = 0; w < kWarps; ++w) {
      const long long wi = tmp[2 * w];
      const int wu = static_cast<int>(tmp[2 * w + 1]);
      if (w < warp) {
        off_i += wi;
        off_u += wu;
      }
      carry_i += wi;
      carry_u += wu;
    }
    if (b < bt.B) {
      items[b] = off_i + si - it;
      units[b] = off_u + su - un;
    }
    __syncthreads();
  }
  const bool none = __syncthreads_or(bad);
  if (tid == 0) {
    items[bt.B] = none ? 0 : carry_i;
    units[bt.B] = none ? 0 : carry_u;
  }
  if ((bad || bad_len) && blockIdx.x == 0) raise(g.error, PNMIX_DEVERR_BATCH);
  __syncthreads();
}

// Calls fn(piece) for every piece of this CTA, in order; uniform across the CTA.
template <typename F>
__device__ __forceinline__ void for_each_piece(const Geo& g, const Batch& bt, int RT, int item, int lead,
                                               const long long* items, const int* units, const Work& wk, int grid,
                                               F&& fn) {
  const long long X = items[bt.B];
  const int N = X < grid ? static_cast<int>(X) : grid, i = blockIdx.x;
  if (i == 0 && threadIdx.x == 0) *wk.count = units[bt.B];
  if (i >= N) return;
  long long x = X * i / N;
  const long long e = X * (i + 1) / N;
  int lo = 0, hi = bt.B - 1;   // the sequence that holds item x: the last b with items[b] <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (items[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  int b = lo;
  while (x < e) {
    while (items[b + 1] <= x) ++b;   // sequences without rows hold no items
    bool bad = false;
    Piece p;
    p.b = b;
    seq_rows(bt, b, p.start, p.T);
    p.len = seq_len(bt, g.page_shift, b, bad);
    const long long per = lead + (p.len + item - 1) / item;
    const int tiles = (p.T * g.G + RT - 1) / RT;
    const int u = static_cast<int>((x - items[b]) / per);
    const long long ustart = items[b] + u * per, uend = ustart + per;
    const long long xe = uend < e ? uend : e;
    p.h = u / tiles;
    p.tile = u - p.h * tiles;
    p.unit = units[b] + u;
    p.lo = static_cast<int>(max(x - ustart - lead, 0ll));
    p.hi = static_cast<int>(max(xe - ustart - lead, 0ll));
    p.first = cta_of_item(ustart, X, N);
    p.last = cta_of_item(uend - 1, X, N);
    if (threadIdx.x == 0 && x == ustart) {
      UnitInfo f;
      f.first = p.first == p.last ? -1 : p.first;
      f.last = p.last;
      f.b = p.b;
      f.h = p.h;
      f.tile = p.tile;
      wk.info[p.unit] = f;
    }
    fn(p);
    x = xe;
  }
}

}  // namespace kv4
}  // namespace pnmix
