// kv4_attn.cuh -- work partition and partial results of the attention over the 4-bit paged
// cache.
//
// A UNIT is a tile of RT query rows of one (sequence b, KV head h): row r of the T * G rows is
// token j = r / G of the sequence's new tokens, query head h * G + r % G.  Its cost is counted
// in tokens: `lead` for its fixed part, and an upper bound of what its last row sees, which
// grows by ceil(RT / G) from one tile to the next.  Units are numbered b-major, then h, then
// tile; their tokens are numbered in that order, X in total, and CTA i of N takes
// [floor(i X / N), floor((i + 1) X / N)).  Every CTA works the numbers out from q_start and
// kv_len itself (a block-wide prefix sum), so any mix of lengths is balanced and the host
// needs to know none.  A CTA that has a unit to itself writes its rows at once.  A piece of a
// unit that does not cover it leaves a partial (m, l, O) per row, and the merge kernel joins
// them: only the first and the last piece of a CTA can be such, so two slots per CTA do.
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
  float* part;        // [2 N][RT][D + 4]: m, l, -, -, O
  UnitInfo* info;     // [units], each written by the CTA that holds the unit's first token
  int* count;         // units
};

__host__ __device__ __forceinline__ int part_stride(int D) { return D + 4; }

// Host bound of the number of units: sum over b of Hkv * ceil(G T_b / RT).
__host__ __forceinline__ long long max_units(const Geo& g, const Batch& bt, int rt) {
  return static_cast<long long>(g.Hkv) * (bt.B + static_cast<long long>(bt.n_tokens) * g.G / rt);
}

struct Piece {
  int b, h, tile;
  int lo, hi;             // counted tokens of the unit past its lead, [lo, hi)
  bool whole;             // the unit is this piece
  int slot;               // of the partial otherwise
  int start, T, len;      // rows and tokens of the sequence
};

__device__ __forceinline__ int cta_of_token(long long x, long long X, int N) {
  return static_cast<int>(((x + 1) * N - 1) / X);
}

// Slot of CTA k's piece of a unit whose first piece is CTA `first`'s.
__device__ __forceinline__ int slot_of(int k, int first) { return 2 * k + (k == first ? 1 : 0); }

// What the units of a sequence cost: tile t counts base + t * step tokens, n tiles.
struct SeqCost {
  int n;
  long long base, step;
  __device__ __forceinline__ long long before(long long t) const { return t * base + step * (t * (t - 1) / 2); }
};

__device__ __forceinline__ SeqCost seq_cost(int G, int RT, int lead, int T, int len) {
  const int rows = T * G;
  SeqCost c;
  c.n = (rows + RT - 1) / RT;
  const int last = min(RT, rows) - 1;   // of the first tile
  c.base = lead + (rows ? max(0, len - T + 1 + last / G) : 0);
  c.step = (RT + G - 1) / G;
  return c;
}

// Shared-memory bytes of the prefix sums.
__host__ __device__ __forceinline__ size_t plan_bytes(int B) { return (static_cast<size_t>(B) + 1) * 12 + 4; }

// Prefix sums over the sequences: cost[b] and units[b] before sequence b.  All threads of the
// CTA call it.  Row ranges that are out of order or out of the tensors could name more rows
// than the workspace is made for, so with any of those there is no work at all.
template <int THREADS>
__device__ __forceinline__ void build_plan(const Geo& g, const Batch& bt, int RT, int lead, long long* cost,
                                           int* units, long long* tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = THREADS / 32;
  long long carry_i = 0;
  int carry_u = 0;
  bool bad = false, bad_len = false;
  for (int first = 0; first < bt.B; first += THREADS) {
    const int b = first + tid;
    long long it = 0;
    int un = 0;
    if (b < bt.B) {
      int start, T;
      if (!seq_rows(bt, b, start, T)) {
        bad = true;
        T = 0;
      }
      const SeqCost c = seq_cost(g.G, RT, lead, T, seq_len(bt, g.page_shift, b, bad_len));
      un = g.Hkv * c.n;
      it = g.Hkv * c.before(c.n);
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
      cost[b] = off_i + si - it;
      units[b] = off_u + su - un;
    }
    __syncthreads();
  }
  const bool none = __syncthreads_or(bad);
  if (tid == 0) {
    cost[bt.B] = none ? 0 : carry_i;
    units[bt.B] = none ? 0 : carry_u;
  }
  if ((bad || bad_len) && blockIdx.x == 0) raise(g.error, PNMIX_DEVERR_BATCH);
  __syncthreads();
}

// Calls fn(piece) for every piece of this CTA, in order, until it returns false.  `writer`:
// the one thread that notes the units for the merge.
template <typename F>
__device__ __forceinline__ void for_each_piece(const Geo& g, const Batch& bt, int RT, int lead,
                                               const long long* cost, const int* units, const Work& wk, int grid,
                                               bool writer, F&& fn) {
  const long long X = cost[bt.B];
  const int N = X < grid ? static_cast<int>(X) : grid, i = blockIdx.x;
  if (i == 0 && writer) *wk.count = units[bt.B];
  if (i >= N) return;
  long long x = X * i / N;
  const long long e = X * (i + 1) / N;
  int lo = 0, hi = bt.B - 1;   // the sequence that holds token x: the last b with cost[b] <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cost[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  int b = lo;
  while (x < e) {
    while (cost[b + 1] <= x) ++b;   // sequences without rows cost nothing
    bool bad = false;
    Piece p;
    p.b = b;
    seq_rows(bt, b, p.start, p.T);
    p.len = seq_len(bt, g.page_shift, b, bad);
    const SeqCost c = seq_cost(g.G, RT, lead, p.T, p.len);
    const long long head = c.before(c.n);
    p.h = static_cast<int>((x - cost[b]) / head);
    const long long hstart = cost[b] + p.h * head;
    int t0 = 0, t1 = c.n - 1;     // the last tile that starts at or before x
    while (t0 < t1) {
      const int mid = (t0 + t1 + 1) >> 1;
      if (hstart + c.before(mid) <= x) t0 = mid;
      else t1 = mid - 1;
    }
    p.tile = t0;
    const long long ustart = hstart + c.before(t0), uend = hstart + c.before(t0 + 1);
    const long long xe = uend < e ? uend : e;
    const int first = cta_of_token(ustart, X, N), last = cta_of_token(uend - 1, X, N);
    p.lo = static_cast<int>(max(x - ustart - lead, 0ll));
    p.hi = static_cast<int>(max(xe - ustart - lead, 0ll));
    p.whole = first == last;
    p.slot = slot_of(i, first);
    if (writer && x == ustart) {
      UnitInfo f;
      f.first = p.whole ? -1 : first;
      f.last = last;
      f.b = p.b;
      f.h = p.h;
      f.tile = p.tile;
      wk.info[units[b] + p.h * c.n + p.tile] = f;
    }
    if (!fn(p)) return;
    x = xe;
  }
}

constexpr int kMaxChunkCtas = 160;   // one per SM

// kv4_chunk.cu; rt 128 or 256 rows per unit.
cudaError_t launch_chunk(const Geo& g, const Batch& bt, const Rows& q, const pnmix_rows& out, const Work& wk, int rt,
                         cudaStream_t s);

}  // namespace kv4
}  // namespace pnmix
