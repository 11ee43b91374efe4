// kv4_attn.cuh -- work partition and partial results of the attention over the 4-bit paged
// cache.
//
// A UNIT is a tile of RT query rows of one (sequence b, KV head h): row r of the T * G rows is
// token j = r / G of the sequence's new tokens, query head h * G + r % G.  Its cost is counted
// in tokens: `lead` for its fixed part (at most a quarter of what a CTA gets), and an upper
// bound of what its last row sees, which grows by ceil(RT / G) from one tile to the next.
// Units are numbered b-major, then h, then tile; their tokens are numbered in that order, X in
// total, and CTA i of N takes [floor(i X / N), floor((i + 1) X / N)).  N is as many as the GPU
// holds, but while it holds more, a whole number for each unit: one for every `slice` tokens of
// a unit, up to eight for every quarter of that, and one at least.  A number that is no multiple
// of the units makes CTAs take the end of one and the beginning of the next, one after the other,
// and two dozen short parts or more cost the merge what they save.  With one CTA for every 256
// tokens of all units together, the first form: 64 tokens of 32 heads at 64 cached ones 51 instead
// of 23 us, 15 of 2 sequences at 16 75 instead of 19, 320 of 7 heads at 344 43 instead of 31, one
// at 100 21 instead of 10 us, and at 777 12.4 instead of 10.4; with one for every 32 of a unit, 22
// of 8 heads at 4698 43 instead of 27 us.  Every CTA works the numbers out from q_start and
// kv_len itself (a block-wide prefix sum), so any mix of lengths is balanced and the host
// needs to know none.  A CTA that has a unit to itself writes its rows at once.  A piece of a
// unit that does not cover it leaves a partial (m, l, O) per row, and the merge kernel joins
// them.  Only the first and the last piece of a CTA can be such, so two slots per CTA do, and
// at most one shared unit begins in a CTA, which notes it.
#pragma once

#include "decode_frag.cuh"
#include "kv4.cuh"

namespace pnmix {
namespace kv4 {

struct UnitInfo {     // of the unit that begins in a CTA and ends in `last`; last < 0: there is none
  int last;
  int start, h;             // the sequence's first row, KV head
  int row_first, rows;      // of the unit
  int pad[3];
};

struct Work {
  float* part;        // [2 N] slots, part_floats each
  UnitInfo* info;     // [N]
};

// Tokens of a unit's fixed cost, and those that a CTA is started for.
struct Grain {
  int lead, slice;
};

// A slot: (m, l) per row, then O as [D / 4][RT][4], so that a warp of rows writes it coalesced.
__host__ __device__ __forceinline__ size_t part_floats(int D, int rt) { return static_cast<size_t>(rt) * (D + 2); }
template <int D>
__device__ __forceinline__ float* part_of(float* part, int slot, int rt) {
  return part + slot * part_floats(D, rt);
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
  long long base, step;    // base without the lead
  __device__ __forceinline__ long long before(long long t) const { return t * base + step * (t * (t - 1) / 2); }
};

__device__ __forceinline__ SeqCost seq_cost(int G, int RT, int T, int len) {
  const int rows = T * G;
  SeqCost c;
  c.n = (rows + RT - 1) / RT;
  const int last = min(RT, rows) - 1;   // of the first tile
  c.base = rows ? max(0, len - T + 1 + last / G) : 0;
  c.step = (RT + G - 1) / G;
  return c;
}

// The numbers of a launch: this, then the tokens and the units before each sequence.
struct Plan {
  long long X;      // tokens in all, the leads included
  int lead, N;
  __device__ __forceinline__ const long long* tokens() const { return reinterpret_cast<const long long*>(this + 1); }
  __device__ __forceinline__ long long before(int b, int B) const {
    const int* units = reinterpret_cast<const int*>(tokens() + B + 1);
    return tokens()[b] + static_cast<long long>(units[b]) * lead;
  }
};
__host__ __device__ __forceinline__ size_t plan_bytes(int B) {
  return (sizeof(Plan) + (static_cast<size_t>(B) + 1) * 12 + 15) / 16 * 16;
}

// All threads of the CTA call it, `at` plan_bytes of its own, `tmp` shared memory, two words per
// warp.  Row ranges that are out of order or out of the tensors could name more rows
// than the workspace is made for, so with any of those there is no work at all.
template <int THREADS>
__device__ __forceinline__ const Plan& build_plan(const Geo& g, const Batch& bt, int RT, const Grain& grain, void* at,
                                                  long long* tmp) {
  Plan* plan = static_cast<Plan*>(at);
  long long* tokens = reinterpret_cast<long long*>(plan + 1);
  int* units = reinterpret_cast<int*>(tokens + bt.B + 1);
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
      const SeqCost c = seq_cost(g.G, RT, T, seq_len(bt, g.page_shift, b, bad_len));
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
      tokens[b] = off_i + si - it;
      units[b] = off_u + su - un;
    }
    __syncthreads();
  }
  const bool none = __syncthreads_or(bad);
  if (none) carry_i = carry_u = 0;
  if (tid == 0) {
    tokens[bt.B] = carry_i;
    units[bt.B] = carry_u;
    const int lead =
        static_cast<int>(min(max(carry_i / (4 * gridDim.x), 16ll), static_cast<long long>(grain.lead)));
    const long long X = carry_i + static_cast<long long>(carry_u) * lead;
    plan->lead = lead;
    plan->X = X;
    const int grid = gridDim.x;
    if (carry_u >= grid || X >= static_cast<long long>(grid + carry_u) * grain.slice) {
      plan->N = grid;
    } else if (X == 0) {
      plan->N = 0;
    } else {      // X < 2 grid slice: 32 bits do
      const int each = static_cast<int>(X) / carry_u;
      const int k = max(max(each / grain.slice, min(min(each / (grain.slice / 4), 8), grid / carry_u)), 1);
      plan->N = min(k * carry_u, grid);
    }
  }
  if ((bad || bad_len) && blockIdx.x == 0) raise(g.error, PNMIX_DEVERR_BATCH);
  __syncthreads();
  return *plan;
}

// Calls fn(piece) for every piece of this CTA, in order, until it returns false.  The piece and
// where to go on lie in shared memory (`at`, of the calling warp), so that they hold no
// registers while fn works.  A sequence's rows and length are read again for each piece.  They are
// not to change while a call runs; where they do all the same, a piece that is no longer there ends
// the walk, and none lies outside the tensors, the pages or the workspace.  SOLO: one lane calls it,
// else a whole warp.  `writer`: the one thread that notes the shared unit for the merge.
struct PieceSlot {
  Piece p;
  long long next;
};

template <bool SOLO, typename F>
__device__ __forceinline__ void for_each_piece(const Geo& g, const Batch& bt, int RT, const Plan& plan, const Work& wk,
                                               PieceSlot* at, bool writer, F&& fn) {
  if (writer) wk.info[blockIdx.x].last = -1;
  if (static_cast<int>(blockIdx.x) >= plan.N) return;
  const bool scribe = SOLO || (threadIdx.x & 31) == 0;
  if (scribe) at->next = plan.X * blockIdx.x / plan.N;
  while (true) {
    if (!SOLO) __syncwarp();
    const long long X = plan.X, x = at->next;
    const int N = plan.N, lead = plan.lead;
    const long long e = X * (blockIdx.x + 1) / N;
    if (x >= e) return;
    int lo = 0, hi = bt.B - 1;   // the sequence that holds token x: the last that starts at or before it
    while (lo < hi) {            // (and holds tokens: empty ones start where the next does)
      const int mid = (lo + hi + 1) >> 1;
      if (plan.before(mid, bt.B) <= x) lo = mid;
      else hi = mid - 1;
    }
    bool bad = false;
    Piece p;
    p.b = lo;
    if (!seq_rows(bt, lo, p.start, p.T)) return;
    p.len = seq_len(bt, g.page_shift, lo, bad);
    SeqCost c = seq_cost(g.G, RT, p.T, p.len);
    c.base += lead;
    const long long head = c.before(c.n), seq = plan.before(lo, bt.B);
    const long long h = (x - seq) / max(head, 1ll);
    if (c.n < 1 || h >= g.Hkv) return;
    p.h = static_cast<int>(h);
    const long long hstart = seq + p.h * head;
    int t0 = 0, t1 = c.n - 1;     // the last tile that starts at or before x
    while (t0 < t1) {
      const int mid = (t0 + t1 + 1) >> 1;
      if (hstart + c.before(mid) <= x) t0 = mid;
      else t1 = mid - 1;
    }
    p.tile = t0;
    const long long ustart = hstart + c.before(t0), uend = hstart + c.before(t0 + 1);
    const long long xe = uend < e ? uend : e;
    const int first = cta_of_token(ustart, X, N), last = cta_of_token(min(uend, X) - 1, X, N);
    p.lo = static_cast<int>(max(x - ustart - lead, 0ll));
    p.hi = static_cast<int>(max(xe - ustart - lead, 0ll));
    p.whole = first == last;
    p.slot = slot_of(blockIdx.x, first);
    if (writer && x == ustart && !p.whole) 
      wk.info[blockIdx.x] = {last, p.start, p.h, p.tile * RT, min(RT, p.T * g.G - p.tile * RT), {0, 0, 0}};
    if (!SOLO) __syncwarp();      // every lane has read the last piece and `next`
    if (scribe) {
      at->p = p;
      at->next = xe;
    }
    if (!SOLO) __syncwarp();
    if (!fn(at->p)) return;
  }
}

constexpr int kMaxChunkCtas = 160;   // one per SM

// kv4_chunk.cu; rt 128 or 256 rows per unit; plans: kMaxChunkCtas x plan_bytes of the
// workspace, 8-byte aligned.  *ctas: the launch's.
cudaError_t launch_chunk(const Geo& g, const Batch& bt, const Rows& q, const pnmix_rows& out, const Work& wk,
                         uint8_t* plans, int rt, int* ctas, cudaStream_t s);

}  // namespace kv4
}  // namespace pnmix
