// kv4_chunk.cu -- attention over the 4-bit paged cache for many query rows per KV head (chunks
// of new tokens, large head groups), on the 5th-generation tensor cores.
//
// What bounds it: 4 * head_dim operations per row and cached token, so the tensor cores, if
// they can be kept fed; next to them stand one exp2 per row and token (16 a cycle per SM: as
// long as both products of 128 x 128 x 128 take) and the shared-memory reads of the operands.
// So one CTA per SM holds two STREAMS whose softmax and products alternate, and everything
// around them has warps of its own (19 warps, 96 registers a thread):
//   warps 0..3, 4..7   softmax of stream 0 and 1: a thread owns a row (a TMEM lane)
//   warps 8..11        write the key tile: 128 tokens x head_dim, fp16(code * s + z)
//   warps 12..15       write the value tile: head_dim x 128 tokens, fp16(code * s + z)
//   warp 16            one thread issues the products (tcgen05.mma, accumulators in TMEM)
//   warp 17            stages the packed pages by bulk copies (8 blocks of 16 tokens a tile)
//   warp 18            works out the CTA's pieces of work, one ahead of the others
// With more than 128 rows per unit the streams are two tiles of 128 query rows, and both meet
// every key and value tile (its unpacking is then paid once per 256 rows); with up to 128 rows
// they are the same rows over the even and the odd tiles, and their sums are joined at the end.
//
//   S = Q K^T   A = query rows (fp16, scaled per row by a power of two that takes the largest
//               channel to [1, 2): bf16 channels down to 2^-17 of it are exact, smaller ones are off
//               by 2^-25 of it at most), B = key tile, both from shared memory; fp32 in TMEM
//   softmax     one pass over S in TMEM, 32 columns at a time: p = 2^(x - m), summed in fp32
//               and rounded to fp16 (2^-11 of each weight, or 2^-30 of the largest) over the S it
//               came from.  The
//               reference m moves only when a row's sum of 32 passes 65504 (so no p is above the
//               fp16 range, and no maximum has to be taken otherwise), once for these 32 at most:
//               behind it their sum is in range by construction (kv4_softmax.cuh).  What the row
//               has so far, in TMEM and out of it, is then rescaled
//   O += P V    A = P from TMEM, B = value tile
// What every role runs once per piece is kept short: straight-line code that is met cold costs
// about ten cycles an instruction here (five roles share the instruction cache), and a spilled
// register costs an access to L2 (the shared memory takes the whole of L1).
//
// The operands lie in shared memory in the K-major form without swizzle: 8-row pieces of 8 x 16
// bytes.  The order of the channels inside K (keys and queries alike) and of the value rows is
// free; it is chosen so that code words unpack without moving codes between lanes and 16-byte
// stores of neighbouring lanes lie side by side.
//
// Measured: 2 x 1024 tokens of 32 query and 8 KV heads (head_dim 128) over 8192 cached ones, the
// merge included, 318 to 327 us by graph replay or 800 TFLOP/s, half of what a library product of
// 8192^3 reaches here (floor 156 us).  At 1 x 1024 the kernel takes 187 us under the profiler with 38 %
// of the tensor and of the exp2 pipe busy, the warps waiting for TMEM loads: a stream's tile is a
// chain of products, their commit, four rounds of load, exp2 and store, and the next products.  TMEM
// is full with two such chains as they stand (the half of a stream's logits that its weights do not
// lie over stays idle meanwhile).  Tried and slower: sixteen softmax warps (324 us then, against 308), value
// products by half tiles (373), 16- or 64-column loads and their double buffering, register
// shares by role (setmaxnreg), a quarter or half of the exp2 as polynomials.
#include <float.h>

#include <atomic>

#include "kv4_attn.cuh"
#include "kv4_launch.cuh"
#include "kv4_softmax.cuh"

namespace pnmix {
namespace kv4 {
namespace {

constexpr int kThreads = 608;
constexpr int kTile = 128;                  // tokens of a key / value tile; rows of a stream
constexpr uint32_t kCommitLimit = 1u << 22; // try_wait rounds of a wait inside the CTA
constexpr float kTop = 65504.f;             // largest sum of 32 weights before the reference moves: none is past fp16
constexpr int kTmemO = 256;                 // TMEM columns: S (and P) of stream s at 128 s, O at 256 + 128 s

// ---- tcgen05

__device__ __forceinline__ int tile_off(int rows, int r, int k) {
  return (k >> 4) * rows * 32 + (r >> 3) * 256 + ((k >> 3) & 1) * 128 + (r & 7) * 16 + (k & 7) * 2;
}
// Descriptor of one K = 16 step: no swizzle, the two 8-element halves of K 128 bytes apart,
// 8-row groups 256 bytes apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t step_base) {
  return static_cast<uint64_t>((step_base >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128u >> 4) << 16) |
         (static_cast<uint64_t>(256u >> 4) << 32) | (1ull << 46);
}
// fp16 A and B, fp32 D, both K-major, M = 128, N = n.
__host__ __device__ constexpr uint32_t mma_idesc(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Consecutive columns of this thread's TMEM lane (warp-collective).
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}

// 32 columns without the wait, and the wait that the registers depend on.
__device__ __forceinline__ void tmem_ld32_start(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// (a0, a1) * b + c, and (a0, a1) + (b0, b1), two fp32 lanes per instruction.
__device__ __forceinline__ float2 fma2(float a0, float a1, float b, float c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %5};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float b0, float b1) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b0), "f"(b1));
  return d;
}

__device__ __forceinline__ __half2 as_h2(uint32_t x) {
  __half2 h;
  memcpy(&h, &x, 4);
  return h;
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) {
  uint32_t x;
  memcpy(&x, &h, 4);
  return x;
}

// Codes at nibbles 0 / 4 (in_high false) or 1 / 5 of w as an exact fp16 pair: 1024 + c has c in
// its low mantissa bits, 1024 + 16 c has it four bits up.
__device__ __forceinline__ __half2 codes_low(uint32_t w) {
  return __hsub2(as_h2((w & 0x000F000Fu) | 0x64006400u), __float2half2_rn(1024.f));
}
__device__ __forceinline__ __half2 codes_high(uint32_t w) {
  return __hfma2(as_h2((w & 0x00F000F0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-64.f));
}

struct ChunkArgs {
  Geo g;
  Batch bt;
  Rows q;
  uint16_t* out;
  long long out_ts, out_hs;
  Work wk;
  Grain grain;
  uint8_t* plans;   // plan_bytes for each CTA: shared memory has no room
  int rt;           // 256 (two row tiles) or 128 (one, even and odd tiles apart)
};

// Shared memory.  The pages pass through the ring in halves of a tile (4 blocks); the one-tile
// form has one query tile less and a ring of six halves instead of three (there a key tile is
// wanted two tiles ahead).
template <int D>
struct Smem {
  static constexpr int kTileBytes = 128 * D * 2;            // any operand tile
  static constexpr int kK = 0;                              // 2 x [128 tokens][D]
  static constexpr int kV = kK + 2 * kTileBytes;            // 2 x [D channels][128 tokens]
  static constexpr int kQ = kV + 2 * kTileBytes;            // [128 rows][D], two in the two-tile form
  static constexpr int kHalfBytes = 4 * 20 * D;             // 4 blocks
  static constexpr int kMl = 0;                             // after the ring: [128][2], stream 1's m, l
  static constexpr int kBase = kMl + 128 * 8;               // [2][128] base of a stream's row (kv4_softmax.cuh)
  static constexpr int kBars = kBase + 2 * 128 * 4;
  static constexpr int kJobs = kBars + 384;                 // two pieces of work
  static constexpr int kSlots = kJobs + 96;                 // the partition's place in its work
  static constexpr int kEnd = kSlots + 64;
  __host__ __device__ static constexpr int ring(bool dual) { return kQ + (dual ? 2 : 1) * kTileBytes; }
  __host__ __device__ static constexpr int stages(bool dual) { return dual ? 3 : 6; }
  __host__ __device__ static constexpr int rest(bool dual) { return ring(dual) + stages(dual) * kHalfBytes; }
};

// Position in the ring: stage and the phase of its barriers.
struct RingPos {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++stage == stages) {
      stage = 0;
      ++phase;
    }
  }
};

// A piece of work as the roles take it; two are on the way at once.
struct Job {
  int b, h, start;          // sequence, KV head, the sequence's first row
  int row_first, rows;      // of the unit
  int base_seen;            // tokens that the sequence's row 0 sees
  int most;                 // tokens that the last row sees
  int lo, n;                // first tile, tiles; n < 0: no more work
  int slot;                 // of the partial, -1 if the unit is this piece
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const __grid_constant__ ChunkArgs a) {
  using S = Smem<D>;
  constexpr int NG = D / 32, BB = 20 * D;
  extern __shared__ __align__(1024) uint8_t smem[];
  const Geo& g = a.g;
  const Batch& bt = a.bt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool dual = a.rt == 256;
  uint8_t* rest = smem + S::rest(dual);
  uint8_t* const ring0 = smem + S::ring(dual);
  const uint32_t stages = S::stages(dual);
  uint64_t* bars = reinterpret_cast<uint64_t*>(rest + S::kBars);
  uint64_t* ring_full = bars + 26;   // [6] the staged blocks are in
  uint64_t* ring_empty = bars + 32;  // [6] both builders are done with them (8 warps)
  uint64_t* k_full = bars;           // [2] key tile written (4 warps, two halves)
  uint64_t* k_empty = bars + 2;      // [2] its products are done
  uint64_t* v_full = bars + 4;       // [2] value tile written
  uint64_t* v_empty = bars + 6;      // [2]
  uint64_t* s_full = bars + 12;      // [2] logits of the stream are in TMEM
  uint64_t* p_full = bars + 14;      // [2] its weights are (4 warps)
  uint64_t* o_done = bars + 16;      // [2] its value products of this piece are done
  uint64_t* q_full = bars + 38;      // [2] the stream's query tile is written (4 warps)
  uint64_t* job_full = bars + 19;    // [2]
  uint64_t* job_empty = bars + 21;   // [2] every role is done with it (16 warps and two more)
  uint64_t* drained = bars + 23;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int* fail = reinterpret_cast<volatile int*>(bars + 25);
  Job* jobs = reinterpret_cast<Job*>(rest + S::kJobs);
  if (tid == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(ring_full + i, 1);
      mbar_init(ring_empty + i, 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 8);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 8);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(q_full + i, 4);
      mbar_init(o_done + i, 1);
      mbar_init(job_full + i, 1);
      mbar_init(job_empty + i, 18);
    }
    mbar_init(drained, 1);
    *fail = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;");
  tc_fence_before();
  const Plan& plan =
      build_plan<kThreads>(g, bt, a.rt, a.grain, a.plans + blockIdx.x * plan_bytes(bt.B),
                           reinterpret_cast<long long*>(rest + S::kMl));
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  // Bounded wait for phase `n` (counted from 0) of a barrier; false once anything in the CTA
  // gave up.  wait() is called by a whole warp and answers all of it alike.  (The lanes vote in
  // every round: at 2 x 1024 tokens of 32 heads over 8192 cached ones a vote behind each lane's own
  // loop took 347 us instead of 320, and one lane waiting for the others 550.)
  auto wait_one = [&](uint64_t* bar, uint32_t n, uint32_t limit) -> bool {
    uint32_t spins = 0;
    while (!mbar_try_wait(bar, n & 1u)) {
      if (*fail) return false;
      if (++spins >= limit) {
        *fail = 1;
        raise(g.error, PNMIX_DEVERR_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  auto wait = [&](uint64_t* bar, uint32_t n, uint32_t limit) -> bool {
    for (uint32_t spins = 0; !__all_sync(0xffffffffu, mbar_try_wait(bar, n & 1u)); ++spins) {
      if (__any_sync(0xffffffffu, *fail != 0)) return false;
      if (spins >= limit) {
        *fail = 1;
        raise(g.error, PNMIX_DEVERR_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  // The builders and the staging take job after job this way.
  auto for_each_job = [&](auto&& fn) {
    for (uint32_t i = 0;; ++i) {
      if (!wait(job_full + (i & 1u), i >> 1, kCommitLimit)) return;
      const Job& jb = jobs[i & 1u];
      if (jb.n < 0 || !fn(jb)) return;
      __syncwarp();
      if (lane == 0) mbar_arrive(job_empty + (i & 1u));
    }
  };

  if (warp < 8) {
    // ================================================================ softmax
    const int stream = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * stream, t_o = tmem + lanes + kTmemO + 128 * stream;
    float* ml = reinterpret_cast<float*>(rest + S::kMl) + 2 * row;
    uint8_t* qa = smem + S::kQ + (dual ? stream * S::kTileBytes : 0);
    uint32_t ns = 0, no = 0;   // logit tiles taken; pieces whose value products were waited for
    // whether any thread says so, of the stream (two-tile form) or of both
    auto either = [&](bool x) -> bool {
      uint32_t any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
          : "=r"(any)
          : "r"(static_cast<uint32_t>(x)), "r"(dual ? 2 + stream : 1), "r"(dual ? 128 : 256)
          : "memory");
      return any != 0;
    };
    bool ok = true;
    for (uint32_t job = 0;; ++job) {
      ok = ok && wait(job_full + (job & 1u), job >> 1, kCommitLimit);
      // In the one-tile form both streams are done with the last piece here (its query tile, O and
      // ml) and go on or stop alike; else a stream's warps are, with its query tile.
      if (either(!ok)) break;
      const Job& jb = jobs[job & 1u];
      const int nt = jb.n;
      if (nt < 0) break;
      const int v = (dual ? 128 * stream : 0) + row;     // row of the unit
      const bool live = v < jb.rows;
      // this thread's row: its token and head in a [tokens][heads][D] tensor
      const int r = jb.row_first + v, j = r / g.G;
      const int tok = live ? jb.start + j : -1, head = jb.h * g.G + r - j * g.G;
      const int seen = live ? jb.base_seen + j : 0;
      float fac = 0.f;
      if (dual || stream == 0) {
        // ---- the query rows -> A.  A warp takes its 32 rows eight at a time, four 16-byte pieces of
        // each per instruction, so eight lanes' stores fill neighbouring 16-byte places.  The rows
        // are copied as they are and scaled in place.
        const int sub = lane & 7, part = lane >> 3;
#pragma unroll 1
        for (int ra = 0; ra < 4; ++ra) {
          const int rtok = __shfl_sync(0xffffffffu, tok, 8 * ra + sub), rhead = __shfl_sync(0xffffffffu, head, 8 * ra + sub);
          const uint16_t* src = a.q.p + rtok * a.q.ts + rhead * a.q.hs + 8 * part;
          uint8_t* dst = qa + tile_off(128, 32 * (warp & 3) + 8 * ra + sub, 8 * part);
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            if (rtok >= 0)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + c * (2 * 128 * 32))),
                           "l"(src + 32 * c)
                           : "memory");
            else
              *reinterpret_cast<uint4*>(dst + c * (2 * 128 * 32)) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
        for (int ra = 0; ra < 4; ++ra) {
          uint8_t* at = qa + tile_off(128, 32 * (warp & 3) + 8 * ra + sub, 8 * part);
          uint32_t w[NG][4];
          float top = 0.f;
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(at + c * (2 * 128 * 32));
            w[c][0] = x.x; w[c][1] = x.y; w[c][2] = x.z; w[c][3] = x.w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[c][i] << 16)), fabsf(__uint_as_float(w[c][i] & 0xFFFF0000u))));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
          const int up = top > 0.f ? min(max(-ex, -90), 120) : 0;      // largest channel to [1, 2)
          const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[2 * i] = __uint_as_float(w[c][i] << 16) * mul;
              f[2 * i + 1] = __uint_as_float(w[c][i] & 0xFFFF0000u) * mul;
            }
            // position order inside 8 channels: 0, 4, 1, 5, 2, 6, 3, 7, as a code word unpacks
            *reinterpret_cast<uint4*>(at + c * (2 * 128 * 32)) = make_uint4(
                pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]), pack_f16x2(f[3], f[7]));
          }
          // the row's owner takes its factor
          // (not 0: a hidden column's -inf times it has to stay -inf)
          const float mine = fmaxf(g.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), FLT_MIN);
          const float got = __shfl_sync(0xffffffffu, mine, lane & 7);
          if (part == ra) fac = got;
        }
        if (!dual) ml[0] = fac;
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + stream);
      if (!dual) {          // stream 1 has the same rows
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (stream == 1) fac = ml[0];
      }

      float ref = kFirstReference, den = 0.f;
      bool far = false;                 // a row of the warp has a base other than 0
      float* const base = reinterpret_cast<float*>(rest + S::kBase) + tid;      // out of the registers
      *base = 0.f;
      int mine = 0;                     // tiles of this stream so far
      int lim = seen - (jb.lo + (dual ? 0 : stream)) * kTile;     // columns of the tile below it are visible
      for (int i = dual ? 0 : stream; i < nt; i += dual ? 1 : 2, lim -= dual ? kTile : 2 * kTile) {
        if (!(ok = wait(s_full + stream, ns, kCommitLimit))) break;
        ++ns;
        tc_fence_after();
        const bool edge = __any_sync(0xffffffffu, lim < kTile);
        // Weights of 32 columns from their logits (bits in, fp16 pairs out); their sum.
        auto weights = [&](int col, uint32_t (&x)[32], uint32_t* p) {
          if (edge) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (col + k >= lim) x[k] = 0xFF800000u;     // -inf
          }
          const float off = -ref;
          float2 d0 = make_float2(0.f, 0.f), d1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float2 e0 = fma2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]), fac, off);
            const float2 e1 = fma2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]), fac, off);
            const float p0 = ex2(e0.x), p1 = ex2(e0.y), p2 = ex2(e1.x), p3 = ex2(e1.y);
            d0 = add2(d0, p0, p1);
            d1 = add2(d1, p2, p3);
            p[k / 2] = pack_f16x2(p0, p1);
            p[k / 2 + 1] = pack_f16x2(p2, p3);
          }
          d0 = add2(d0, d1.x, d1.y);
          return d0.x + d0.y;
        };
        for (int c = 0; c < 4;) {
          float sum = 0.f;
          // The weights of 32 columns stay in registers until their sum is found to be in range, so
          // their logits can still be read again.
          if (!far) {
#pragma unroll 1
            for (; c < 4; ++c) {
              uint32_t cur[32], p[16];
              tmem_ld32_start(t_s + 32 * c, cur);
              tmem_ld_wait(cur);
              sum = weights(32 * c, cur, p);
              if (__any_sync(0xffffffffu, sum > kTop)) break;
              den += sum;
              tmem_st16(t_s + 16 * c, p);     // over columns that were read
            }
            if (c == 4) break;
          }
          // Out of range, or rows with a base: 32 columns with a move of the reference, one at most (the
          // commit of these logits covers the stream's earlier value products, so O is idle).
          uint32_t cur[32], p[16];
          for (bool known = !far, moved = false;; known = false, moved = true) {
            if (!known) {
              tmem_ld32_start(t_s + 32 * c, cur);
              tmem_ld_wait(cur);
              const float b = *base;
#pragma unroll
              for (int k = 0; k < 32; ++k) cur[k] = __float_as_uint(__uint_as_float(cur[k]) - b);
              sum = weights(32 * c, cur, p);
              if (moved || !__any_sync(0xffffffffu, sum > kTop)) break;
            }
            uint32_t y[16];
            float mx = -INFINITY;
#pragma unroll 1
            for (int k = 32 * c; k < kTile; k += 16) {      // the rest of the tile
              tmem_ld16(t_s + k, y);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (k + e < lim) mx = fmaxf(mx, __uint_as_float(y[e]));
            }
            float f = 1.f;
            if (sum > kTop) {      // some weight is 2^10 and more
              const RowRef from = {*base, ref}, to = move_reference(from, mx, fac);
              f = ex2(move_exponent(from, to, fac));
              *base = to.base;
              ref = to.ref;
              den *= f;
            }
            far = __any_sync(0xffffffffu, *base != 0.f);
            if (mine > 0) {
#pragma unroll 1
              for (int k = 0; k < D; k += 16) {
                tmem_ld16(t_o + k, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                tmem_st16(t_o + k, y);
              }
            }
            tmem_wait_st();
#pragma unroll 1
            for (int k = 0; k < 16 * c; k += 16) {     // this tile's weights that are written already
              tmem_ld16(t_s + k, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 w = __half22float2(as_h2(y[e]));
                y[e] = pack_f16x2(w.x * f, w.y * f);
              }
              tmem_st16(t_s + k, y);
            }
          }
          den += sum;
          tmem_st16(t_s + 16 * c, p);
          ++c;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + stream);
        ++mine;
      }
      // ---- the stream's last product
      if (ok && mine > 0) ok = wait(o_done + stream, no++, kCommitLimit);
      tc_fence_after();
      float w0 = 1.f, w1 = 0.f, top = reference_of({*base, ref}, fac);
      if (!dual) {        // join the streams: stream 0's threads read both rows of O
        if (stream == 1) {
          ml[0] = top;
          ml[1] = den;
        }
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tc_fence_after();
        if (stream == 0) {
          const float m1 = ml[0], l1 = ml[1];
          const float m = l1 == 0.f ? top : den == 0.f ? m1 : fmaxf(top, m1);
          w0 = den == 0.f ? 0.f : ex2(top - m);
          w1 = l1 == 0.f ? 0.f : ex2(m1 - m);
          den = (den == 0.f ? 0.f : den * w0) + (l1 == 0.f ? 0.f : l1 * w1);
          top = m;
        }
      }
      if (dual || stream == 0) {
        const int slot = jb.slot;
        const bool has0 = mine > 0, has1 = !dual && nt > 1;
        const float inv = den == 0.f ? 0.f : 1.f / den;
        float* part = part_of<D>(a.wk.part, slot, a.rt);
        if (slot >= 0 && live) reinterpret_cast<float2*>(part)[v] = make_float2(top, den);
        // the stream's logits are done, so its query tile is free to turn the rows around in
        uint8_t* turn = qa + (warp & 3) * (64 * D);
#pragma unroll 1
        for (int c = 0; c < NG; ++c) {
          uint32_t o[32];
          if (has0) {
            tmem_ld32_start(t_o + 32 * c, o);
            tmem_ld_wait(o);
          }
          if (!has0 || w0 != 1.f) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = !has0 || w0 == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k]) * w0);
          }
          if (has1) {
            uint32_t o1[32];
            tmem_ld32_start(t_o + 128 + 32 * c, o1);
            tmem_ld_wait(o1);
            if (w1 != 0.f) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                o[k] = __float_as_uint(fmaf(__uint_as_float(o1[k]), w1, __uint_as_float(o[k])));
            }
          }
          // column 8 i + w of a group is channel 4 w + i
          if (slot < 0) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {      // channels 8 h .. 8 h + 7: w = 2 h, 2 h + 1
              uint32_t wd[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int w = 2 * h + (k >> 1), i = 2 * (k & 1);
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[8 * i + w]) * inv,
                                                                __uint_as_float(o[8 * (i + 1) + w]) * inv);
                memcpy(&wd[k], &b2, 4);
              }
              *reinterpret_cast<uint4*>(turn + lane * (2 * D) + (((4 * c + h) ^ (lane & 7)) * 16)) =
                  make_uint4(wd[0], wd[1], wd[2], wd[3]);
            }
          } else if (live) {
#pragma unroll
            for (int w = 0; w < 8; ++w)
              reinterpret_cast<uint4*>(part + 2 * a.rt)[(8 * c + w) * a.rt + v] =
                  make_uint4(o[w], o[8 + w], o[16 + w], o[24 + w]);
          }
        }
        if (slot < 0) {
          __syncwarp();
          constexpr int kPer = 32 / (D / 8);     // rows a warp writes at once
          const int piece = lane & (D / 8 - 1);
#pragma unroll 1
          for (int x = lane / (D / 8); x < 32; x += kPer) {
            const int rtok = __shfl_sync(0xffffffffu, tok, x), rhead = __shfl_sync(0xffffffffu, head, x);
            const uint4 w = *reinterpret_cast<const uint4*>(turn + x * (2 * D) + ((piece ^ (x & 7)) * 16));
            if (rtok >= 0)
              *(reinterpret_cast<uint4*>(a.out + rtok * a.out_ts + rhead * a.out_hs) + piece) = w;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(job_empty + (job & 1u));
    }
  } else if (warp < 12) {
    // ================================================================ key tiles
    const int t = tid & 63, pieces = ((tid >> 6) & 1) * 2;      // token of the half, two of its row's pieces
    const int blk = t >> 4, r = t & 15;
    uint32_t nr = 0;                            // halves so far
    RingPos rp;
    for_each_job([&](const Job& jb) -> bool {
      const int n = 2 * jb.n;
      int left = jb.most - jb.lo * kTile;       // tokens from the half's first on
      __syncwarp();
      for (int i = 0; i < n; ++i, ++nr, left -= kTile / 2) {
        const uint32_t buf = (nr >> 1) & 1u;
        if (!wait(ring_full + rp.stage, rp.phase, g.wait_limit)) return false;
        if (nr >= 4 && !(nr & 1u) && !wait(k_empty + buf, (nr >> 2) - 1, kCommitLimit)) return false;
        const uint8_t* src = ring0 + rp.stage * S::kHalfBytes + blk * BB;
        uint8_t* dst = smem + S::kK + buf * S::kTileBytes + tile_off(kTile, 64 * (nr & 1u) + t, 0);
        const bool there = t < left;            // behind: whatever the page holds
        uint32_t sz[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k)
          sz[k] = there ? *reinterpret_cast<const uint32_t*>(src + 8 * D + r * (4 * NG) + 4 * k) : 0u;
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) {
          const int piece = (pieces + pp) ^ ((t >> 1) & 3);     // eight lanes' pieces lie in different banks
          uint32_t w[NG];
          const uint8_t* at = src + r * (D / 2) + piece * (4 * NG);
          if constexpr (NG == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(at);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            w[0] = x.x; w[1] = x.y;
          }
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            const __half2 s = as_h2(__byte_perm(sz[k], 0u, 0x1010)), z = as_h2(__byte_perm(sz[k], 0u, 0x3232));
            const uint32_t w8 = w[k] >> 8;
            const uint32_t x0 = as_u32(__hfma2(codes_low(w[k]), s, z)), x1 = as_u32(__hfma2(codes_high(w[k]), s, z));
            const uint32_t x2 = as_u32(__hfma2(codes_low(w8), s, z)), x3 = as_u32(__hfma2(codes_high(w8), s, z));
            *reinterpret_cast<uint4*>(dst + (2 * k + (piece >> 1)) * (kTile * 32) + (piece & 1) * 128) =
                make_uint4(x0, x1, x2, x3);
          }
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(k_full + buf);
          mbar_arrive(ring_empty + rp.stage);
        }
        rp.next(stages);
      }
      return true;
    });
  } else if (warp < 16) {
    // ================================================================ value tiles
    const int bw = warp - 12;
    const int w = lane & 7, half = (lane >> 3) & 1, odd = lane >> 4;   // piece, pair of groups, octet parity
    uint32_t nr = 0;
    RingPos rp;
    for_each_job([&](const Job& jb) -> bool {
      const int n = 2 * jb.n;
      int left = jb.most - jb.lo * kTile;
      __syncwarp();
      for (int i = 0; i < n; ++i, ++nr, left -= kTile / 2) {
        const uint32_t buf = (nr >> 1) & 1u;
        if (!wait(ring_full + rp.stage, rp.phase, g.wait_limit)) return false;
        if (nr >= 4 && !(nr & 1u) && !wait(v_empty + buf, (nr >> 2) - 1, kCommitLimit)) return false;
        // an item: 8 tokens (octet of the half), piece w, one pair of groups.  With D = 64 there is
        // one pair: half of the lanes have nothing to do.
        constexpr bool kAll = NG == 4;
        const int octet = 2 * bw + odd, pair = kAll ? half : 0;
        if (kAll || half == 0) {
          const uint8_t* blk = ring0 + rp.stage * S::kHalfBytes + 10 * D + (octet >> 1) * BB;
          uint8_t* dst = smem + S::kV + buf * S::kTileBytes + (4 * (nr & 1u) + (octet >> 1)) * (D * 32) +
                         (octet & 1) * 128 + w * 16;
          uint32_t cw[8], sz[8][2];
          // lanes of odd octets take each token pair the other way round: the two octets of a warp
          // then read rows of different parity
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int t = (octet & 1) * 8 + (k ^ odd);
            cw[k] = *reinterpret_cast<const uint32_t*>(blk + t * (D / 2) + value_place<D>(t, w) * (2 * NG) + 4 * pair);
            const uint2 x = *reinterpret_cast<const uint2*>(blk + 8 * D + t * (4 * NG) + 8 * pair);
            const bool there = 8 * octet + (k ^ odd) < left;
            sz[k][0] = there ? x.x : 0u;
            sz[k][1] = there ? x.y : 0u;
          }
          const uint32_t lo_sel = odd ? 0x1054u : 0x5410u, hi_sel = odd ? 0x3276u : 0x7632u;
#pragma unroll
          for (int gp = 0; gp < 2; ++gp) {        // group 2 * pair + gp
            uint32_t x[4][4];                     // [channel 4 w + i][token pair]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t c2 = __byte_perm(cw[2 * k], cw[2 * k + 1], gp ? hi_sel : lo_sel);
              const __half2 s = as_h2(__byte_perm(sz[2 * k][gp], sz[2 * k + 1][gp], lo_sel));
              const __half2 z = as_h2(__byte_perm(sz[2 * k][gp], sz[2 * k + 1][gp], hi_sel));
              const uint32_t c8 = c2 >> 8;
              x[0][k] = as_u32(__hfma2(codes_low(c2), s, z));
              x[1][k] = as_u32(__hfma2(codes_high(c2), s, z));
              x[2][k] = as_u32(__hfma2(codes_low(c8), s, z));
              x[3][k] = as_u32(__hfma2(codes_high(c8), s, z));
            }
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)        // value row (4 group + ch) * 8 + w
              *reinterpret_cast<uint4*>(dst + (4 * (2 * pair + gp) + ch) * 256) =
                  make_uint4(x[ch][0], x[ch][1], x[ch][2], x[ch][3]);
          }
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v_full + buf);
          mbar_arrive(ring_empty + rp.stage);
        }
        rp.next(stages);
      }
      return true;
    });
  } else {
    if (warp == 16 && lane == 0) {
      // ============================================================== products
      const uint32_t q0 = smem_u32(smem + S::kQ), k0 = smem_u32(smem + S::kK), v0 = smem_u32(smem + S::kV);
      constexpr uint32_t kIdescS = mma_idesc(kTile), kIdescO = mma_idesc(D);
      uint32_t nk = 0, nv = 0, nq = 0, np0 = 0, np1 = 0;   // tiles, query tiles, weights of either stream taken
      auto logits = [&](int stream, uint32_t buf) {
        const uint64_t qd = tile_desc(q0 + (dual ? stream * S::kTileBytes : 0)), kd = tile_desc(k0 + buf * S::kTileBytes);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_ss(tmem + 128 * stream, qd + s * (128 * 32 >> 4), kd + s * (kTile * 32 >> 4), kIdescS, s > 0);
        tc_commit(s_full + stream);
      };
      auto values = [&](int stream, uint32_t buf, bool accumulate, bool last) {
        const uint64_t vd = tile_desc(v0 + buf * S::kTileBytes);
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
          mma_ts(tmem + kTmemO + 128 * stream, tmem + 128 * stream + 8 * s, vd + s * (D * 32 >> 4), kIdescO,
                 accumulate || s > 0);
        if (last) tc_commit(o_done + stream);
      };
      auto products = [&](const Job& jb) -> bool {
        const int n = jb.n, ahead = dual ? 1 : 2;
        // (in the one-tile form the second stream reads the first one's tile)
        if (!wait_one(q_full, nq, kCommitLimit)) return false;
        // the next key tile, once written
        auto key_tile = [&]() -> bool {
          if (!wait_one(k_full + (nk & 1u), nk >> 1, kCommitLimit)) return false;
          tc_fence_after();
          return true;
        };
        for (int i = 0; i < ahead && i < n; ++i) {
          if (!key_tile()) return false;
          logits(dual ? 0 : i, nk & 1u);
          if (dual) {
            if (!wait_one(q_full + 1, nq, kCommitLimit)) return false;
            logits(1, nk & 1u);
          }
          tc_commit(k_empty + (nk & 1u));
          ++nk;
        }
        if (dual && n == 0 && !wait_one(q_full + 1, nq, kCommitLimit)) return false;     // no phase is skipped
        ++nq;
        for (int i = 0; i < n; ++i) {
          for (int x = 0; x < (dual ? 2 : 1); ++x) {
            const int stream = dual ? x : i & 1;
            if (x == 0 && !wait_one(v_full + (nv & 1u), nv >> 1, kCommitLimit)) return false;
            if (!wait_one(p_full + stream, stream ? np1 : np0, kCommitLimit)) return false;
            if (stream) ++np1;
            else ++np0;
            tc_fence_after();
            values(stream, nv & 1u, i >= ahead, i + ahead >= n);
            if (x == (dual ? 1 : 0)) tc_commit(v_empty + (nv++ & 1u));
            if (i + ahead < n) {
              if (x == 0 && !key_tile()) return false;
              logits(stream, nk & 1u);
              if (x == (dual ? 1 : 0)) {
                tc_commit(k_empty + (nk & 1u));
                ++nk;
              }
            }
          }
        }
        return true;
      };
      for (uint32_t i = 0; wait_one(job_full + (i & 1u), i >> 1, kCommitLimit); ++i) {
        const Job& jb = jobs[i & 1u];
        if (jb.n < 0 || !products(jb)) break;
        mbar_arrive(job_empty + (i & 1u));
      }
    }
    if (warp == 17) {
      // ============================================================== staging
      uint32_t nr = 0;
      RingPos rp;
      const size_t head_bytes = static_cast<size_t>(1 << (g.page_shift - 4)) * BB, page_bytes = head_bytes * g.Hkv;
      const int per_copy = min(g.page_shift, 6);       // log2 tokens of a copy: 16 to 64 of a page
      const int copies = (kTile / 2) >> per_copy;
      for_each_job([&](const Job& jb) -> bool {
        const int n = 2 * jb.n, first = jb.lo * kTile, most = jb.most;
        const int32_t* table = bt.table + static_cast<size_t>(jb.b) * bt.max_pages;
        const uint8_t* base = g.pages + static_cast<size_t>(jb.h) * head_bytes;
        __syncwarp();
        auto page_of = [&](int i) {        // of this lane's copy of half i
          const int tok = first + i * (kTile / 2) + (lane << per_copy);
          if (lane >= copies || i >= n || tok >= most) return 0;
          const int id = __ldg(table + (tok >> g.page_shift));
          if (id >= 0 && id < g.n_pages) return id;
          raise(g.error, PNMIX_DEVERR_PAGE);
          return 0;
        };
        if (jb.b == g.skip_seq) return false;      // the test hook: what waits for these pages gives up
        int id = page_of(0);
        for (int i = 0; i < n; ++i, ++nr) {
          if (nr >= stages && !wait(ring_empty + rp.stage, rp.phase - 1, kCommitLimit)) return false;
          const int tok = first + i * (kTile / 2) + (lane << per_copy);
          // blocks of the half (the second half of a last tile may have none) and of this lane's copy
          const int blocks = max(0, min(4, (most - first - i * (kTile / 2) + 15) >> 4));
          const int mine = min(1 << (per_copy - 4), blocks - (lane << (per_copy - 4)));
          if (lane == 0) {
            proxy_fence();
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(ring_full + rp.stage)),
                         "r"(blocks * BB)
                         : "memory");
          }
          __syncwarp();
          if (lane < copies && mine > 0)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(ring0 + rp.stage * S::kHalfBytes) + (lane << (per_copy - 4)) * BB),
                         "l"(base + id * page_bytes + static_cast<size_t>((tok & ((1 << g.page_shift) - 1)) >> 4) * BB),
                         "r"(mine * BB), "r"(smem_u32(ring_full + rp.stage))
                         : "memory");
          id = page_of(i + 1);
          rp.next(stages);
        }
        return true;
      });
      // every staged copy lands before the CTA's shared memory is given up
      for (uint32_t k = 0; k < stages && k < nr; ++k) {
        const uint32_t last = (nr - 1 - k) / stages;      // phase of the stage's last use
        uint64_t* bar = ring_full + (nr - 1 - k) % stages;
        for (uint32_t spins = 0; spins < kCommitLimit && !mbar_try_wait(bar, last & 1u); ++spins) {
        }
      }
    }
    if (warp == 18 && lane == 0) {
      // ============================================================== the pieces of work
      uint32_t i = 0;
      auto give = [&](const Job& jb) -> bool {
        if (i >= 2 && !wait_one(job_empty + (i & 1u), (i >> 1) - 1, kCommitLimit)) return false;
        jobs[i & 1u] = jb;
        mbar_arrive(job_full + (i & 1u));
        ++i;
        return true;
      };
      bool more = true;
      for_each_piece<true>(g, bt, a.rt, plan, a.wk, reinterpret_cast<PieceSlot*>(rest + S::kSlots), true,
                           [&](const Piece& pc) -> bool {
        Job jb;
        jb.b = pc.b;
        jb.h = pc.h;
        jb.start = pc.start;
        jb.row_first = pc.tile * a.rt;
        jb.rows = min(a.rt, pc.T * g.G - jb.row_first);
        jb.base_seen = pc.len - pc.T + 1;
        jb.most = max(0, jb.base_seen + (jb.row_first + jb.rows - 1) / g.G);
        const int nt = (jb.most + kTile - 1) / kTile;
        jb.lo = min((pc.lo + kTile - 1) / kTile, nt);                        // the tiles that start in [lo, hi)
        jb.n = min((pc.hi + kTile - 1) / kTile, nt) - jb.lo;
        jb.slot = pc.whole ? -1 : pc.slot;
        return more = give(jb);
      });
      Job end{};
      end.n = -1;
      if (more) give(end);
    }
    __syncwarp();
  }
  __syncthreads();
  // After a stop products may still run: they are done before TMEM and the tiles are given up.
  if (*fail && warp == 16 && lane == 0) {
    tc_commit(drained);
    for (uint32_t spins = 0; spins < kCommitLimit && !mbar_try_wait(drained, 0u); ++spins) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

}  // namespace

constexpr int kMaxDevices = 64;

template <int D>
static cudaError_t launch_chunk_d(const ChunkArgs& a, int* ctas, cudaStream_t s) {
  static std::atomic<int> cache[kMaxDevices];
  const size_t smem = Smem<D>::rest(a.rt == 256) + Smem<D>::kEnd;
  auto kern = chunk_kernel<D>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (known) sms = cache[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  Smem<D>::rest(true) + Smem<D>::kEnd)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return e;
    if (known) cache[dev].store(sms, std::memory_order_relaxed);
  }
  *ctas = sms < kMaxChunkCtas ? sms : kMaxChunkCtas;
  kern<<<*ctas, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_chunk(const Geo& g, const Batch& bt, const Rows& q, const pnmix_rows& out, const Work& wk, uint8_t* plans,
                         int rt, int* ctas, cudaStream_t s) {
  ChunkArgs a{};
  a.g = g;
  a.bt = bt;
  a.q = q;
  a.out = out.data;
  a.out_ts = out.token_stride;
  a.out_hs = out.head_stride;
  a.wk = wk;
  a.grain = {256, 128};
  a.plans = plans;
  a.rt = rt;
  return g.D == 64 ? launch_chunk_d<64>(a, ctas, s) : launch_chunk_d<128>(a, ctas, s);
}

}  // namespace kv4
}  // namespace pnmix
