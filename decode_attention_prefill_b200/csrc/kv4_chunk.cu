// kv4_chunk.cu -- attention over the 4-bit paged cache for many query rows per KV head (chunks
// of new tokens, large head groups), on the 5th-generation tensor cores.
//
// What bounds it: 4 * head_dim operations per row and cached token, so the tensor cores, if
// they can be kept fed; next to them stand one exp2 per row and token (16 a cycle per SM: as
// long as both products of 128 x 128 x 128 take) and the shared-memory reads of the operands.
// So one CTA per SM holds two STREAMS whose softmax and products alternate, and everything
// around them has warps of its own (18 warps):
//   warps 0..3, 4..7   softmax of stream 0 and 1: a thread owns a row (a TMEM lane)
//   warps 8..11        write the key tile: 128 tokens x head_dim, fp16(code * s + z)
//   warps 12..15       write the value tile: head_dim x 128 tokens, fp16(code * s + z)
//   warp 16            one thread issues the products (tcgen05.mma, accumulators in TMEM)
//   warp 17            stages the packed pages by bulk copies (8 blocks of 16 tokens a tile)
// With more than 128 rows per unit the streams are two tiles of 128 query rows, and both meet
// every key and value tile (its unpacking is then paid once per 256 rows); with up to 128 rows
// they are the same rows over the even and the odd tiles, and their sums are joined at the end.
//
//   S = Q K^T   A = query rows (fp16, scaled by a power of two per row so that bf16 channels
//               are exact), B = key tile, both from shared memory; fp32 in TMEM
//   softmax     row maximum of the tile (one pass over S in TMEM), a reference that moves only
//               when a logit would give p above 2^14 (then the row of O is rescaled in TMEM),
//               p = 2^(x - m) rounded to fp16 (2^-12 of each weight at most) over the S it came
//               from, the denominator summed in fp32
//   O += P V    A = P from TMEM, B = value tile
// The operands lie in shared memory in the K-major form without swizzle: 8-row pieces of 8 x 16
// bytes.  The order of the channels inside K (keys and queries alike) and of the value rows is
// free; it is chosen so that code words unpack without moving codes between lanes and 16-byte
// stores of neighbouring lanes lie side by side.
#include <atomic>

#include "kv4_attn.cuh"
#include "kv4_launch.cuh"

namespace pnmix {
namespace kv4 {
namespace {

constexpr int kThreads = 576;
constexpr int kTile = 128;                  // tokens of a key / value tile; rows of a stream
constexpr uint32_t kCommitLimit = 1u << 22; // try_wait rounds of a wait inside the CTA
constexpr float kSlack = 14.f;              // log2 of the largest p before the reference moves
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

// 32 consecutive columns of this thread's TMEM lane (warp-collective).
__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(at), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
        "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
        "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
        "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
        "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
        "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
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
  int lead, rt;     // rt: 256 (two row tiles) or 128 (one, even and odd tiles apart)
};

template <int D>
struct Smem {
  static constexpr int kQ = 0;                              // 2 x [128 rows][D]
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kK = kQ + 2 * kQBytes;               // 2 x [128 tokens][D]
  static constexpr int kKBytes = kTile * D * 2;
  static constexpr int kV = kK + 2 * kKBytes;               // [D channels][128 tokens]
  static constexpr int kVBytes = D * kTile * 2;
  static constexpr int kRing = kV + kVBytes;                // 2 x 8 blocks
  static constexpr int kRingBytes = 8 * 20 * D;
  static constexpr int kMl = kRing + 2 * kRingBytes;        // [128][2]: stream 1's m, l
  static constexpr int kBars = kMl + 128 * 8;
  static constexpr int kPlan = kBars + 256;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const __grid_constant__ ChunkArgs a) {
  using S = Smem<D>;
  constexpr int NG = D / 32, BB = 20 * D, kStride = D + 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  const Geo& g = a.g;
  const Batch& bt = a.bt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* ring_full = bars;        // [2] the staged blocks are in
  uint64_t* ring_empty = bars + 2;   // [2] both builders are done with them (8 warps)
  uint64_t* k_full = bars + 4;       // [2] key tile written (4 warps)
  uint64_t* k_empty = bars + 6;      // [2] its products are done
  uint64_t* v_full = bars + 8;       // value tile written (4 warps)
  uint64_t* v_empty = bars + 9;
  uint64_t* s_full = bars + 10;      // [2] logits of the stream are in TMEM
  uint64_t* p_full = bars + 12;      // [2] its weights are (4 warps)
  uint64_t* o_done = bars + 14;      // [2] its value products of this piece are done
  uint64_t* q_full = bars + 16;      // query tiles written (8 warps)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 17);
  volatile int* fail = reinterpret_cast<volatile int*>(bars + 18);
  long long* cost = reinterpret_cast<long long*>(smem + S::kPlan);
  int* units = reinterpret_cast<int*>(cost + bt.B + 1);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(ring_full + i, 1);
      mbar_init(ring_empty + i, 8);
      mbar_init(k_full + i, 4);
      mbar_init(k_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
    }
    mbar_init(v_full, 4);
    mbar_init(v_empty, 1);
    mbar_init(q_full, 8);
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
  build_plan<kThreads>(g, bt, a.rt, a.lead, cost, units, reinterpret_cast<long long*>(smem + S::kMl));
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool dual = a.rt == 256;

  // Bounded wait for phase `n` (counted from 0) of a barrier; false once anything in the CTA
  // gave up.
  auto wait = [&](uint64_t* bar, uint32_t n, uint32_t limit) -> bool {
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
  struct Span {
    int lo, n;              // first tile, tiles
    int rows, base_seen, row_first, most;
  };
  auto span_of = [&](const Piece& pc) {
    Span s;
    s.row_first = pc.tile * a.rt;
    s.rows = min(a.rt, pc.T * g.G - s.row_first);
    s.base_seen = pc.len - pc.T + 1;
    s.most = max(0, s.base_seen + (s.row_first + s.rows - 1) / g.G);   // tokens the last row sees
    const int nt = (s.most + kTile - 1) / kTile;
    s.lo = min((pc.lo + kTile - 1) / kTile, nt);                        // the tiles that start in [lo, hi)
    s.n = min((pc.hi + kTile - 1) / kTile, nt) - s.lo;
    return s;
  };

  if (warp < 8) {
    // ================================================================ softmax
    const int stream = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * stream, t_o = tmem + lanes + kTmemO + 128 * stream;
    float* ml = reinterpret_cast<float*>(smem + S::kMl) + 2 * row;
    uint32_t ns = 0, no = 0;   // logit tiles taken; pieces whose value products were waited for
    for_each_piece(g, bt, a.rt, a.lead, cost, units, a.wk, gridDim.x, tid == 0, [&](const Piece& pc) -> bool {
      const Span sp = span_of(pc);
      const int v = dual ? 128 * stream + row : row;     // row of the unit
      const bool live = v < sp.rows;
      const int r = sp.row_first + v, j = r / g.G, hg = r - j * g.G;
      // ---- this thread's query row -> A (in the one-tile form stream 1 has stream 0's)
      float fac = 0.f;
      {
        uint8_t* qa = smem + S::kQ + stream * S::kQBytes;
        const uint16_t* src = a.q.p + static_cast<long long>(pc.start + j) * a.q.ts + (pc.h * g.G + hg) * a.q.hs;
        float top = 0.f;
        for (int c = 0; live && c < D / 8; ++c) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + c);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xFFFF0000u))));
        }
        const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const int up = top > 0.f ? min(max(-ex, -90), 120) : 0;      // largest channel to [1, 2)
        const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        fac = g.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (live) w = __ldg(reinterpret_cast<const uint4*>(src) + c);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(x[i] << 16) * mul;
            f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u) * mul;
          }
          // position order inside 8 channels: 0, 4, 1, 5, 2, 6, 3, 7, as a code word unpacks
          *reinterpret_cast<uint4*>(qa + tile_off(128, row, 8 * c)) =
              make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]), pack_f16x2(f[3], f[7]));
        }
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      const int seen = live ? sp.base_seen + j : 0;

      float ref = -1e30f, den = 0.f;
      int mine = 0;       // tiles of this stream so far
      bool ok = true;
      for (int i = dual ? 0 : stream; i < sp.n; i += dual ? 1 : 2) {
        if (!(ok = wait(s_full + stream, ns, kCommitLimit))) break;
        ++ns;
        tc_fence_after();
        const int lim = seen - (sp.lo + i) * kTile;     // columns below it are visible
        const bool edge = __any_sync(0xffffffffu, lim < kTile);
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float x[32];
          tmem_ld32(t_s + 32 * c, x);
          if (edge) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * c + k >= lim) x[k] = -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) mx = fmaxf(mx, x[k]);
        }
        mx *= fac;          // -inf (or NaN from 0 * inf in a row that is not live) if nothing is visible
        bool move = mx > ref + kSlack;
        if (__any_sync(0xffffffffu, move)) {
          float f = 1.f;
          if (move) {
            f = ex2(ref - mx);
            ref = mx;
            den *= f;
          }
          if (mine > 0) {   // the commit of these logits covers the stream's earlier value products
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld32(t_o + 32 * c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= f;
              tmem_st32(t_o + 32 * c, o);
            }
          }
        }
        const float off = -ref;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float x[32];
          tmem_ld32(t_s + 32 * c, x);
          uint32_t p[16];
          float d0 = 0.f, d1 = 0.f;
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float p0 = ex2(fmaf(x[k], fac, off)), p1 = ex2(fmaf(x[k + 1], fac, off));
            if (edge) {
              if (32 * c + k >= lim) p0 = 0.f;
              if (32 * c + k + 1 >= lim) p1 = 0.f;
            }
            d0 += p0;
            d1 += p1;
            p[k / 2] = pack_f16x2(p0, p1);
          }
          den += d0 + d1;
          tmem_st16(t_s + 16 * c, p);     // over columns that were read
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
      float w0 = 1.f, w1 = 0.f;
      if (!dual) {        // join the streams: stream 0's threads read both rows of O
        if (stream == 1) {
          ml[0] = ref;
          ml[1] = den;
        }
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tc_fence_after();
        if (stream == 0) {
          const float m1 = ml[0], l1 = ml[1];
          const float m = l1 == 0.f ? ref : den == 0.f ? m1 : fmaxf(ref, m1);
          w0 = den == 0.f ? 0.f : ex2(ref - m);
          w1 = l1 == 0.f ? 0.f : ex2(m1 - m);
          den = (den == 0.f ? 0.f : den * w0) + (l1 == 0.f ? 0.f : l1 * w1);
          ref = m;
        }
      }
      if (dual || stream == 0) {
        const bool has0 = mine > 0, has1 = !dual && sp.n > 1;
        const float inv = den == 0.f ? 0.f : 1.f / den;
        float* part = a.wk.part + (static_cast<size_t>(pc.slot) * a.rt + v) * kStride;
        uint16_t* dst = a.out + static_cast<long long>(pc.start + j) * a.out_ts + (pc.h * g.G + hg) * a.out_hs;
        if (!pc.whole && live) *reinterpret_cast<float2*>(part) = make_float2(ref, den);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          if (has0) {
            tmem_ld32(t_o + 32 * c, o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0.f;
          }
          if (w0 != 1.f) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = w0 == 0.f ? 0.f : o[k] * w0;
          }
          if (has1) {
            float o1[32];
            tmem_ld32(t_o + 128 + 32 * c, o1);
            if (w1 != 0.f) {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = fmaf(o1[k], w1, o[k]);
            }
          }
          // column 8 i + w of a group is channel 4 w + i
          if (live && pc.whole) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {      // channels 8 h .. 8 h + 7: w = 2 h, 2 h + 1
              uint32_t wd[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int w = 2 * h + (k >> 1), i = 2 * (k & 1);
                const float x0 = den == 0.f ? 0.f : o[8 * i + w] * inv, x1 = den == 0.f ? 0.f : o[8 * (i + 1) + w] * inv;
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(x0, x1);
                memcpy(&wd[k], &b2, 4);
              }
              *reinterpret_cast<uint4*>(dst + 32 * c + 8 * h) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
            }
          } else if (live) {
#pragma unroll
            for (int w = 0; w < 8; ++w)
              *reinterpret_cast<float4*>(part + 4 + 32 * c + 4 * w) = make_float4(o[w], o[8 + w], o[16 + w], o[24 + w]);
          }
        }
      }
      tc_fence_before();
      // both streams are done with TMEM, and go on or stop alike
      uint32_t stop;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
          : "=r"(stop)
          : "r"(static_cast<uint32_t>(!ok || *fail))
          : "memory");
      return !stop;
    });
  } else if (warp < 12) {
    // ================================================================ key tiles
    const int t = tid - 256;                   // token of the tile
    const int blk = t >> 4, r = t & 15;
    uint32_t nr = 0;                            // tiles so far
    for_each_piece(g, bt, a.rt, a.lead, cost, units, a.wk, gridDim.x, false, [&](const Piece& pc) -> bool {
      const Span sp = span_of(pc);
      for (int i = 0; i < sp.n; ++i, ++nr) {
        const uint32_t buf = nr & 1u;
        if (!wait(ring_full + buf, nr >> 1, g.wait_limit)) return false;
        if (nr >= 2 && !wait(k_empty + buf, (nr >> 1) - 1, kCommitLimit)) return false;
        const uint8_t* src = smem + S::kRing + buf * S::kRingBytes + blk * BB;
        uint8_t* dst = smem + S::kK + buf * S::kKBytes;
        const bool there = (sp.lo + i) * kTile + t < sp.most;    // behind: whatever the page holds
        uint32_t sz[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k)
          sz[k] = there ? *reinterpret_cast<const uint32_t*>(src + 8 * D + r * (4 * NG) + 4 * k) : 0u;
#pragma unroll
        for (int pp = 0; pp < 4; ++pp) {
          const int piece = pp ^ ((t >> 1) & 3);     // eight lanes' pieces lie in different banks
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
            *reinterpret_cast<uint4*>(dst + tile_off(kTile, t, 32 * k) + (piece >> 1) * (kTile * 32) + (piece & 1) * 128) =
                make_uint4(x0, x1, x2, x3);
          }
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(k_full + buf);
          mbar_arrive(ring_empty + buf);
        }
      }
      return true;
    });
  } else if (warp < 16) {
    // ================================================================ value tiles
    const int bw = warp - 12;
    const int w = lane & 7, half = (lane >> 3) & 1, odd = lane >> 4;   // piece, pair of groups, octet parity
    uint32_t nr = 0;
    for_each_piece(g, bt, a.rt, a.lead, cost, units, a.wk, gridDim.x, false, [&](const Piece& pc) -> bool {
      const Span sp = span_of(pc);
      for (int i = 0; i < sp.n; ++i, ++nr) {
        const uint32_t buf = nr & 1u;
        if (!wait(ring_full + buf, nr >> 1, g.wait_limit)) return false;
        if (nr >= 1 && !wait(v_empty, nr - 1, kCommitLimit)) return false;
        const uint8_t* ring = smem + S::kRing + buf * S::kRingBytes + 10 * D;
        uint8_t* dst = smem + S::kV;
        const int left = sp.most - (sp.lo + i) * kTile;
        constexpr int kHalves = NG / 2;                   // pairs of channel groups
#pragma unroll
        for (int rep = 0; rep < 2; ++rep) {
          // an item: 8 tokens (octet), piece w, one pair of groups; D = 64 has one pair, so the
          // `half` bit names two more octets
          int octet, pair;
          if constexpr (kHalves == 2) {
            octet = 4 * bw + 2 * rep + odd;
            pair = half;
          } else {
            octet = 4 * bw + 2 * half + odd;
            pair = 0;
          }
          if (kHalves == 1 && rep) break;
          const uint8_t* blk = ring + (octet >> 1) * BB;
          const int r0 = (octet & 1) * 8;
          uint32_t cw[8], sz[8][2];
          // lanes of odd octets take each token pair the other way round: the two octets of a warp
          // then read rows of different parity
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int t = r0 + (k ^ odd);
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
              *reinterpret_cast<uint4*>(dst + (octet >> 1) * (D * 32) + (octet & 1) * 128 +
                                        (4 * (2 * pair + gp) + ch) * 256 + w * 16) =
                  make_uint4(x[ch][0], x[ch][1], x[ch][2], x[ch][3]);
          }
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v_full);
          mbar_arrive(ring_empty + buf);
        }
      }
      return true;
    });
  } else if (warp == 16) {
    // ================================================================ products
    if (lane == 0) {
      const uint32_t q0 = smem_u32(smem + S::kQ), k0 = smem_u32(smem + S::kK), v0 = smem_u32(smem + S::kV);
      constexpr uint32_t kIdescS = mma_idesc(kTile), kIdescO = mma_idesc(D);
      uint32_t nk = 0, nv = 0, nq = 0, np[2] = {0, 0};   // tiles taken, query tiles, weights taken
      auto logits = [&](int stream, uint32_t buf) {
        const uint64_t qa = tile_desc(q0 + stream * S::kQBytes), kb = tile_desc(k0 + buf * S::kKBytes);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_ss(tmem + 128 * stream, qa + s * (128 * 32 >> 4), kb + s * (kTile * 32 >> 4), kIdescS, s > 0);
        tc_commit(s_full + stream);
      };
      auto values = [&](int stream, bool accumulate, bool last) {
        const uint64_t vb = tile_desc(v0);
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
          mma_ts(tmem + kTmemO + 128 * stream, tmem + 128 * stream + 8 * s, vb + s * (D * 32 >> 4), kIdescO,
                 accumulate || s > 0);
        if (last) tc_commit(o_done + stream);
      };
      for_each_piece(g, bt, a.rt, a.lead, cost, units, a.wk, gridDim.x, false, [&](const Piece& pc) -> bool {
        const Span sp = span_of(pc);
        if (!wait(q_full, nq++, kCommitLimit)) return false;
        tc_fence_after();
        // the next key tile, once written
        auto key_tile = [&]() -> bool {
          if (!wait(k_full + (nk & 1u), nk >> 1, kCommitLimit)) return false;
          tc_fence_after();
          return true;
        };
        const int ahead = dual ? 1 : 2;
        for (int i = 0; i < ahead && i < sp.n; ++i) {
          if (!key_tile()) return false;
          logits(dual ? 0 : i, nk & 1u);
          if (dual) logits(1, nk & 1u);
          tc_commit(k_empty + (nk & 1u));
          ++nk;
        }
        for (int i = 0; i < sp.n; ++i) {
          for (int x = 0; x < (dual ? 2 : 1); ++x) {
            const int stream = dual ? x : i & 1;
            if (!wait(p_full + stream, np[stream]++, kCommitLimit)) return false;
            if (x == 0 && !wait(v_full, nv++, kCommitLimit)) return false;
            tc_fence_after();
            values(stream, i >= ahead, i + ahead >= sp.n);
            if (x == (dual ? 1 : 0)) tc_commit(v_empty);
            if (i + ahead < sp.n) {
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
      });
    }
    __syncwarp();
  } else {
    // ================================================================ staging
    uint32_t nr = 0;
    const size_t head_bytes = static_cast<size_t>(1 << (g.page_shift - 4)) * BB, page_bytes = head_bytes * g.Hkv;
    const int per_copy = g.page_shift > 7 ? 7 : g.page_shift;       // log2 tokens of a copy
    const int copies = kTile >> per_copy;
    uint32_t landed = 0;
    for_each_piece(g, bt, a.rt, a.lead, cost, units, a.wk, gridDim.x, false, [&](const Piece& pc) -> bool {
      const Span sp = span_of(pc);
      const int32_t* table = bt.table + static_cast<size_t>(pc.b) * bt.max_pages;
      const uint8_t* base = g.pages + static_cast<size_t>(pc.h) * head_bytes;
      auto page_of = [&](int i) {        // of this lane's copy of tile i
        const int tok = (sp.lo + i) * kTile + (lane << per_copy);
        if (lane >= copies || i >= sp.n || tok >= sp.most) return 0;
        const int id = __ldg(table + (tok >> g.page_shift));
        if (id >= 0 && id < g.n_pages) return id;
        raise(g.error, PNMIX_DEVERR_PAGE);
        return 0;
      };
      int id = page_of(0);
      for (int i = 0; i < sp.n; ++i, ++nr) {
        const uint32_t buf = nr & 1u;
        if (nr >= 2 && !__all_sync(0xffffffffu, wait(ring_empty + buf, (nr >> 1) - 1, kCommitLimit))) return false;
        const int tok = (sp.lo + i) * kTile + (lane << per_copy);
        const int blocks = min(8, (sp.most - (sp.lo + i) * kTile + 15) >> 4);       // of the tile
        const int mine = min(1 << (per_copy - 4), blocks - (lane << (per_copy - 4)));
        if (lane == 0) {
          proxy_fence();
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(ring_full + buf)),
                       "r"(blocks * BB)
                       : "memory");
        }
        __syncwarp();
        if (lane < copies && mine > 0)
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           smem_u32(smem + S::kRing + buf * S::kRingBytes) + (lane << (per_copy - 4)) * BB),
                       "l"(base + id * page_bytes + static_cast<size_t>((tok & ((1 << g.page_shift) - 1)) >> 4) * BB),
                       "r"(mine * BB), "r"(smem_u32(ring_full + buf))
                       : "memory");
        id = page_of(i + 1);
      }
      return true;
    });
    // every staged copy lands before the CTA's shared memory is given up
    landed = nr >= 2 ? nr - 2 : 0;
    for (; landed < nr; ++landed) {
      uint32_t spins = 0;
      while (!mbar_try_wait(ring_full + (landed & 1u), (landed >> 1) & 1u) && ++spins < g.wait_limit) {
      }
    }
  }
  __syncthreads();
  // After a stop products may still run: they are done before TMEM and the tiles are given up.
  if (*fail && warp == 16 && lane == 0) {
    mbar_init(bars + 24, 1);
    fence_mbar_init();
    tc_commit(bars + 24);
    for (uint32_t spins = 0; spins < kCommitLimit && !mbar_try_wait(bars + 24, 0u); ++spins) {
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
static cudaError_t launch_chunk_d(ChunkArgs& a, cudaStream_t s) {
  static std::atomic<int> cache[kMaxDevices];
  const size_t smem = Smem<D>::kPlan + plan_bytes(a.bt.B);
  auto kern = chunk_kernel<D>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (known) sms = cache[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(Smem<D>::kPlan + plan_bytes(kMaxBatch)))) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return e;
    if (known) cache[dev].store(sms, std::memory_order_relaxed);
  }
  kern<<<sms < kMaxChunkCtas ? sms : kMaxChunkCtas, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_chunk(const Geo& g, const Batch& bt, const Rows& q, const pnmix_rows& out, const Work& wk, int rt,
                         cudaStream_t s) {
  ChunkArgs a{};
  a.g = g;
  a.bt = bt;
  a.q = q;
  a.out = out.data;
  a.out_ts = out.token_stride;
  a.out_hs = out.head_stride;
  a.wk = wk;
  a.lead = 256;
  a.rt = rt;
  return g.D == 64 ? launch_chunk_d<64>(a, s) : launch_chunk_d<128>(a, s);
}

}  // namespace kv4
}  // namespace pnmix
