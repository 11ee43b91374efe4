// kv4_decode.cu -- attention over the 4-bit paged cache for few query rows per KV head (the
// decode step, a few drafted tokens), and the merge of split-K partials.
//
// What bounds it: each cached token of a KV head is 160 bytes (head_dim 128) and is met by the
// unit's few query rows once, so the kernel streams the pages; everything else has to hide
// behind that stream.  A warp takes a run of 32-token stages, two 16-token blocks each, through
// a ring of its own in shared memory, filled by bulk copies (a stage of one page is one
// contiguous copy).  A block is one 16-row tile of m16n8k16 products with the query rows as the
// 8 columns (NT column tiles of 8 rows):
//
//   logits   A = key codes, 16 tokens x 16 channels; a 32-bit code word holds four A registers,
//            each one AND (and one shift for two of them) away: nibbles 0 / 4 of the word
//            masked in place are an exact fp16 pair of code * 2^-24 (subnormals, which the
//            tensor cores take exactly), nibbles 1 / 5 of code * 2^-20, whose factor 16 is
//            divided out of the query operand.  B = query channels in the same order.  The
//            products run per group of 32 channels and the group's fp32 sum enters the logit
//            as s * sum + z * (sum of the query's channels of that group), both fp32.
//   softmax  p = 2^(x - m'), x the scaled logit in the log2 domain; the reference m' of a row
//            is moved only when p times the token's largest value scale would pass 2^15 (then to
//            2^8), so p * s stays inside fp16 whatever the size of the values and logits
//            (kv4_softmax.cuh), and the accumulators are rescaled a few times per run.
//   values   A = value codes, 16 channels x 16 tokens; two tokens' words are joined by a byte
//            permute and masked like the keys.  B = p * s_v per channel group, rounded once to
//            fp16 (2^-11 of each weight at most) and transposed by movmatrix from the logits'
//            register layout.  The zero points add sum(p * z_v) per group in fp32.
//
// The token that row i of an A tile holds is i / 2 for even i < 8 and 7 - i / 2 for odd (and 8
// more for i >= 8): with it neither the key rows (16-byte loads) nor the value pieces (8-byte
// loads) of a warp meet in a bank.  The query row is scaled by a power of two so its largest
// channel is in [2^13, 2^14): every bf16 channel down to 2^-24 of it is exact in fp16.
//
// Measured, the merge included: one token of 16 sequences of 32768 with 32 query and 8 KV heads
// (head_dim 128, so half of a column tile is empty) 142 us by graph replay, 4.7 TB/s or 72 % of a
// plain copy.  At half the length 51 % of DRAM and 52 % of the integer pipe are busy at 2.4
// instructions a cycle: nothing is full, and twelve warps per SM do not hide each other's latency
// (the `wait` of dependent instructions is the largest stall).  Tried and not faster: the blocks of a stage unrolled at four CTAs per SM (152 us),
// warps without work leaving early.
#include <atomic>

#include "kv4_attn.cuh"
#include "kv4_launch.cuh"
#include "kv4_softmax.cuh"

namespace pnmix {
namespace kv4 {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kStageTok = 32;
constexpr int kStages = 3;          // ring slots per warp
constexpr uint32_t kDrainLimit = 1u << 22;      // try_wait rounds for copies in flight after a wait ran out
constexpr float kTop = 32768.f;     // largest p * s before the row's reference moves
constexpr float kMinScale = 6.103515625e-05f;   // 2^-14: floor of a token's value scale in that test

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float2 half_pair(uint32_t w) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}

__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }

// n words (2 or 4) of a row, as one load.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = lds32(p);
  }
}

struct AttnArgs {
  Geo g;
  Batch bt;
  Rows q;
  uint16_t* out;
  long long out_ts, out_hs;
  Work wk;
  Grain grain;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
decode_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int NG = D / 32, RT = 8 * NT, BB = 20 * D, kStageBytes = 2 * BB, kStride = D + 4;
  extern __shared__ __align__(128) uint8_t smem[];
  const Geo& g = a.g;
  const Batch& bt = a.bt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  float* merge = reinterpret_cast<float*>(smem);           // [kWarps][RT][kStride], after the ring's use
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ long long tmp[2 * kWarps];
  __shared__ PieceSlot slots[kWarps];
  __shared__ float bases[kWarps][RT];      // of the warp's rows (kv4_softmax.cuh)
  uint64_t* full = bars[warp];
  if (lane == 0) {
    for (int k = 0; k < kStages; ++k) mbar_init(full + k, 1);
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;");
  const Plan& plan = build_plan<kThreads>(g, bt, RT, a.grain, smem + kWarps * kStages * kStageBytes, tmp);

  // tokens of this lane inside a block: A rows gq and gq + 8 (keys), tq's four (values)
  const int r0 = (gq & 1) ? 7 - (gq >> 1) : gq >> 1;
  const int tA = tq, tB = 7 - tq;
  const int vA = tA * (D / 2) + value_place<D>(tA, gq) * (2 * NG);
  const int vB = tB * (D / 2) + value_place<D>(tB, gq) * (2 * NG);
  const int page_shift = g.page_shift;
  const size_t head_bytes = static_cast<size_t>(1 << (page_shift - 4)) * BB;
  uint32_t nis = 0, ncons = 0;   // stages this warp issued and consumed
  bool dead = false;             // a staging wait ran out

  for_each_piece<false>(g, bt, RT, plan, a.wk, slots + warp, tid == 0, [&](const Piece& pc) -> bool {
    const int row_first = pc.tile * RT, nrows = min(RT, pc.T * g.G - row_first);
    // tokens that row r sees, and the tile's most
    const int base_seen = pc.len - pc.T + 1;
    const int tile_seen = max(0, base_seen + (row_first + nrows - 1) / g.G);
    const int least_seen = base_seen + row_first / g.G;
    const int nstage = (tile_seen + kStageTok - 1) / kStageTok;
    const int p_lo = min((pc.lo + kStageTok - 1) / kStageTok, nstage);   // the stages that start in [lo, hi)
    const int p_hi = min((pc.hi + kStageTok - 1) / kStageTok, nstage);
    const int per = (p_hi - p_lo + kWarps - 1) / kWarps;
    const int s_lo = min(p_lo + warp * per, p_hi), s_hi = min(s_lo + per, p_hi);

    // ---- staging: lane k holds the page(s) of the k-th stage of a run of 32
    const int32_t* table = bt.table + static_cast<size_t>(pc.b) * bt.max_pages;
    const uint8_t* head_pages = g.pages + static_cast<size_t>(pc.h) * head_bytes;
    const size_t page_bytes = head_bytes * g.Hkv;
    int issued = s_lo, id0 = 0, id1 = 0;
    auto page_of = [&](int token) {
      if (token >= tile_seen) return 0;
      const int id = __ldg(table + (token >> page_shift));
      if (id >= 0 && id < g.n_pages) return id;
      raise(g.error, PNMIX_DEVERR_PAGE);
      return 0;
    };
    auto issue = [&]() {
      if (issued >= s_hi || dead) return;
      const int k = (issued - s_lo) & 31;
      if (k == 0) {
        const int tok = (issued + lane) * kStageTok;
        id0 = issued + lane < s_hi ? page_of(tok) : 0;
        if (page_shift == 4) id1 = issued + lane < s_hi ? page_of(tok + kBlock) : 0;
      }
      const int p0 = __shfl_sync(0xffffffffu, id0, k), p1 = __shfl_sync(0xffffffffu, id1, k);
      const int tok = issued * kStageTok;
      const bool two = tile_seen - tok > kBlock;
      const uint32_t slot = nis % kStages;
      uint8_t* dst = ring + slot * kStageBytes;
      if (lane == 0 && pc.b != g.skip_seq) {
        const uint8_t* src = head_pages + p0 * page_bytes + static_cast<size_t>((tok & ((1 << page_shift) - 1)) >> 4) * BB;
        const bool split = two && page_shift == 4;
        const uint32_t n0 = two && !split ? 2 * BB : BB;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(full + slot)),
                     "r"(two ? 2 * BB : BB)
                     : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(dst)),
                     "l"(src), "r"(n0), "r"(smem_u32(full + slot))
                     : "memory");
        if (split)
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           smem_u32(dst + BB)),
                       "l"(head_pages + p1 * page_bytes), "r"(BB), "r"(smem_u32(full + slot))
                       : "memory");
      }
      ++nis;
      ++issued;
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) issue();

    // ---- the query rows as B operands: this lane holds row 8 nt + gq's channels 32 g + 8 tq ..
    uint32_t qb[NT][NG][4];
    float qsum[NT][NG][2];   // of columns 2 tq, 2 tq + 1, times 2^-24
    float fac[NT][2];        // scaled logit (log2) = fac * (sum_g s acc + z qsum)
    int seen[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int v = 8 * nt + gq, row = row_first + v;
      uint4 raw[NG];
      if (v < nrows) {
        const int j = row / g.G, hg = row - j * g.G;
        const uint16_t* src = a.q.p + static_cast<long long>(pc.start + j) * a.q.ts + (pc.h * g.G + hg) * a.q.hs;
#pragma unroll
        for (int k = 0; k < NG; ++k) raw[k] = __ldg(reinterpret_cast<const uint4*>(src + 32 * k + 8 * tq));
      } else {
#pragma unroll
        for (int k = 0; k < NG; ++k) raw[k] = make_uint4(0u, 0u, 0u, 0u);
      }
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;   // 2^ex <= top < 2^(ex + 1)
      const int up = top > 0.f ? min(max(13 - ex, -90), 120) : 0;
      const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
      float fs[NG];
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
        float x[8], s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16) * mul;
          x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * mul;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i];
        qb[nt][k][0] = pack_f16x2(x[0], x[4]);
        qb[nt][k][1] = pack_f16x2(x[1] * 0.0625f, x[5] * 0.0625f);
        qb[nt][k][2] = pack_f16x2(x[2], x[6]);
        qb[nt][k][3] = pack_f16x2(x[3] * 0.0625f, x[7] * 0.0625f);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        fs[k] = s * 0x1p-24f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int from = (2 * tq + c) * 4;   // a lane of that row
#pragma unroll
        for (int k = 0; k < NG; ++k) qsum[nt][k][c] = __shfl_sync(0xffffffffu, fs[k], from);
        const int u = __shfl_sync(0xffffffffu, up, from);
        fac[nt][c] = g.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + 24 - u) << 23);
        const int vc = 8 * nt + 2 * tq + c;
        seen[nt][c] = vc < nrows ? base_seen + (row_first + vc) / g.G : 0;
      }
    }

    float ref[NT][2], den[NT][2], acc[NT][2 * NG][4], zac[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ref[nt][c] = kFirstReference;
        if (gq == 0) bases[warp][8 * nt + 2 * tq + c] = 0.f;
        den[nt][c] = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k) zac[nt][k][c] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 2 * NG; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][j][i] = 0.f;
    }

    bool far = false;        // a row of the warp has a base other than 0
    __syncwarp();
    for (int st = s_lo; st < s_hi && !dead; ++st) {
      const uint32_t slot = ncons % kStages;
      {
        uint32_t spins = 0;
        while (!mbar_try_wait(full + slot, (ncons / kStages) & 1u)) {
          if (++spins >= g.wait_limit) {
            dead = true;
            break;
          }
        }
        dead = __any_sync(0xffffffffu, dead);
        if (dead) {
          if (lane == 0) raise(g.error, PNMIX_DEVERR_TIMEOUT);
          break;
        }
      }
      const uint8_t* buf = ring + slot * kStageBytes;
      const bool edge = (st + 1) * kStageTok > least_seen;   // some row does not see the whole stage

      // ---- logits of two blocks: x[nt][block][row of A][column]
      float x[NT][2][2][2];
#pragma unroll
      for (int bk = 0; bk < 2; ++bk) {
        const uint8_t* kc = buf + bk * BB;
        uint32_t w0[NG], w1[NG], s0[NG], s1[NG];
        load_words<NG>(kc + r0 * (D / 2) + tq * (4 * NG), w0);
        load_words<NG>(kc + (r0 + 8) * (D / 2) + tq * (4 * NG), w1);
        load_words<NG>(kc + 8 * D + r0 * (4 * NG), s0);
        load_words<NG>(kc + 8 * D + (r0 + 8) * (4 * NG), s1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) x[nt][bk][0][c] = x[nt][bk][1][c] = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const uint32_t h0 = w0[k] >> 8, h1 = w1[k] >> 8;
          const float2 f0 = half_pair(s0[k]), f1 = half_pair(s1[k]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816_free(d, w0[k] & 0x000F000Fu, w1[k] & 0x000F000Fu, w0[k] & 0x00F000F0u, w1[k] & 0x00F000F0u,
                          qb[nt][k][0], qb[nt][k][1]);
            mma16816_free(d, h0 & 0x000F000Fu, h1 & 0x000F000Fu, h0 & 0x00F000F0u, h1 & 0x00F000F0u, qb[nt][k][2],
                          qb[nt][k][3]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              x[nt][bk][0][c] = fmaf(f0.x, d[c], fmaf(f0.y, qsum[nt][k][c], x[nt][bk][0][c]));
              x[nt][bk][1][c] = fmaf(f1.x, d[2 + c], fmaf(f1.y, qsum[nt][k][c], x[nt][bk][1][c]));
            }
          }
        }
      }
      // ---- value scales of the same tokens, and the largest of each token
      uint32_t vs[2][2][NG];
      float top[2][2];
#pragma unroll
      for (int bk = 0; bk < 2; ++bk)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          load_words<NG>(buf + bk * BB + 18 * D + (r0 + 8 * r) * (4 * NG), vs[bk][r]);
          const int tok = st * kStageTok + bk * kBlock + 8 * r + r0;
          if (edge && tok >= tile_seen) {   // past the sequence: whatever the page holds there
#pragma unroll
            for (int k = 0; k < NG; ++k) vs[bk][r][k] = 0u;
          }
          __half2 m;
          memcpy(&m, &vs[bk][r][0], 4);
#pragma unroll
          for (int k = 1; k < NG; ++k) {
            __half2 o;
            memcpy(&o, &vs[bk][r][k], 4);
            m = __hmax2(m, o);
          }
          top[bk][r] = fmaxf(__low2float(m), kMinScale);
        }
      // ---- softmax weights
      float p[NT][2][2][2];
      bool over = far;         // rows with a base take the long way every time
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int bk = 0; bk < 2; ++bk)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float& xv = x[nt][bk][r][c];
              xv *= fac[nt][c];
              if (edge && st * kStageTok + bk * kBlock + 8 * r + r0 >= seen[nt][c]) xv = -INFINITY;
              p[nt][bk][r][c] = ex2(xv - ref[nt][c]);
              over |= p[nt][bk][r][c] * top[bk][r] > kTop;
            }
      if (__any_sync(0xffffffffu, over)) {
        far = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& base = bases[warp][8 * nt + 2 * tq + c];
            const float from = base;
            float mx = -INFINITY, m = -INFINITY;
            over = false;
#pragma unroll
            for (int bk = 0; bk < 2; ++bk)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float xv = x[nt][bk][r][c];
                over |= ex2((xv - from) - ref[nt][c]) * top[bk][r] > kTop;
                mx = fmaxf(mx, xv);
                m = fmaxf(m, xv + log2f(top[bk][r]));
              }
            const bool move = __ballot_sync(0xffffffffu, over) & (0x11111111u << tq);     // some lane of the column
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            const float to = move ? row_base(from, mx, m) : from;
            m = -INFINITY;
#pragma unroll
            for (int bk = 0; bk < 2; ++bk)
#pragma unroll
              for (int r = 0; r < 2; ++r) m = fmaxf(m, (x[nt][bk][r][c] - to) + log2f(top[bk][r]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (move) {
              const RowRef now = {to, row_reference(m)};
              const float f = ex2(move_exponent({from, ref[nt][c]}, now, 1.f));
              ref[nt][c] = now.ref;
              if (gq == 0) base = to;
              den[nt][c] *= f;
#pragma unroll
              for (int k = 0; k < NG; ++k) zac[nt][k][c] *= f;
#pragma unroll
              for (int j = 0; j < 2 * NG; ++j) {
                acc[nt][j][c] *= f;
                acc[nt][j][2 + c] *= f;
              }
            }
            far |= __any_sync(0xffffffffu, to != 0.f);
#pragma unroll
            for (int bk = 0; bk < 2; ++bk)
#pragma unroll
              for (int r = 0; r < 2; ++r) p[nt][bk][r][c] = ex2((x[nt][bk][r][c] - to) - ref[nt][c]);
          }
        __syncwarp();      // the bases are written
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          den[nt][c] += (p[nt][0][0][c] + p[nt][0][1][c]) + (p[nt][1][0][c] + p[nt][1][1][c]);
      // ---- values
#pragma unroll
      for (int bk = 0; bk < 2; ++bk) {
        const uint8_t* vc = buf + bk * BB + 10 * D;
        uint32_t wA[NG / 2], wB[NG / 2], wC[NG / 2], wD[NG / 2];   // two groups' 16 bits each
        load_words<NG / 2>(vc + vA, wA);
        load_words<NG / 2>(vc + vB, wB);
        load_words<NG / 2>(vc + vA + 8 * (D / 2), wC);
        load_words<NG / 2>(vc + vB + 8 * (D / 2), wD);
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const uint32_t sel = (k & 1) ? 0x7632u : 0x5410u;
          const uint32_t lo = __byte_perm(wA[k >> 1], wB[k >> 1], sel), hi = __byte_perm(wC[k >> 1], wD[k >> 1], sel);
          const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
          const float2 f0 = half_pair(vs[bk][0][k]), f1 = half_pair(vs[bk][1][k]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float(&pb)[2][2] = p[nt][bk];
            const uint32_t b0 = movmatrix(pack_f16x2(pb[0][0] * f0.x, pb[0][1] * f0.x));
            const uint32_t b1 = movmatrix(pack_f16x2(pb[1][0] * f1.x, pb[1][1] * f1.x));
#pragma unroll
            for (int c = 0; c < 2; ++c) zac[nt][k][c] = fmaf(pb[0][c], f0.y, fmaf(pb[1][c], f1.y, zac[nt][k][c]));
            mma16816_free(acc[nt][2 * k], lo & 0x000F000Fu, lo & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u, b0,
                          b1);
            mma16816_free(acc[nt][2 * k + 1], lo8 & 0x000F000Fu, lo8 & 0x00F000F0u, hi8 & 0x000F000Fu,
                          hi8 & 0x00F000F0u, b0, b1);
          }
        }
      }
      ++ncons;
      __syncwarp();   // the slot is read; the next copy may overwrite it
      issue();
    }
    // a wait ran out: let the copies in flight land before the ring is used again
    if (dead) {
      for (; ncons < nis; ++ncons) {
        uint32_t spins = 0;
        if (pc.b == g.skip_seq) continue;      // the test hook: there are none
        while (!mbar_try_wait(full + ncons % kStages, (ncons / kStages) & 1u) && ++spins < kDrainLimit) {
        }
      }
    }
    __syncthreads();   // every warp is done with its ring: the merge may overlay it
    if (far) {         // rows with a base: their sums to that reference, which fp32 holds
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float base = bases[warp][8 * nt + 2 * tq + c];
          if (base == 0.f) continue;
          const float f = ex2(ref[nt][c]);
          ref[nt][c] = base;
          den[nt][c] *= f;
#pragma unroll
          for (int k = 0; k < NG; ++k) zac[nt][k][c] *= f;
#pragma unroll
          for (int j = 0; j < 2 * NG; ++j) {
            acc[nt][j][c] *= f;
            acc[nt][j][2 + c] *= f;
          }
        }
    }

    // ---- join the lanes of a column, then the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          den[nt][c] += __shfl_xor_sync(0xffffffffu, den[nt][c], o);
#pragma unroll
          for (int k = 0; k < NG; ++k) zac[nt][k][c] += __shfl_xor_sync(0xffffffffu, zac[nt][k][c], o);
        }
        float* row = merge + (warp * RT + 8 * nt + 2 * tq + c) * kStride;
        if (gq == 0) {
          row[0] = ref[nt][c];
          row[1] = den[nt][c];
        }
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const float z = zac[nt][k][c];
          *reinterpret_cast<float4*>(row + 4 + 32 * k + 4 * gq) =
              make_float4(fmaf(acc[nt][2 * k][c], 0x1p24f, z), fmaf(acc[nt][2 * k][2 + c], 0x1p20f, z),
                          fmaf(acc[nt][2 * k + 1][c], 0x1p24f, z), fmaf(acc[nt][2 * k + 1][2 + c], 0x1p20f, z));
        }
      }
    __syncthreads();
    for (int i = tid; i < nrows * (D / 4); i += kThreads) {
      const int v = i / (D / 4), c4 = i - v * (D / 4);
      float m = kFirstReference, l = 0.f;
      float w[kWarps];
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float* row = merge + (k * RT + v) * kStride;
        // a warp that saw nothing has l = 0 (a NaN counts as something)
        m = row[1] == 0.f ? m : fmaxf(m, row[0]);
      }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float* row = merge + (k * RT + v) * kStride;
        w[k] = row[1] == 0.f ? 0.f : ex2(row[0] - m);
        if (row[1] != 0.f) {
          const float4 r = *reinterpret_cast<const float4*>(row + 4 + 4 * c4);
          l = fmaf(row[1], w[k], l);
          o.x = fmaf(r.x, w[k], o.x);
          o.y = fmaf(r.y, w[k], o.y);
          o.z = fmaf(r.z, w[k], o.z);
          o.w = fmaf(r.w, w[k], o.w);
        }
      }
      if (pc.whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int row = row_first + v, j = row / g.G, hg = row - j * g.G;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        uint2 pk;
        memcpy(&pk.x, &lo, 4);
        memcpy(&pk.y, &hi, 4);
        *reinterpret_cast<uint2*>(a.out + static_cast<long long>(pc.start + j) * a.out_ts +
                                  (pc.h * g.G + hg) * a.out_hs + 4 * c4) = pk;
      } else {
        float* part = part_of<D>(a.wk.part, pc.slot, RT);
        if (c4 == 0) reinterpret_cast<float2*>(part)[v] = make_float2(m, l);
        reinterpret_cast<float4*>(part + 2 * RT)[c4 * RT + v] = o;
      }
    }
    __syncthreads();
    return true;
  });
}

// out_r = sum_s O_s 2^(m_s - m*) / sum_s l_s 2^(m_s - m*) over the partials of a unit's rows.
// CTA x takes the unit that begins in CTA x of the launch before, 8 rows of it (rows inner, as
// the partials lie), and turns them around in shared memory
// for the stores.
// AHEAD partials at a time, all of their loads first.  After the row kernels eight (108
// registers): a unit has many partials and the merge is a few round trips (with four, 5 ragged
// tokens of 8 sequences 36.9 instead of 35.6 us).  After the tcgen05 kernel, whose units have two
// or three mostly but 128 or 256 rows, four (72 registers, seven CTAs per SM instead of four):
// 2 x 1024 tokens over 8192 cached ones 314 instead of 319 us.
template <int D, int AHEAD>
__global__ void __launch_bounds__(kThreads)
merge_kernel(const __grid_constant__ AttnArgs a, int RT) {
  constexpr int C4 = D / 4, kRows = 8, kLanes = kThreads / kRows;    // threads per row
  __shared__ float2 out_tile[kRows][C4 + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = blockIdx.x;
  const UnitInfo f = a.wk.info[first];
  if (f.last < 0) return;
  const int n = f.last - first + 1;
  const int v0 = blockIdx.y * kRows, r = threadIdx.x & (kRows - 1), c0 = threadIdx.x / kRows, v = v0 + r;
  if (v0 >= f.rows) return;
  constexpr int kC = C4 / kLanes;
  float m = kFirstReference, l = 0.f;
  float4 o[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (v < f.rows) {
    for (int k0 = 0; k0 < n; k0 += AHEAD) {
      float2 x[AHEAD];
      float4 t[AHEAD][kC];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        x[k] = make_float2(kFirstReference, 0.f);
        if (k0 + k < n) {
          const float* p = part_of<D>(a.wk.part, slot_of(first + k0 + k, first), RT);
          x[k] = reinterpret_cast<const float2*>(p)[v];
#pragma unroll
          for (int i = 0; i < kC; ++i) t[k][i] = reinterpret_cast<const float4*>(p + 2 * RT)[(c0 + i * kLanes) * RT + v];
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (x[k].y != 0.f) top = fmaxf(top, x[k].x);      // a partial that saw nothing has l = 0
      const float old = ex2(m - top);
      m = top;
      l *= old;
#pragma unroll
      for (int i = 0; i < kC; ++i) o[i] = make_float4(o[i].x * old, o[i].y * old, o[i].z * old, o[i].w * old);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (x[k].y == 0.f) continue;
        const float w = ex2(x[k].x - m);
        l = fmaf(x[k].y, w, l);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          o[i].x = fmaf(t[k][i].x, w, o[i].x);
          o[i].y = fmaf(t[k][i].y, w, o[i].y);
          o[i].z = fmaf(t[k][i].z, w, o[i].z);
          o[i].w = fmaf(t[k][i].w, w, o[i].w);
        }
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o[i].x * inv, o[i].y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o[i].z * inv, o[i].w * inv);
    float2 pk;
    memcpy(&pk.x, &lo, 4);
    memcpy(&pk.y, &hi, 4);
    out_tile[r][c0 + i * kLanes] = pk;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * C4; i += kThreads) {
    const int rr = i / C4, c = i - rr * C4;
    if (v0 + rr >= f.rows) break;
    const int row = f.row_first + v0 + rr, j = row / a.g.G, hg = row - j * a.g.G;
    uint16_t* dst = a.out + static_cast<long long>(f.start + j) * a.out_ts + (f.h * a.g.G + hg) * a.out_hs;
    reinterpret_cast<float2*>(dst)[c] = out_tile[rr][c];
  }
}

constexpr int kMaxDevices = 64;

// CTAs that fit the current device at once; for up to 1024 sequences and for more, whose plan
// leaves room for one CTA less (the answer must not depend on what was called first).
template <int D, int NT>
cudaError_t wave_of(int batch, int* wave) {
  constexpr int kSmall = 1024;
  static std::atomic<int> caches[2][kMaxDevices];
  std::atomic<int>* cache = caches[batch > kSmall];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (known && (*wave = cache[dev].load(std::memory_order_relaxed)) != 0) return cudaSuccess;
  auto kern = decode_kernel<D, NT>;
  const size_t ring = kWarps * kStages * 40 * D;
  const int most = static_cast<int>(ring + plan_bytes(kMaxBatch));
  int sms = 0, per = 0;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
      (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
           &per, kern, kThreads, ring + plan_bytes(batch > kSmall ? kMaxBatch : kSmall))) != cudaSuccess)
    return e;
  *wave = sms * (per > 0 ? per : 1);
  if (known) cache[dev].store(*wave, std::memory_order_relaxed);
  return cudaSuccess;
}

constexpr int kMaxCtas = 1024;

}  // namespace

// Query rows of a unit: 8 or 16 in the kernel above, which passes over the pages once per unit,
// 128 or 256 in the tcgen05 one, whose time hardly depends on the rows up to 128.  By the rows
// that a sequence has on the average for a KV head (rows = G * tokens), measured:
//   head_dim 128, 16 x 32K x 8 heads:  16 rows 283 us, 24 rows 416 against 398 us, 48 rows 618
//     against 394 us; 8 x 8K x 8 heads:  24 rows 70 against 72 us, 48 rows 98 against 73 us
//   head_dim 64, 8 x 8K x 8 heads:  20 rows 48 against 68 us, 48 rows 66 against 68 us, 64 rows
//     82 against 66 us
// Where some sequence may have more than 128 rows the average says less.  16 against 256 rows, 4
// rows per token and KV head, 8 heads:  64 tokens of 64 sequences, 4K cached, 127 against 363 us;
// a chunk of 256 tokens at 8K among 127 single ones at 2K (12 rows on the average) 353 against
// 437 us; but a chunk of 128 at 32K among 31 single ones at 512 (20 rows) 436 against 170 us, and
// of 64 among 63 (8 rows) 244 against 153 us.  So up to 16, one tile of most sequences.  (All of it
// measured before the many-row kernel's reference stood lower, which costs it 2 to 4 %, at head_dim 64
// 10 %, and before the row kernel's logits had a base, 1 %.)
static int tile_rows(const Geo& g, const Batch& bt) {
  const int most = g.G * bt.max_q;
  const double mean = static_cast<double>(g.G) * bt.n_tokens / bt.B;
  if (most <= 8) return 8;
  if (most <= 16 || mean <= (most > 128 ? 16 : g.D == 128 ? 24 : 48)) return 16;
  return most <= 128 ? 128 : 256;
}

static int most_ctas(int rt) { return rt > 16 ? kMaxChunkCtas : kMaxCtas; }

// First the notes on shared units, then the partials, and the plans of the tcgen05 kernel.
static size_t info_bytes(int rt) { return (most_ctas(rt) * sizeof(UnitInfo) + 255) / 256 * 256; }

static size_t part_bytes(const Geo& g, int rt) { return 2 * most_ctas(rt) * part_floats(g.D, rt) * sizeof(float); }

size_t attention_workspace_bytes(const Geo& g, const Batch& bt) {
  const int rt = tile_rows(g, bt);
  return info_bytes(rt) + part_bytes(g, rt) + (rt > 16 ? kMaxChunkCtas * plan_bytes(bt.B) : 0);
}

template <int D, int NT>
static cudaError_t launch_rows(const AttnArgs& a, int* ctas, cudaStream_t s) {
  const size_t smem = kWarps * kStages * 40 * D + plan_bytes(a.bt.B);
  int wave = 0;
  const cudaError_t e = wave_of<D, NT>(a.bt.B, &wave);
  if (e != cudaSuccess) return e;
  *ctas = wave < kMaxCtas ? wave : kMaxCtas;
  decode_kernel<D, NT><<<*ctas, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_merge(const AttnArgs& a, int ctas, int rt, cudaStream_t s) {
  // the merge is resident early and waits for the partials (griddepcontrol)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, rt / 8);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return rt > 16 ? cudaLaunchKernelEx(&cfg, merge_kernel<D, 4>, a, rt) : cudaLaunchKernelEx(&cfg, merge_kernel<D, 8>, a, rt);
}

cudaError_t launch_attention(const Geo& g, const Batch& bt, const pnmix_rows& q, const pnmix_rows& out, void* ws,
                             cudaStream_t s) {
  const int rt = tile_rows(g, bt);
  AttnArgs a{};
  a.g = g;
  a.bt = bt;
  a.q = {q.data, q.token_stride, q.head_stride};
  a.out = out.data;
  a.out_ts = out.token_stride;
  a.out_hs = out.head_stride;
  a.grain = {384, 256};
  a.wk.info = static_cast<UnitInfo*>(ws);
  a.wk.part = reinterpret_cast<float*>(static_cast<char*>(ws) + info_bytes(rt));
  int ctas = 0;
  cudaError_t e;
  if (rt > 16)
    e = launch_chunk(g, bt, a.q, out, a.wk, reinterpret_cast<uint8_t*>(a.wk.part) + part_bytes(g, rt), rt, &ctas, s);
  else if (g.D == 64)
    e = rt == 8 ? launch_rows<64, 1>(a, &ctas, s) : launch_rows<64, 2>(a, &ctas, s);
  else
    e = rt == 8 ? launch_rows<128, 1>(a, &ctas, s) : launch_rows<128, 2>(a, &ctas, s);
  if (e != cudaSuccess) return e;
  return g.D == 64 ? launch_merge<64>(a, ctas, rt, s) : launch_merge<128>(a, ctas, rt, s);
}

}  // namespace kv4
}  // namespace pnmix
