// kv4_io.cu -- rows in and out of the 4-bit paged cache: per-head norm and rotation of
// queries and keys, the quantised write (alone or fused behind the rotation) and the
// read-back.  One kernel for the first two, one for the last.
//
// All three move bytes: a bf16 row of 128 channels is 256 bytes and its packed form 80, so
// device memory bounds long inputs, closely followed by the instructions (7 to 10 a channel),
// and latency the decode step.  Four lanes hold a head's row, lane w the channels 8w .. 8w + 7
// of every group of 32: then the norm's sum and a group's minimum and maximum are two
// shuffles, the partner channels of a whole-head rotation (D / 2 away, D / 64 groups) are in
// the same lane, and a lane's codes are one key piece or two neighbouring value pieces, each
// one store.  (With D / 8 lanes of 8 channels, the first form, every row took eight more
// shuffles and narrow stores: 123 us instead of 59 for 16384 tokens of 40 heads, and the
// read-back, with integer conversions at a quarter of the rate, 96 us instead of 62 for
// 2 x 32768 tokens of 8 heads.  These are 5.6 and 5.7 TB/s, 86 % of a plain copy; the write of
// 16384 tokens of 8 + 8 heads takes 25 us, 3.5 TB/s or 54 %, and is held by its instructions.)
// A warp's eight rows are eight tokens of a head where there are that many: their packed rows
// lie side by side.  A token's angles (fp64, reduced to a turn, one sincospi per pair) and its
// place in the cache are worked out once per CTA, while the first rows' loads are in flight; the
// next row's loads are issued before a row is worked on.
//
// Query rows are normed and rotated in fp32, key rows in fp64: a key is rounded to bf16 and then
// to a 4-bit code, and neither forgives a last bit.  In fp32 one key in 21000 became the
// neighbouring bf16, and where that key was its group's end the scale, the zero and codes of the
// group moved by a step.  In fp64 the key is bf16(fp32(y)) of the definition's y but for a chance
// of 2^-28 or so.  The products, sums and roundings of both are written out, so every form of the
// kernel rounds alike and the fused write gives the bits of the separate calls.
#include "kv4.cuh"
#include "kv4_launch.cuh"

namespace pnmix {
namespace kv4 {
namespace {

// Threads of a CTA; a row takes four.  Measured at the large cases (128 / 256 threads): norm and
// rotation, then all in fp32, 59 / 66 us, write and read back 54 / 57 us with 128 threads in the read-back's kernel
// too, which alone takes 66 / 61 us.
constexpr int kInThreads = 128, kOutThreads = 256;
constexpr int kInRows = kInThreads / 4, kOutRows = kOutThreads / 4;   // rows a CTA works on at once
constexpr int kMaxTok = 16;                 // tokens per CTA at most
constexpr uint32_t kOnes = 0x3F803F80u;     // 1, 1 in bf16
constexpr int kSms = 148;                   // of a B200: small calls are cut so that each has work

// Sequence of packed row `row`: the last b with q_start[b] <= row, or -1 for a row outside
// every sequence.  Called by a whole warp.
__device__ __forceinline__ int seq_of_row(const Batch& bt, int row, int lane) {
  if (!bt.q_start) return row < bt.B * bt.uniform ? row / bt.uniform : -1;
  int c = 0;   // entries <= row among the batch + 1
  for (int base = 0; base <= bt.B; base += 32) {
    const int i = base + lane;
    const bool le = i <= bt.B && __ldg(bt.q_start + i) <= row;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    c += n;
    if (n < 32) break;   // ascending: nothing further is <= row
  }
  return c > bt.B ? -1 : c - 1;
}

// Byte offset in the pages of the block (head 0) that holds row `row`, and the row's token
// in it; offset -1: no place, -2: the row belongs to no sequence.  Called by a whole warp.
__device__ __forceinline__ void row_place(const Geo& g, const Batch& bt, int row, int lane, long long& off, int& tok) {
  off = -2;
  tok = 0;
  if (row >= bt.n_tokens) return;
  const int b = seq_of_row(bt, row, lane);
  if (b < 0) return;
  const int s = bt.q_start ? __ldg(bt.q_start + b) : b * bt.uniform;
  const int e = bt.q_start ? __ldg(bt.q_start + b + 1) : s + bt.uniform;
  const long long pos = static_cast<long long>(__ldg(bt.kv_len + b)) - e + row;   // kv_len - T + (row - s)
  off = -1;
  if (pos < 0 || pos >= (static_cast<long long>(bt.max_pages) << g.page_shift)) {
    if (lane == 0) raise(g.error, PNMIX_DEVERR_BATCH);
    return;
  }
  const int page = __ldg(bt.table + static_cast<size_t>(b) * bt.max_pages + (pos >> g.page_shift));
  if (page < 0 || page >= g.n_pages) {
    if (lane == 0) raise(g.error, PNMIX_DEVERR_PAGE);
    return;
  }
  const int inside = static_cast<int>(pos) & ((1 << g.page_shift) - 1);
  const int per = 1 << (g.page_shift - 4);   // blocks of a page and head
  off = (static_cast<long long>(page) * g.Hkv * per + (inside >> 4)) * block_bytes(g.D);
  tok = inside & 15;
}

__device__ __forceinline__ void unpack8(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    memcpy(&w[i], &h, 4);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Minimum / maximum of bf16 pairs that return NaN where either is one.
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two fp32 lanes to an instruction, rounded like the scalar ones: the write is bound by the
// instructions it issues (16384 tokens of 8 + 8 heads 24.8 instead of 26.7 us; in the read-back
// they gained nothing).
__device__ __forceinline__ uint64_t both(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 lanes_of(uint64_t a) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The contract's code is rint(fl(fl(x - z) / s)) clamped to [0, 15].  The correctly rounded
// quotient comes from the correctly rounded reciprocal inv = fl(1 / s) without a division
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): with d = fl(x - z) and q = fl(d inv), fl(q + fl(d - q s) inv) = fl(d / s), the residual
// being exact.  The rounding to a whole number is an addition of 1.5 * 2^23.  (Deciding by q
// alone and dividing only near half-integers took longer: bf16 differences over an fp16 scale
// are exact half-integers once in 1500 values, so half of the warps had one to divide.)
__device__ __forceinline__ uint64_t code_sum(uint64_t x, uint64_t minus_z, uint64_t minus_s, uint64_t inv) {
  constexpr float kMagic = 12582912.f;
  const uint64_t d = add2(x, minus_z), q = mul2(d, inv);
  return add2(fma2(fma2(q, minus_s, d), inv, q), both(kMagic, kMagic));      // the codes in the low bits
}

// Codes of the eight values of a bf16 row piece; `plain`: none needs the clamp.
__device__ __forceinline__ uint32_t codes_of(uint4 raw, uint32_t sz, float inv, bool plain) {
  const float s = -__half2float(__ushort_as_half(static_cast<uint16_t>(sz & 0xFFFFu)));
  const float z = -__half2float(__ushort_as_half(static_cast<uint16_t>(sz >> 16)));
  const uint64_t s2 = both(s, s), z2 = both(z, z), inv2 = both(inv, inv);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t word = plain ? 0u - 0x4B400000u * 0x11111111u : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 c = lanes_of(code_sum(both(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), z2, s2, inv2));
    if (plain) {
      word += __float_as_uint(c.x) << (8 * i);
      word += __float_as_uint(c.y) << (8 * i + 4);
    } else {
      word |= static_cast<uint32_t>(min(max(__float_as_int(c.x) - 0x4B400000, 0), 15)) << (8 * i);
      word |= static_cast<uint32_t>(min(max(__float_as_int(c.y) - 0x4B400000, 0), 15)) << (8 * i + 4);
    }
  }
  return word;
}

// n words (2 or 4) as one access.
template <int N>
__device__ __forceinline__ void put_words(uint8_t* p, const uint32_t (&w)[N]) {
  if constexpr (N == 4)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int N>
__device__ __forceinline__ void get_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  }
}

// A lane's codes (word g: eight channels of group g) <-> its two neighbouring value pieces (a
// piece has four channels of every group, 16 bits each).
template <int NG>
__device__ __forceinline__ void to_pieces(const uint32_t (&w)[NG], uint32_t (&p)[NG]) {
#pragma unroll
  for (int i = 0; i < NG / 2; ++i) {
    p[i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
    p[NG / 2 + i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
  }
}
template <int NG>
__device__ __forceinline__ void from_pieces(const uint32_t (&p)[NG], uint32_t (&w)[NG]) {
#pragma unroll
  for (int i = 0; i < NG / 2; ++i) {
    w[2 * i] = __byte_perm(p[i], p[NG / 2 + i], 0x5410);
    w[2 * i + 1] = __byte_perm(p[i], p[NG / 2 + i], 0x7632);
  }
}

// x c + o s: a rotated channel x of a pair whose other one is o (s negative for the pair's first).
__device__ __forceinline__ float turned(float x, float o, float c, float s) { return __fmaf_rn(x, c, __fmul_rn(o, s)); }
__device__ __forceinline__ double turned(double x, double o, double c, double s) {
  return __fma_rn(x, c, __dmul_rn(o, s));
}
__device__ __forceinline__ void turn(float& p, float& q, float c, float s) {
  const float p0 = p;
  p = turned(p0, q, c, -s);
  q = turned(q, p0, c, s);
}
// The pair (y, z), turned and times r.
__device__ __forceinline__ void turn64(double y, double z, double c, double s, double r, float& p, float& q) {
  p = static_cast<float>(__dmul_rn(turned(y, z, c, -s), r));
  q = static_cast<float>(__dmul_rn(turned(z, y, c, s), r));
}

// How the rotation finds a channel's partner: in the same lane (pairs D / 2 apart), next to it
// (interleaved), or through shared memory (any other distance).
enum { kHalves = 0, kNext = 1, kAnywhere = 2 };

struct IoArgs {
  Geo g;
  Batch bt;
  pnmix_rope rope;
  int n_tokens;
  int nq, nk, nv;          // heads of q (rotated, stored as bf16), k (rotated, stored or packed), v (packed)
  int tok_shift;           // log2 of the CTA's tokens
  Rows q, k, v;
  uint16_t* qo;
  uint16_t* ko;
  long long qo_ts, qo_hs, ko_ts, ko_hs;
  const uint16_t* qw;
  const uint16_t* kw;
  const int32_t* positions;
};

// Entries of a token's angles in shared memory: cos, sin, and a step of 16 bytes so that the
// eight tokens of a warp meet in no bank.  In fp64 for the keys, in fp32 for the queries.
__host__ __device__ __forceinline__ int turn_stride(int half) { return 2 * half + 4; }
__host__ __device__ __forceinline__ int turn_stride64(int half) { return 2 * half + 2; }

// cos and sin of pos * freq.  The fp64 product of a 31-bit and a 24-bit number is off by 2^-53 of
// itself; what is left of it after n turns by Cody and Waite's reduction (2 pi in two parts, n
// below 2^29) by 2^-51.
__device__ __forceinline__ void turn_of(int pos, float freq, double& c, double& s) {
  const double a = __dmul_rn(static_cast<double>(pos), static_cast<double>(freq));
  const double n = rint(__dmul_rn(a, 0.15915494309189533577));
  double r = __fma_rn(-n, 6.28318530717958647693, a);
  r = __fma_rn(-n, 2.44929359829470635445e-16, r);
  sincospi(__dmul_rn(r, 0.31830988618379067154), &s, &c);
}

// ROPE: q and k rows are normed and rotated.  QUANT: k and v rows go to the cache (otherwise
// k rows are stored like q's).
// CTAs per SM.  Rotating kernels of 128 channels: six (80 registers, 16 to 128 bytes of spills in four
// of the six forms).  At seven the fp64 of the keys spills 250 bytes: 94 instead of 66 us for the norm
// of 16384 tokens of 32 + 8 heads, 28.6 instead of 24.0 us for the fused write of 3900 ragged tokens of
// 28 + 4 + 4 heads; five take 68 and 26.  (All rows in fp32 at seven took 58 and 21 us.)  64 channels:
// seven, which is what 72 registers leave room for.  The plain write: eight (64 registers); ten took
// 28.7 instead of 26.7 us, before two lanes an instruction.  256 channels: three, the registers that
// they need.
template <int D, bool ROPE, bool QUANT, int PAIRS>
__global__ void __launch_bounds__(kInThreads, D == 256 ? 3 : !ROPE ? 8 : D == 128 ? 6 : 7)
rows_in_kernel(const __grid_constant__ IoArgs a) {
  constexpr int NG = D / 32;
  // [token][cos, sin] in fp64, the same in fp32, then [warp][8 rows][D + 4]
  extern __shared__ __align__(16) double turns64[];
  __shared__ long long place[kMaxTok];
  __shared__ int place_tok[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, w = lane & 3;
  const int ntok = 1 << a.tok_shift, tok0 = blockIdx.x << a.tok_shift;
  const int total = (a.nq + a.nk + a.nv) << a.tok_shift;   // rows of this CTA, tokens inner
  const int half = a.rope.rot_dim >> 1;
  float* const turns32 = reinterpret_cast<float*>(turns64 + (turn_stride64(half) << a.tok_shift));

  // row of a lane group: kind 0 q, 1 k, 2 v; -1 none
  auto find = [&](int rho, int& t, int& head) {
    t = rho & (ntok - 1);
    head = rho >> a.tok_shift;
    if (rho >= total || tok0 + t >= a.n_tokens) return -1;
    if (head < a.nq) return 0;
    head -= a.nq;
    if (head < a.nk) return 1;
    head -= a.nk;
    return 2;
  };
  auto load = [&](int rho, uint4 (&v)[NG]) {
    int t, head;
    const int kind = find(rho, t, head);
    if (kind < 0) {
#pragma unroll
      for (int k = 0; k < NG; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    const Rows& r = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const uint4* src = reinterpret_cast<const uint4*>(r.p + (tok0 + t) * r.ts + head * r.hs) + w;
#pragma unroll
    for (int k = 0; k < NG; ++k) v[k] = src[4 * k];
  };

  uint4 next[NG];
  const int mine = tid >> 2;
  load(mine, next);

  if (QUANT) {
    for (int i = warp; i < ntok; i += kInThreads / 32) {
      long long off;
      int tok;
      row_place(a.g, a.bt, tok0 + i, lane, off, tok);
      if (lane == 0) {
        place[i] = off;
        place_tok[i] = tok;
      }
    }
  }
  if (ROPE) {
    for (int i = tid; i < half << a.tok_shift; i += kInThreads) {
      const int t = i / half, p = i - t * half;
      double s = 0., c = 1.;
      if (tok0 + t < a.n_tokens)
        turn_of(__ldg(a.positions + static_cast<size_t>(a.rope.axis[p]) * a.n_tokens + tok0 + t), a.rope.inv_freq[p], c, s);
      turns64[t * turn_stride64(half) + p] = c;
      turns64[t * turn_stride64(half) + half + p] = s;
      turns32[t * turn_stride(half) + p] = static_cast<float>(c);
      turns32[t * turn_stride(half) + half + p] = static_cast<float>(s);
    }
  }
  if (ROPE) __syncthreads();      // without a rotation the places are first needed behind the codes

  for (int rho = mine; rho - mine < total; rho += kInRows) {
    uint4 raw[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) raw[k] = next[k];
    if (rho - mine + kInRows < total) load(rho + kInRows, next);
    int t, head;
    const int kind = find(rho, t, head);
    if (ROPE && __any_sync(0xffffffffu, kind == 0 || kind == 1)) {
      // value rows in the same warp go through it too, as rows without a rotation
      float x[8 * NG];
#pragma unroll
      for (int k = 0; k < NG; ++k) unpack8(raw[k], x + 8 * k);
      const bool query = kind == 0, key = kind == 1;
      const uint16_t* wt = query ? a.qw : a.kw;
      if (__any_sync(0xffffffffu, query)) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * NG; ++i) ss = __fmaf_rn(x[i], x[i], ss);
        ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, 1));
        ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, 2));
        if (query && wt) {
          const float r = rsqrtf(__fmaf_rn(ss, 1.0f / D, a.rope.eps));
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            float wf[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(wt) + 4 * k + w), wf);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[8 * k + i] = __fmul_rn(x[8 * k + i], __fmul_rn(r, wf[i]));
          }
        }
      }
      double r64 = 1.;
      if (__any_sync(0xffffffffu, key) && a.kw) {
        double ss = 0.;
#pragma unroll
        for (int i = 0; i < 8 * NG; ++i) ss = __fma_rn(static_cast<double>(x[i]), static_cast<double>(x[i]), ss);
        ss = __dadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, 1));
        ss = __dadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, 2));
        r64 = rsqrt(__fma_rn(ss, 1.0 / D, static_cast<double>(a.rope.eps)));
      }
      // a channel of the key row times its weight (the i-th of the octet's bf16 weights g): exact in
      // fp32, as both have eight bits, inside its range.  The norm's factor is left for the end.
      auto weighted = [&](float v, const uint4& g, int i) {
        const uint32_t pair = i < 2 ? g.x : i < 4 ? g.y : i < 6 ? g.z : g.w;
        return static_cast<double>(__fmul_rn(v, __uint_as_float((i & 1) ? pair & 0xFFFF0000u : pair << 16)));
      };
      auto weights = [&](int ch) {
        return wt ? __ldg(reinterpret_cast<const uint4*>(wt + ch)) : make_uint4(kOnes, kOnes, kOnes, kOnes);
      };
      const float* cs = turns32 + t * turn_stride(half);
      const double* cs64 = turns64 + t * turn_stride64(half);
      if constexpr (PAIRS == kHalves) {
        if (query) {
#pragma unroll
          for (int k = 0; k < NG / 2; ++k) {
            float c[8], s[8];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
              *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + 32 * k + 8 * w + i);
              *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + half + 32 * k + 8 * w + i);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) turn(x[8 * k + i], x[8 * (k + NG / 2) + i], c[i], s[i]);
          }
        } else if (key) {
#pragma unroll
          for (int k = 0; k < NG / 2; ++k) {
            const int ch = 32 * k + 8 * w;
            const uint4 g = weights(ch), h = weights(ch + D / 2);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const double2 c = *reinterpret_cast<const double2*>(cs64 + ch + i);
              const double2 s = *reinterpret_cast<const double2*>(cs64 + half + ch + i);
              float &p0 = x[8 * k + i], &q0 = x[8 * (k + NG / 2) + i];
              float &p1 = x[8 * k + i + 1], &q1 = x[8 * (k + NG / 2) + i + 1];
              turn64(weighted(p0, g, i), weighted(q0, h, i), c.x, s.x, r64, p0, q0);
              turn64(weighted(p1, g, i + 1), weighted(q1, h, i + 1), c.y, s.y, r64, p1, q1);
            }
          }
        }
      } else if constexpr (PAIRS == kNext) {
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const bool turns = 32 * k + 8 * w < a.rope.rot_dim;
          if (query && turns) {
            float c[4], s[4];
            *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(cs + 16 * k + 4 * w);
            *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(cs + half + 16 * k + 4 * w);
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(x[8 * k + 2 * i], x[8 * k + 2 * i + 1], c[i], s[i]);
          } else if (key) {
            const uint4 g = weights(32 * k + 8 * w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int pair = 16 * k + 4 * w + i;
              float &p = x[8 * k + 2 * i], &q = x[8 * k + 2 * i + 1];
              const double y = weighted(p, g, 2 * i), z = weighted(q, g, 2 * i + 1);
              if (turns) {
                turn64(y, z, cs64[pair], cs64[half + pair], r64, p, q);
              } else {
                p = static_cast<float>(__dmul_rn(y, r64));
                q = static_cast<float>(__dmul_rn(z, r64));
              }
            }
          }
        }
      } else {
        float* row = turns32 + (turn_stride(half) << a.tok_shift) + (warp * 8 + (lane >> 2)) * (D + 4);
        __syncwarp();   // the rows before were read
#pragma unroll
        for (int i = 0; i < 8 * NG; i += 4)
          *reinterpret_cast<float4*>(row + 32 * (i >> 3) + 8 * w + (i & 7)) = *reinterpret_cast<float4*>(x + i);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const int ch = 32 * k + 8 * w;
          const bool turns = ch < a.rope.rot_dim, first = ch < half;
          const int p = first ? ch : ch - half, to = first ? ch + half : ch - half;    // the pair, the partner channel
          if (query && turns) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
              const float4 o = *reinterpret_cast<const float4*>(row + to + i);
              const float4 c = *reinterpret_cast<const float4*>(cs + p + i);
              float4 s = *reinterpret_cast<const float4*>(cs + half + p + i);
              if (first) s = make_float4(-s.x, -s.y, -s.z, -s.w);
              float* y = x + 8 * k + i;
              y[0] = turned(y[0], o.x, c.x, s.x);
              y[1] = turned(y[1], o.y, c.y, s.y);
              y[2] = turned(y[2], o.z, c.z, s.z);
              y[3] = turned(y[3], o.w, c.w, s.w);
            }
          } else if (key) {
            const uint4 g = weights(ch), h = turns ? weights(to) : g;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              double y = weighted(x[8 * k + i], g, i);
              if (turns) {
                const double s = cs64[half + p + i];
                y = turned(y, weighted(row[to + i], h, i), cs64[p + i], first ? -s : s);
              }
              x[8 * k + i] = static_cast<float>(__dmul_rn(y, r64));
            }
          }
        }
      }
      uint4 b[NG];
#pragma unroll
      for (int k = 0; k < NG; ++k) b[k] = pack8(x + 8 * k);
      if ((kind == 0 && (!QUANT || place[t] != -2)) || (!QUANT && kind == 1)) {
        uint16_t* dst = kind == 0 ? a.qo + (tok0 + t) * a.qo_ts + head * a.qo_hs
                                  : a.ko + (tok0 + t) * a.ko_ts + head * a.ko_hs;
#pragma unroll
        for (int k = 0; k < NG; ++k) reinterpret_cast<uint4*>(dst)[4 * k + w] = b[k];
      }
      if (QUANT) {   // keys enter the cache as the bf16 row a separate call would write
#pragma unroll
        for (int k = 0; k < NG; ++k) raw[k] = b[k];
      }
    }
    if constexpr (QUANT) {
      if (ROPE && !__any_sync(0xffffffffu, kind > 0)) continue;
      float mn[NG], mx[NG];
      auto range = [&]() {
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          uint32_t lo = min2_nan(min2_nan(raw[k].x, raw[k].y), min2_nan(raw[k].z, raw[k].w));
          uint32_t hi = max2_nan(max2_nan(raw[k].x, raw[k].y), max2_nan(raw[k].z, raw[k].w));
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            lo = min2_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max2_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
          }
          lo = min2_nan(lo, lo >> 16);      // the pair's, in the low half
          hi = max2_nan(hi, hi >> 16);
          mn[k] = __uint_as_float(lo << 16);
          mx[k] = __uint_as_float(hi << 16);
        }
      };
      range();
      bool odd = false;
#pragma unroll
      for (int k = 0; k < NG; ++k) odd |= !(mn[k] >= -kLimit && mx[k] <= kLimit);
      if (__any_sync(0xffffffffu, odd)) {   // a NaN or a number past the limit: taken inside
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          float y[8];
          unpack8(raw[k], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] == y[i] ? fminf(fmaxf(y[i], -kLimit), kLimit) : 0.f;
          raw[k] = pack8(y);                // exact: the limit is a bf16
        }
        range();
      }
      // lane w works out the scale, zero and reciprocal of group w (of w % 2 with two groups)
      const int own = w & (NG - 1);
      float lo = mn[0], hi = mx[0];
#pragma unroll
      for (int k = 1; k < NG; ++k) {
        lo = own == k ? mn[k] : lo;
        hi = own == k ? mx[k] : hi;
      }
      const QParams qp = quant_params(lo, hi, 4);
      const uint32_t sz_own = static_cast<uint32_t>(qp.s16) | (static_cast<uint32_t>(qp.z16) << 16);
      const float inv_own = qp.s != 0.f ? __frcp_rn(qp.s) : 0.f;      // 0 makes every code 0
      // the codes of a group lie between those of its ends, which the rounding of s and z can push
      // out of [0, 15]
      const float2 ends = lanes_of(code_sum(both(lo, hi), both(-qp.z, -qp.z), both(-qp.s, -qp.s), both(inv_own, inv_own)));
      const bool in_range = __float_as_uint(ends.x) >= 0x4B400000u && __float_as_uint(ends.y) <= 0x4B40000Fu;
      const bool plain = __all_sync(0xffffffffu, in_range);
      uint32_t code[NG], sz[NG];
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        sz[k] = __shfl_sync(0xffffffffu, sz_own, k, 4);
        const float inv = __shfl_sync(0xffffffffu, inv_own, k, 4);
        code[k] = codes_of(raw[k], sz[k], inv, plain);
      }
      if (!ROPE && rho == mine) __syncthreads();      // every thread's first row
      if (kind > 0 && place[t] >= 0) {
        const int tok = place_tok[t];
        uint8_t* blk = a.g.pages + place[t] + static_cast<size_t>(head) * ((1 << (a.g.page_shift - 4)) * block_bytes(D)) +
                       (kind == 2 ? 10 * D : 0);
        uint8_t* row = blk + tok * (D / 2);
        if (kind == 1) {
          put_words<NG>(row + w * (4 * NG), code);
        } else {
          uint32_t p[NG];
          to_pieces<NG>(code, p);
          put_words<NG>(row + value_place<D>(tok, 2 * w) * (2 * NG), p);
        }
        if (w == 0) put_words<NG>(blk + 8 * D + tok * (4 * NG), sz);
        if (odd) raise(a.g.error, PNMIX_DEVERR_NONFINITE);
      }
    }
  }
}

struct OutArgs {
  Geo g;
  Batch bt;
  int tok_shift, rows_y;   // log2 of the CTA's tokens; head rows (k and v) per CTA in y
  uint16_t* k;
  uint16_t* v;
  long long k_ts, k_hs, v_ts, v_hs;
};

template <int D>
__global__ void __launch_bounds__(kOutThreads)
rows_out_kernel(const __grid_constant__ OutArgs a) {
  constexpr int NG = D / 32, kAhead = 2;
  __shared__ long long place[kMaxTok];
  __shared__ int place_tok[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, w = lane & 3;
  const int ntok = 1 << a.tok_shift, tok0 = blockIdx.x << a.tok_shift;
  const int row0 = blockIdx.y * a.rows_y, rows = min(a.rows_y, 2 * a.g.Hkv - row0);
  const int total = rows << a.tok_shift;
  for (int i = warp; i < ntok; i += kOutThreads / 32) {
    long long off;
    int tok;
    row_place(a.g, a.bt, tok0 + i, lane, off, tok);
    if (lane == 0) {
      place[i] = off;
      place_tok[i] = tok;
    }
  }
  __syncthreads();
  const size_t head_bytes = static_cast<size_t>(1 << (a.g.page_shift - 4)) * block_bytes(D);
  for (int rho0 = tid >> 2; rho0 < total; rho0 += kAhead * kOutRows) {
    uint32_t code[kAhead][NG], sz[kAhead][NG];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int rho = rho0 + u * kOutRows, t = rho & (ntok - 1), r = row0 + (rho >> a.tok_shift);
#pragma unroll
      for (int k = 0; k < NG; ++k) code[u][k] = sz[u][k] = 0u;
      if (rho < total && place[t] >= 0) {
        const int tok = place_tok[t];
        const uint8_t* blk = a.g.pages + place[t] + (r >> 1) * head_bytes + ((r & 1) ? 10 * D : 0);
        const uint8_t* row = blk + tok * (D / 2);
        get_words<NG>((r & 1) ? row + value_place<D>(tok, 2 * w) * (2 * NG) : row + w * (4 * NG), code[u]);
        get_words<NG>(blk + 8 * D + tok * (4 * NG), sz[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int rho = rho0 + u * kOutRows, t = rho & (ntok - 1), r = row0 + (rho >> a.tok_shift);
      if (rho >= total || place[t] == -2) continue;
      if (r & 1) {
        uint32_t c[NG];
        from_pieces<NG>(code[u], c);
#pragma unroll
        for (int k = 0; k < NG; ++k) code[u][k] = c[k];
      }
      const int head = r >> 1;
      uint16_t* dst = (r & 1) ? a.v + (tok0 + t) * a.v_ts + head * a.v_hs : a.k + (tok0 + t) * a.k_ts + head * a.k_hs;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(sz[u][k] & 0xFFFFu)));
        const float z = __half2float(__ushort_as_half(static_cast<uint16_t>(sz[u][k] >> 16)));
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // channels i and i + 4: 1024 + c is an fp16 with c in its low mantissa bits
          const uint32_t pair = ((code[u][k] >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
          __half2 h;
          memcpy(&h, &pair, 4);
          const float2 c = __half22float2(__hsub2(h, __float2half2_rn(1024.f)));
          x[i] = fmaf(c.x, s, z);       // c * s is exact
          x[i + 4] = fmaf(c.y, s, z);
        }
        reinterpret_cast<uint4*>(dst)[4 * k + w] = pack8(x);
      }
    }
  }
}

// Tokens per CTA at most (log2; neighbours in the cache are written by one warp), fewer while
// the grid would not fill the GPU.  Measured at 16384 tokens with 1, 2, 4 and 8 tokens: norm and
// rotation of 40 heads, then all in fp32, -, 59, 61 and 72 us; the write of 16 rows a token (and its read-back) -,
// 55, 54 and 55 us.
int token_shift(int n_tokens, int most) {
  int s = most;
  while (s > 0 && (n_tokens >> s) < 4 * kSms) --s;
  return s;
}

template <int D, bool ROPE, bool QUANT, int PAIRS>
cudaError_t launch_pairs(const IoArgs& a, cudaStream_t s) {
  const int ctas = (a.n_tokens + (1 << a.tok_shift) - 1) >> a.tok_shift;
  const int half = a.rope.rot_dim >> 1;
  size_t bytes = 0;
  if (ROPE)
    bytes += (turn_stride64(half) * sizeof(double) + turn_stride(half) * sizeof(float)) << a.tok_shift;
  if (ROPE && PAIRS == kAnywhere) bytes += kInRows * (D + 4) * sizeof(float);
  rows_in_kernel<D, ROPE, QUANT, PAIRS><<<ctas, kInThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <int D, bool ROPE, bool QUANT>
cudaError_t launch_in(IoArgs& a, cudaStream_t s) {
  a.tok_shift = token_shift(a.n_tokens, ROPE ? 1 : 2);
  if constexpr (!ROPE) {
    return launch_pairs<D, ROPE, QUANT, kHalves>(a, s);
  } else {
    if (a.rope.interleaved) return launch_pairs<D, ROPE, QUANT, kNext>(a, s);
    if (a.rope.rot_dim == D) return launch_pairs<D, ROPE, QUANT, kHalves>(a, s);
    return launch_pairs<D, ROPE, QUANT, kAnywhere>(a, s);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const pnmix_rope& rope, int n_tokens, int nq, int nk, const pnmix_rows& q,
                             const pnmix_rows& k, const uint16_t* qw, const uint16_t* kw, const int32_t* positions,
                             const pnmix_rows& qo, const pnmix_rows& ko, cudaStream_t s) {
  IoArgs a{};
  a.rope = rope;
  a.n_tokens = n_tokens;
  a.nq = nq;
  a.nk = nk;
  a.q = {q.data, q.token_stride, q.head_stride};
  a.k = {k.data, k.token_stride, k.head_stride};
  a.qo = qo.data;
  a.qo_ts = qo.token_stride;
  a.qo_hs = qo.head_stride;
  a.ko = ko.data;
  a.ko_ts = ko.token_stride;
  a.ko_hs = ko.head_stride;
  a.qw = qw;
  a.kw = kw;
  a.positions = positions;
  switch (rope.head_dim) {
    case 64: return launch_in<64, true, false>(a, s);
    case 128: return launch_in<128, true, false>(a, s);
    default: return launch_in<256, true, false>(a, s);
  }
}

cudaError_t launch_append(const Geo& g, const Batch& bt, const pnmix_rows& k, const pnmix_rows& v, cudaStream_t s) {
  IoArgs a{};
  a.g = g;
  a.bt = bt;
  a.n_tokens = bt.n_tokens;
  a.nk = a.nv = g.Hkv;
  a.k = {k.data, k.token_stride, k.head_stride};
  a.v = {v.data, v.token_stride, v.head_stride};
  return g.D == 64 ? launch_in<64, false, true>(a, s) : launch_in<128, false, true>(a, s);
}

cudaError_t launch_append_qkv(const Geo& g, const Batch& bt, const pnmix_rope& rope, const pnmix_rows& q,
                              const pnmix_rows& k, const pnmix_rows& v, const uint16_t* qw, const uint16_t* kw,
                              const int32_t* positions, const pnmix_rows& qo, cudaStream_t s) {
  IoArgs a{};
  a.g = g;
  a.bt = bt;
  a.rope = rope;
  a.n_tokens = bt.n_tokens;
  a.nq = g.Hq;
  a.nk = a.nv = g.Hkv;
  a.q = {q.data, q.token_stride, q.head_stride};
  a.k = {k.data, k.token_stride, k.head_stride};
  a.v = {v.data, v.token_stride, v.head_stride};
  a.qo = qo.data;
  a.qo_ts = qo.token_stride;
  a.qo_hs = qo.head_stride;
  a.qw = qw;
  a.kw = kw;
  a.positions = positions;
  return g.D == 64 ? launch_in<64, true, true>(a, s) : launch_in<128, true, true>(a, s);
}

cudaError_t launch_read(const Geo& g, const Batch& bt, const pnmix_rows& k, const pnmix_rows& v, cudaStream_t s) {
  OutArgs a{};
  a.g = g;
  a.bt = bt;
  a.k = k.data;
  a.k_ts = k.token_stride;
  a.k_hs = k.head_stride;
  a.v = v.data;
  a.v_ts = v.token_stride;
  a.v_hs = v.head_stride;
  // tokens inner: the rows of a block lie together; few tokens leave room for more CTAs in y
  a.tok_shift = 4;
  while (a.tok_shift > 0 && (bt.n_tokens >> a.tok_shift) < kSms) --a.tok_shift;
  const int x = (bt.n_tokens + (1 << a.tok_shift) - 1) >> a.tok_shift, rows = 2 * g.Hkv;
  a.rows_y = max(1, 2 * kOutRows >> a.tok_shift);
  while (a.rows_y < rows && static_cast<long long>(x) * ((rows + a.rows_y - 1) / a.rows_y) > kSms * 16) a.rows_y *= 2;
  const dim3 grid(x, (rows + a.rows_y - 1) / a.rows_y);
  if (g.D == 64)
    rows_out_kernel<64><<<grid, kOutThreads, 0, s>>>(a);
  else
    rows_out_kernel<128><<<grid, kOutThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace pnmix
