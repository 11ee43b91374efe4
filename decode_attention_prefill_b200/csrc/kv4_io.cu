// kv4_io.cu -- rows in and out of the 4-bit paged cache: per-head norm and rotation of
// queries and keys, the quantised write (alone or fused behind the rotation) and the
// read-back.  One kernel for the first two, one for the last.
//
// All three move bytes: a bf16 row of 128 channels is 256 bytes and its packed form 80, the
// arithmetic is a few tens of instructions per 8 channels, so device memory bounds long
// inputs and latency the decode step.  A head's row is held by D / 8 lanes, 8 channels (one
// 16-byte load) each: the norm's sum, the group's minimum and maximum and the rotation's
// partner channels are shuffles inside the row, and nothing but the angles passes through
// shared memory.  A CTA takes a few tokens and all their heads, so a token's angles (fp64
// product, reduced to a turn, one sincospi per pair) and its place in the cache are worked
// out once per CTA, while the first rows' loads are in flight.
#include "kv4.cuh"
#include "kv4_launch.cuh"

namespace pnmix {
namespace kv4 {
namespace {

constexpr int kIoThreads = 256;
constexpr int kMaxTok = 16;       // tokens per CTA at most
constexpr int kAhead = 4;         // rows a lane group loads before it works on the first

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

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    memcpy(&w[i], &h, 4);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Between lanes l and l ^ 4 (neighbouring channel groups of a row): a lane's eight codes
// (its low half one value piece, its high half the next) against the stored words, which
// hold one piece of both groups.  The exchange is its own inverse.
__device__ __forceinline__ uint32_t cross_groups(uint32_t w, bool odd) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? (w & 0xFFFFu) : (w >> 16), 4);
  return odd ? (other | (w & 0xFFFF0000u)) : ((w & 0xFFFFu) | (other << 16));
}

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

// L: lanes of a row (head_dim / 8).  ROPE: q and k rows are normed and rotated.  QUANT: k and
// v rows go to the cache (otherwise k rows are stored like q's).
template <int L, bool ROPE, bool QUANT>
__global__ void __launch_bounds__(kIoThreads)
rows_in_kernel(const __grid_constant__ IoArgs a) {
  constexpr int D = 8 * L, kRows = kIoThreads / L, kGroups = D / 32;
  extern __shared__ float turn[];             // [token][cos, sin][rot / 2]
  __shared__ long long place[kMaxTok];
  __shared__ int place_tok[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid & (L - 1);
  const int ntok = 1 << a.tok_shift, tok0 = blockIdx.x << a.tok_shift;
  const int total = (a.nq + a.nk + a.nv) << a.tok_shift;   // rows of this CTA, tokens inner
  const int half = a.rope.rot_dim >> 1;

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
  auto load = [&](int rho) {
    int t, head;
    const int kind = find(rho, t, head);
    if (kind < 0) return make_uint4(0u, 0u, 0u, 0u);
    const Rows& r = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    return *(reinterpret_cast<const uint4*>(r.p + (tok0 + t) * r.ts + head * r.hs) + l);
  };

  uint4 buf[kAhead];
  const int mine = tid / L;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) buf[u] = load(u * kRows + mine);

  if (QUANT) {
    for (int i = warp; i < ntok; i += kIoThreads / 32) {
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
    for (int i = tid; i < half << a.tok_shift; i += kIoThreads) {
      const int t = i / half, p = i - t * half;
      float s = 0.f, c = 1.f;
      if (tok0 + t < a.n_tokens) {
        // angle in turns: the fp64 product of a 31-bit and a 24-bit number is off by 2^-53 of
        // itself, 2^-31 of a turn at a million turns; reduced to [-1/2, 1/2] before it is
        // rounded to fp32
        const int pos = __ldg(a.positions + static_cast<size_t>(a.rope.axis[p]) * a.n_tokens + tok0 + t);
        double turns = static_cast<double>(pos) * static_cast<double>(a.rope.inv_freq[p]) * 0.15915494309189533577;
        turns -= rint(turns);
        sincospif(2.f * static_cast<float>(turns), &s, &c);
      }
      turn[(2 * t) * half + p] = c;
      turn[(2 * t + 1) * half + p] = s;
    }
  }
  __syncthreads();

  for (int rho0 = mine; rho0 - mine < total; rho0 += kAhead * kRows) {
    if (rho0 != mine) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) buf[u] = load(rho0 + u * kRows);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (rho0 - mine + u * kRows >= total) break;   // the same for the whole CTA
      int t, head;
      const int kind = find(rho0 + u * kRows, t, head);
      float x[8];
      unpack8(buf[u], x);
      if (ROPE) {   // every lane takes part in the shuffles; value rows keep x
        float y[8];
        const uint16_t* w = kind == 0 ? a.qw : a.kw;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (w && kind >= 0 && kind < 2) {
          const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.rope.eps);
          float wf[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(w) + l), wf);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i] * r * wf[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i];
        }
        const float* cs = turn + (2 * t) * half;
        if (a.rope.interleaved) {
          if (8 * l < a.rope.rot_dim) {
            const float4 c = *reinterpret_cast<const float4*>(cs + 4 * l);
            const float4 s = *reinterpret_cast<const float4*>(cs + half + 4 * l);
            const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = y[2 * i], q = y[2 * i + 1];
              y[2 * i] = p * cc[i] - q * sn[i];
              y[2 * i + 1] = q * cc[i] + p * sn[i];
            }
          }
        } else {
          const int hl = half >> 3;   // lanes of a row's first half
          const bool first = l < hl, turned = l < 2 * hl;
          const int base = first ? l : l - hl;
          const int src = turned ? (first ? l + hl : l - hl) : l;
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, y[i], src, L);
          if (turned) {
            const float4 c0 = *reinterpret_cast<const float4*>(cs + 8 * base);
            const float4 c1 = *reinterpret_cast<const float4*>(cs + 8 * base + 4);
            const float4 s0 = *reinterpret_cast<const float4*>(cs + half + 8 * base);
            const float4 s1 = *reinterpret_cast<const float4*>(cs + half + 8 * base + 4);
            const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = first ? y[i] * cc[i] - o[i] * sn[i] : y[i] * cc[i] + o[i] * sn[i];
          }
        }
        if (kind >= 0 && kind < 2) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = y[i];
        }
        if (kind == 0 && (!QUANT || place[t] != -2))
          *(reinterpret_cast<uint4*>(a.qo + (tok0 + t) * a.qo_ts + head * a.qo_hs) + l) = pack8(x);
        if (!QUANT && kind == 1)
          *(reinterpret_cast<uint4*>(a.ko + (tok0 + t) * a.ko_ts + head * a.ko_hs) + l) = pack8(x);
        if (QUANT) unpack8(pack8(x), x);   // keys enter the cache as the bf16 row a separate call would write
      }
      if constexpr (QUANT) {
        bool odd_number = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          odd_number |= !(fabsf(x[i]) <= kLimit);
          x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -kLimit), kLimit) : 0.f;
        }
        float mn = x[0], mx = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          mn = fminf(mn, x[i]);
          mx = fmaxf(mx, x[i]);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        const QParams qp = quant_params(mn, mx, 4);
        uint32_t w = 0u;
        if (qp.s != 0.f) {
          const float inv = __frcp_rn(qp.s);
#pragma unroll
          for (int i = 0; i < 8; ++i) w |= quant_code_rcp(x[i], qp.z, qp.s, inv, 15) << (4 * i);
        }
        const int grp = l >> 2, piece = l & 3;
        const uint32_t crossed = cross_groups(w, grp & 1);
        if (kind > 0 && place[t] >= 0) {
          const int tok = place_tok[t];
          uint8_t* blk = a.g.pages + place[t] + static_cast<size_t>(head) * ((1 << (a.g.page_shift - 4)) * block_bytes(D)) +
                         (kind == 2 ? 10 * D : 0);
          uint8_t* row = blk + tok * (D / 2);
          if (kind == 1)
            *reinterpret_cast<uint32_t*>(row + piece * (4 * kGroups) + grp * 4) = w;
          else
            *reinterpret_cast<uint32_t*>(row + value_place<D>(tok, 2 * piece + (grp & 1)) * (2 * kGroups) +
                                         (grp >> 1) * 4) = crossed;
          if (piece == 0)
            *reinterpret_cast<uint32_t*>(blk + 8 * D + tok * (4 * kGroups) + grp * 4) =
                static_cast<uint32_t>(qp.s16) | (static_cast<uint32_t>(qp.z16) << 16);
          if (odd_number) raise(a.g.error, PNMIX_DEVERR_NONFINITE);
        }
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

template <int L>
__global__ void __launch_bounds__(kIoThreads)
rows_out_kernel(const __grid_constant__ OutArgs a) {
  constexpr int D = 8 * L, kRows = kIoThreads / L, kGroups = D / 32;
  __shared__ long long place[kMaxTok];
  __shared__ int place_tok[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid & (L - 1);
  const int ntok = 1 << a.tok_shift, tok0 = blockIdx.x << a.tok_shift;
  const int row0 = blockIdx.y * a.rows_y, rows = min(a.rows_y, 2 * a.g.Hkv - row0);
  const int total = rows << a.tok_shift;
  for (int i = warp; i < ntok; i += kIoThreads / 32) {
    long long off;
    int tok;
    row_place(a.g, a.bt, tok0 + i, lane, off, tok);
    if (lane == 0) {
      place[i] = off;
      place_tok[i] = tok;
    }
  }
  __syncthreads();
  const int grp = l >> 2, piece = l & 3;
  const size_t head_bytes = static_cast<size_t>(1 << (a.g.page_shift - 4)) * block_bytes(D);
  for (int rho0 = tid / L; rho0 - static_cast<int>(tid / L) < total; rho0 += kAhead * kRows) {
    uint32_t w[kAhead], sz[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int rho = rho0 + u * kRows, t = rho & (ntok - 1), r = row0 + (rho >> a.tok_shift);
      w[u] = sz[u] = 0u;
      if (rho < total && place[t] >= 0) {
        const int tok = place_tok[t], head = r >> 1;
        const uint8_t* blk = a.g.pages + place[t] + head * head_bytes + ((r & 1) ? 10 * D : 0);
        const uint8_t* row = blk + tok * (D / 2);
        w[u] = *reinterpret_cast<const uint32_t*>(
            (r & 1) ? row + value_place<D>(tok, 2 * piece + (grp & 1)) * (2 * kGroups) + (grp >> 1) * 4
                    : row + piece * (4 * kGroups) + grp * 4);
        sz[u] = *reinterpret_cast<const uint32_t*>(blk + 8 * D + tok * (4 * kGroups) + grp * 4);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int rho = rho0 + u * kRows, t = rho & (ntok - 1), r = row0 + (rho >> a.tok_shift);
      const uint32_t crossed = cross_groups(w[u], grp & 1);   // every lane takes part
      if (rho >= total || place[t] == -2) continue;
      const uint32_t c = (r & 1) ? crossed : w[u];
      const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(sz[u] & 0xFFFFu)));
      const float z = __half2float(__ushort_as_half(static_cast<uint16_t>(sz[u] >> 16)));
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(static_cast<float>((c >> (4 * i)) & 15u), s, z);   // c * s is exact
      const int head = r >> 1;
      uint16_t* dst = (r & 1) ? a.v + (tok0 + t) * a.v_ts + head * a.v_hs : a.k + (tok0 + t) * a.k_ts + head * a.k_hs;
      *(reinterpret_cast<uint4*>(dst) + l) = pack8(x);
    }
  }
}

// Tokens per CTA: enough that a CTA's rows keep its loads busy, few enough that the grid
// covers the GPU (8 CTAs of 256 threads fit an SM).
int token_shift(int n_tokens, int rows, int most) {
  int s = 0;
  while (s < most && (rows << s) < 64 && (n_tokens >> (s + 1)) >= 2 * 148) ++s;
  return s;
}

template <int L, bool ROPE, bool QUANT>
cudaError_t launch_in(IoArgs& a, cudaStream_t s) {
  a.tok_shift = token_shift(a.n_tokens, a.nq + a.nk + a.nv, 4);
  const int ctas = (a.n_tokens + (1 << a.tok_shift) - 1) >> a.tok_shift;
  const size_t smem = ROPE ? sizeof(float) * a.rope.rot_dim << a.tok_shift : 0;
  rows_in_kernel<L, ROPE, QUANT><<<ctas, kIoThreads, smem, s>>>(a);
  return cudaGetLastError();
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
    case 64: return launch_in<8, true, false>(a, s);
    case 128: return launch_in<16, true, false>(a, s);
    default: return launch_in<32, true, false>(a, s);
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
  return g.D == 64 ? launch_in<8, false, true>(a, s) : launch_in<16, false, true>(a, s);
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
  return g.D == 64 ? launch_in<8, true, true>(a, s) : launch_in<16, true, true>(a, s);
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
  while (a.tok_shift > 0 && (bt.n_tokens >> a.tok_shift) < 148) --a.tok_shift;
  const int x = (bt.n_tokens + (1 << a.tok_shift) - 1) >> a.tok_shift;
  const int rows = 2 * g.Hkv, per_pass = kIoThreads / (g.D / 8) * kAhead;   // rows of one round of loads
  a.rows_y = max(1, per_pass >> a.tok_shift);
  while (a.rows_y < rows && static_cast<long long>(x) * ((rows + a.rows_y - 1) / a.rows_y) > 148 * 16) a.rows_y *= 2;
  const dim3 grid(x, (rows + a.rows_y - 1) / a.rows_y);
  if (g.D == 64)
    rows_out_kernel<8><<<grid, kIoThreads, 0, s>>>(a);
  else
    rows_out_kernel<16><<<grid, kIoThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace pnmix
