// kv4_softmax.cuh -- where a row's softmax reference stands in the attention over the 4-bit paged
// cache, and how it moves.  Plain arithmetic that compiles for the host too, where it is tested.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define PNMIX_BOTH __host__ __device__ __forceinline__
#else
#define PNMIX_BOTH inline
#endif

namespace pnmix {
namespace kv4 {

// A weight of a raw logit x of a row with factor fac (to the log2 domain) is 2^e with
// e = fl((x - base) fac - ref), one fma behind the difference.  base is 0 while the scaled logits are
// moderate: then fl(mx fac) is within 2^-5 of the largest one, so a reference made from it bounds
// the weights.  From 2^20 on the spacing of fp32 makes such a reference useless (at 2^28 it is 32,
// and e may be 16 for the maximum itself), so the row's largest raw logit is taken away first: e is
// then at most -ref by its sign alone, whatever the size of the logits.
//
// A move leaves the largest of the tile's weights at 2^5 to 2^6.  Weights become fp16, whose step is
// 2^-24 at the least, so each is off by 2^-11 of itself or 2^-30 of the row's largest.  (With the
// largest at 1, the first form, 2^-25 of it: a first token 2^21 times as strong as each of 30000 others
// cost their sum 6 %.)  More room below leaves less above before the reference has to move again, and
// each move reads O and writes it: 2 x 1024 tokens over 8192 cached ones, logits of a few outlier
// channels, with 3, 4, 6 and 9 here 312, 314, 322 and 355 us (9 and a maximum over 32 columns instead
// of the tile's rest: 415; all with moves from a sum of 2^15 on, at 65504 6 takes 319).
constexpr float kRoom = 6.f;
constexpr float kFarLogit = 1048576.f;
constexpr float kFirstReference = -3.4e38f;   // lower than any logit: the first one moves it

struct RowRef {
  float base, ref;
};

// The reference after a move to the largest raw logit mx: no weight is above 2^(kRoom + 2^-5).
PNMIX_BOTH RowRef move_reference(const RowRef& old, float mx, float fac) {
  const float t = mx * fac;
  if (old.base == 0.f && fabsf(t) < kFarLogit) return {0.f, ceilf(t) - kRoom};
  return {mx, -kRoom};
}

// log2 of what the row's sums so far are multiplied by in that move.
PNMIX_BOTH float move_exponent(const RowRef& old, const RowRef& now, float fac) {
  return fmaf(old.base - now.base, fac, old.ref - now.ref);
}

// The reference in the log2 domain, for joining partial sums of a row.
PNMIX_BOTH float reference_of(const RowRef& r, float fac) { return fmaf(r.base, fac, r.ref); }

// The row kernel takes logits that are scaled already (fac 1) and weights their value scale as well:
// 2^((x - base) - ref) times it stays within fp16.  Its reference after a move: base from the largest
// logit mx and the largest m of logit + log2 of the token's value scale (within 2^-4 of the exact one
// below 2^20), then ref from that m with base taken away, so no product is above 2^(8 + 2^-4).
PNMIX_BOTH float row_base(float base, float mx, float m) { return base == 0.f && fabsf(m) < kFarLogit ? 0.f : mx; }
PNMIX_BOTH float row_reference(float m) { return ceilf(m) - 8.f; }

}  // namespace kv4
}  // namespace pnmix
