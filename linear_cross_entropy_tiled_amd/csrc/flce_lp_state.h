// The running base-2 softmax state of a row (flce_logprobs.hip has the formulas).
#pragma once

#include "flce_device.h"

namespace flce {

// A row's state over some of its logits.  With nothing seen: m = kMasked, l = T = 0.
struct LpState {
  float m, l, T, yt;
};

__device__ __forceinline__ void lp_merge(LpState& a, const LpState& b) {
  const float mn = fmaxf(a.m, b.m);
  // a state without any finite logit (l = 0) may have m = -inf or kMasked: its shift
  // is not used, so that 0 times it is no NaN
  const float da = a.l == 0.0f ? 0.0f : a.m - mn, db = b.l == 0.0f ? 0.0f : b.m - mn;
  const float fa = fast_exp2(da), fb = fast_exp2(db);
  a.T = fmaf(da, a.l, a.T) * fa + fmaf(db, b.l, b.T) * fb;
  a.l = a.l * fa + b.l * fb;
  a.m = mn;
  a.yt = fmaxf(a.yt, b.yt);
}

template <typename T> struct BiasOf { typedef T type; };
template <> struct BiasOf<int8_t> { typedef float type; };

}  // namespace flce
