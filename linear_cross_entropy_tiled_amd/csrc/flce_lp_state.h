// The running base-2 softmax state of a row (flce_logprobs.hip has the formulas).
#pragma once

#include "flce_device.h"
#include "flce_mx.h"

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

// tanh(w), for the softcap z = cap tanh(v / cap).  Up to |w| = 0.8 (logits up to two
// thirds of the cap) w + w^3 p(w^2), p of degree 6: with its coefficients rounded to fp32
// 7.5e-9 off tanh, as evaluated in fp32 about 1e-7 of it.  1 - 2 / (e^2w + 1) is off by 1e-7
// of 1 there, and the logit by 1e-7 of the cap, however small it is (at a cap of 1000 the
// log-probabilities of 1000 x 32000 were 7e-6 off, 15 to 80 times elementary torch's error).
// The eight multiply-adds cost what the exponential and the reciprocal do.
// WIDE, for a wave that holds a larger w somewhere: the formula for those and only those,
// so that no value depends on its neighbours.
constexpr float kTanhNear = 0.8f;
template <bool WIDE> __device__ __forceinline__ float tanh_of(float w) {
  const float t = w * w;
  float p = fmaf(t, -0.0005726429517380893f, 0.002854352118447423f);
  p = fmaf(t, p, -0.008510654792189598f);
  p = fmaf(t, p, 0.02177303470671177f);
  p = fmaf(t, p, -0.0539538599550724f);
  p = fmaf(t, p, 0.133332297205925f);
  p = fmaf(t, p, -0.3333333134651184f);
  p = fmaf(w * t, p, w);
  if constexpr (WIDE) {
    const float far = fmaf(-2.0f, fast_rcp(fast_exp2(2.0f * kLog2e * w) + 1.0f), 1.0f);
    p = fabsf(w) > kTanhNear ? far : p;
  }
  return p;
}

// The same with the slope, 1 - tanh^2.  Where tanh comes near 1 that would lose its digits,
// and 4 r (1 - r) of r = 1 / (e^2w + 1) does not.
template <bool WIDE> __device__ __forceinline__ float tanh_of(float w, float* slope) {
  float th = tanh_of<false>(w);
  *slope = fmaf(-th, th, 1.0f);
  if (WIDE && fabsf(w) > kTanhNear) {
    const float r = fast_rcp(fast_exp2(2.0f * kLog2e * w) + 1.0f);
    th = fmaf(-2.0f, r, 1.0f);
    *slope = 4.0f * fmaf(-r, r, r);
  }
  return th;
}

// Four at a time, the formula only where some lane of the wave needs it.
__device__ __forceinline__ void tanh4(const float (&w)[4], float (&th)[4]) {
  float size = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; r++) {
    th[r] = tanh_of<false>(w[r]);
    size = fmaxf(size, fabsf(w[r]));
  }
  if (__builtin_amdgcn_ballot_w64(size > kTanhNear)) {
#pragma unroll
    for (int r = 0; r < 4; r++) th[r] = tanh_of<true>(w[r]);
  }
}
__device__ __forceinline__ void tanh4(const float (&w)[4], float (&th)[4], float (&slope)[4]) {
  float size = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; r++) {
    th[r] = tanh_of<false>(w[r], &slope[r]);
    size = fmaxf(size, fabsf(w[r]));
  }
  if (__builtin_amdgcn_ballot_w64(size > kTanhNear)) {
#pragma unroll
    for (int r = 0; r < 4; r++) th[r] = tanh_of<true>(w[r], &slope[r]);
  }
}

template <typename T> struct BiasOf { typedef T type; };
template <> struct BiasOf<int8_t> { typedef float type; };
template <> struct BiasOf<mx4> { typedef float type; };

}  // namespace flce
