// The arithmetic of the gated feed-forward block's elements on the device: activations
// and their derivatives, and the three bf16 parts of an fp32 number.
#pragma once

#include "device.h"
#include "muon.h"

namespace muon {

// x = hi + mid + lo, each the rest rounded toward zero to bf16 (24 bits of numbers
// of at least 2^-110). Infinities and NaNs stay in hi alone.
MUON_INLINE void cut3(float x, float& hi, float& mid, float& lo) {
  const uint32_t bits = __float_as_uint(x);
  const bool fine = (bits & 0x7f800000u) != 0x7f800000u;
  hi = fine ? __uint_as_float(bits & 0xffff0000u) : x;
  const float r = fine ? x - hi : 0.f;
  mid = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  lo = __uint_as_float(__float_as_uint(r - mid) & 0xffff0000u);
}

// 1 / (1 + e^-x); e^-x in the hardware's exponential of base 2: a relative error of
// (|x| + 2) 2^-24 or so.
MUON_INLINE float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x)); }

// act(a) and act'(a) of eight values, given to `to` one by one. ACT -1: as act says.
template <int ACT, class F>
MUON_INLINE void activations(const float v[8], int act_, F to) {
  const int act = ACT < 0 ? act_ : ACT;
  if (act == MUON_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(v[i]), f = v[i] * s;
      to(i, f, fmaf(f, 1.f - s, s));
    }
  } else if (act == MUON_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[i], phi = 0.5f + 0.5f * erff(a * 0.70710678f);
      to(i, a * phi, fmaf(a * 0.39894228f, __builtin_amdgcn_exp2f(-0.72134752f * a * a), phi));
    }
  } else if (act == MUON_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = sigmoid(2 u); from |a| = 100 on it is 0 or 1 whatever a^2 is
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[i], a2 = fminf(a * a, 1e4f), s = sigmoid(1.5957691216f * a * fmaf(0.044715f, a2, 1.f)), f = a * s;
      to(i, f, fmaf(f * (1.f - s), 1.5957691216f * fmaf(0.134145f, a2, 1.f), s));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) to(i, v[i] > 0.f ? v[i] : v[i] == v[i] ? 0.f : v[i], v[i] > 0.f ? 1.f : 0.f);  // NaN stays
  }
}

// act(v).
MUON_INLINE float activation(float v, int act) {
  float x[8] = {v, v, v, v, v, v, v, v}, r = 0.f;
  activations<-1>(x, act, [&](int i, float f, float) __attribute__((always_inline)) {
    if (i == 0) r = f;
  });
  return r;
}

}  // namespace muon
