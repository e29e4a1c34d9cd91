// The arithmetic of the gated feed-forward block's elements on the device: activations
// and their derivatives, and the three bf16 parts of an fp32 number.
#pragma once

#include "device.h"
#include "muon.h"

namespace muon {

// Eight fp32 numbers as bf16 operands that add up to them: x = hi + mid + lo, each the
// rest rounded toward zero (24 bits of numbers of at least 2^-110); `parts` are the
// eight lo, mid and hi. A part of which nothing is left is 2^-64 of x in place of 0: less
// than a sum in fp32 sees, but an infinity in the other operand keeps its sign in that
// product too, where 0 would make it a NaN. All parts of an infinity are that infinity,
// and one of a NaN's at least is a NaN.
MUON_INLINE void cut3(const float v[8], u32x4 parts[3]) {
  uint32_t p[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    auto cut = [](float f) __attribute__((always_inline)) { return __uint_as_float(__float_as_uint(f) & 0xffff0000u); };
    // The maxima are the rest itself where there is one, 2^-23 of x at least; of the NaN
    // that an infinity leaves, and a number, they are the number.
    const float x = v[i], least = fabsf(x * 0x1p-64f), r = x - cut(x);
    const float mid = copysignf(fmaxf(fabsf(r), least), x), rest = r - cut(mid);
    p[2][i] = __float_as_uint(x);
    p[1][i] = __float_as_uint(mid);
    p[0][i] = __float_as_uint(copysignf(fmaxf(fabsf(rest), least), x));
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) parts[q][i] = __builtin_amdgcn_perm(p[q][2 * i + 1], p[q][2 * i], 0x07060302u);  // the upper halves
}

// An fp32 number as two bf16 ones that add up to 16 bits of it, with the same care for
// infinities in the other operand.
MUON_INLINE void cut2(float x, u16& hi, u16& lo) {
  const float most = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  hi = (u16)(__float_as_uint(x) >> 16);
  lo = f32_to_bf16(copysignf(fmaxf(fabsf(x - most), fabsf(x * 0x1p-64f)), x));
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
      // Phi from its smaller side: (1 + erf) / 2 would keep nothing of it from a = -5 on.
      // Below 2^-110 (a < -12.1) it is 0: its products would underflow in part.
      const float a = v[i], near = 0.5f * erfcf(fabsf(a) * 0.70710678f), tail = near < 0x1p-110f ? 0.f : near;
      const float phi = a < 0.f ? tail : 1.f - tail;
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
