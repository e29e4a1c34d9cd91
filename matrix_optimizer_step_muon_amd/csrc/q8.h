// The 8-bit checkpoint format on the device (see muon.h): encoding and decoding
// eight elements.
#pragma once

#include "device.h"
#include "layer_internal.h"

namespace muon {

typedef uint8_t __attribute__((address_space(1))) g_u8;

// max over the four lanes of a group
MUON_INLINE uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));  // lanes 1 0 3 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));  // lanes 2 3 0 1
}

// The eight bytes of v and the exponent byte of the group whose other elements
// sit in the same quad of lanes. Magnitudes are compared as integers, which
// orders floats and puts infinities and NaNs above all numbers. The scale is a
// power of two, so v / 2^(E-127) is exact and rounding happens once: for int8
// in the addition of 1.5 * 2^23 (its low byte is then the two's complement
// integer nearest to the quotient, ties to even), for e4m3 in the conversion.
MUON_INLINE uint32_t q8_encode(const float v[8], int kind, u32x2& w) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = quad_max(top);
  const bool fine = top < 0x7f800000u;
  // 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8
  const int ex = (int)(top >> 23), man = (int)(top & 0x7fffffu);
  int E = kind == MUON_Q8_INT8 ? ex - 6 + (man > 0x7e0000) : ex - 8 + (man > 0x600000);
  E = fine ? max(E, kMinExp) : 255;
  const float inv = __uint_as_float((uint32_t)(254 - min(E, 253)) << 23);
  uint32_t o[2];
  if (kind == MUON_Q8_INT8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(v[4 * h + i], inv, 12582912.f));
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
      o[h] = lo | hi;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int t = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
      o[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, t, true);
    }
  }
  w[0] = fine ? o[0] : 0u;
  w[1] = fine ? o[1] : 0u;
  return (uint32_t)E;
}

// 2^(E-127); NaN for E = 255.
MUON_INLINE float q8_unit(uint32_t E) { return __uint_as_float(E == 255u ? 0x7fc00000u : E << 23); }

MUON_INLINE void q8_decode4(uint32_t w, float unit, int kind, float v[4]) {
  if (kind == MUON_Q8_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i)) * unit;
  } else {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = a[0] * unit; v[1] = a[1] * unit; v[2] = b[0] * unit; v[3] = b[1] * unit;
  }
}

MUON_INLINE void q8_decode(u32x2 w, uint32_t E, int kind, float v[8]) {
  const float unit = q8_unit(E);
  q8_decode4(w[0], unit, kind, v);
  q8_decode4(w[1], unit, kind, v + 4);
}

// Four bytes as packed bf16, for an exponent byte that several of them share;
// `live` false gives zeros. Both ways are exact, since q has at most 8
// significant bits and the unit is a power of two.
// int8: bytes with the sign bit flipped are put behind 0x64, which makes the
// fp16 numbers 1024 + 128 + q; times the unit minus 1152 units is the value
// (one mixed-precision fma per element, two instructions per element in all).
// From E = kQ8WideExp on, 1152 units are past the largest fp32 number: there the
// caller takes q8_bf16x4_wide instead, or its results in place of these.
// e4m3: the converting instruction scales by the unit itself (three
// instructions per four elements); q is replaced by NaN codes for E = 255.
constexpr uint32_t kQ8WideExp = 245;

template <int KIND>
struct Q8Group {
  float unit, bias;
  uint32_t keep, set;
  MUON_INLINE Q8Group(uint32_t E, bool live) {
    if constexpr (KIND == MUON_Q8_INT8) {
      unit = live ? q8_unit(E) : 0.f;
      bias = -1152.f * unit;
    } else {
      unit = __uint_as_float(E << 23);
      keep = live ? ~0u : 0u;
      set = live && E == 255u ? 0x7f7f7f7fu : 0u;
    }
  }
  MUON_INLINE u32x2 bf16x4(uint32_t w) const {
    u32x2 o;
    if constexpr (KIND == MUON_Q8_INT8) {
      typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
      const uint32_t t = w ^ 0x80808080u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f16x2 f = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, t, h ? 0x04030402u : 0x04010400u));
        o[h] = pack_bf16x2(fmaf((float)f[0], unit, bias), fmaf((float)f[1], unit, bias));
      }
    } else {
      const int t = (int)((w & keep) | set);
      o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(t, unit, false));
      o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(t, unit, true));
    }
    return o;
  }
};

// The same of int8 bytes for every exponent byte (255: NaN), an instruction more
// per element.
MUON_INLINE u32x2 q8_bf16x4_wide(uint32_t w, uint32_t E, bool live) {
  float v[4];
  q8_decode4(w, live ? q8_unit(E) : 0.f, MUON_Q8_INT8, v);
  return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

}  // namespace muon
