// Device helpers shared by the gfx950 kernels: element access, direct
// global -> LDS copies with explicit waits, and the transposing LDS read.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

typedef uint16_t u16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------ element access
//
// Every global access goes through an address_space(1) pointer, so it
// compiles to global_load / global_store. Generic (flat) accesses would also
// count against the LDS wait counter and serialise the GEMM pipeline.

#define MUON_INLINE __device__ __forceinline__ __attribute__((always_inline))

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((address_space(1))) g_u32x4;
typedef u32x2 __attribute__((address_space(1))) g_u32x2;
typedef f32x4 __attribute__((address_space(1))) g_f32x4;
typedef u16 __attribute__((address_space(1))) g_u16;
typedef float __attribute__((address_space(1))) g_f32;

MUON_INLINE u32x4 gload16(const void* p) { return *((const g_u32x4*)(p)); }

// 16 bytes at any element's address: one instruction too, which the hardware
// takes apart where it has to.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x4_any __attribute__((address_space(1))) g_u32x4_any;
MUON_INLINE u32x4 gload16_any(const void* p) { return *((const g_u32x4_any*)(p)); }
MUON_INLINE void gstore16_any(void* p, u32x4 v) { *((g_u32x4_any*)(p)) = v; }

MUON_INLINE float bf16_to_f32(u16 v) { return __uint_as_float((uint32_t)v << 16); }

// fp32 -> bf16 with gfx950's v_cvt_pk_bf16_f32: rounds to nearest even under
// the default rounding mode, and a NaN stays a quiet NaN.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
MUON_INLINE u16 f32_to_bf16(float f) { return __builtin_bit_cast(u16, (__bf16)f); }
MUON_INLINE uint32_t pack_bf16x2(float lo, float hi) {
  const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

template <class T> struct Elem;
template <> struct Elem<float> {
  static MUON_INLINE float load(const float* p) { return *((const g_f32*)(p)); }
  static MUON_INLINE void store(float* p, float v) { *((g_f32*)(p)) = v; }
  static MUON_INLINE float lds_load(const float* p) { return *p; }
  static MUON_INLINE float round(float v) { return v; }
  static MUON_INLINE float to_storage(float v) { return v; }
};
template <> struct Elem<u16> {
  static MUON_INLINE float load(const u16* p) { return bf16_to_f32(*((const g_u16*)(p))); }
  static MUON_INLINE void store(u16* p, float v) { *((g_u16*)(p)) = f32_to_bf16(v); }
  static MUON_INLINE float lds_load(const u16* p) { return bf16_to_f32(*p); }
  static MUON_INLINE float round(float v) { return bf16_to_f32(f32_to_bf16(v)); }
  static MUON_INLINE u16 to_storage(float v) { return f32_to_bf16(v); }
};

// Four consecutive elements, as one 8-byte (bf16) or 16-byte (fp32) access.
template <class T> struct Vec4;
template <> struct Vec4<float> {
  static MUON_INLINE void load(const float* p, float v[4]) {
    f32x4 t = *((const g_f32x4*)(p));
    v[0] = t[0]; v[1] = t[1]; v[2] = t[2]; v[3] = t[3];
  }
  static MUON_INLINE void store(float* p, const float v[4]) {
    f32x4 t = {v[0], v[1], v[2], v[3]};
    *((g_f32x4*)(p)) = t;
  }
};
template <> struct Vec4<u16> {
  static MUON_INLINE void load(const u16* p, float v[4]) {
    u32x2 t = *((const g_u32x2*)(p));
    v[0] = __uint_as_float(t[0] << 16); v[1] = __uint_as_float(t[0] & 0xffff0000u);
    v[2] = __uint_as_float(t[1] << 16); v[3] = __uint_as_float(t[1] & 0xffff0000u);
  }
  static MUON_INLINE void store(u16* p, const float v[4]) {
    u32x2 t;
    t[0] = pack_bf16x2(v[0], v[1]);
    t[1] = pack_bf16x2(v[2], v[3]);
    *((g_u32x2*)(p)) = t;
  }
};

// ------------------------------------------------------------ LDS access

// Direct global -> LDS copy of 16 bytes per lane (global_load_lds_dwordx4).
// Lane l's bytes land at LDS address lds + 16*l, so one wave instruction
// fills 1 KB of LDS. It is issued from inline asm, with M0 saved and restored
// around it. The compiler then does not track these loads, and would not put a
// conservative vmcnt(0) in front of every LDS read. The engine waits for them
// itself, with the exact counts of its ring of stages. Untracked loads can
// only make the compiler's own vmcnt waits stricter, never looser.
MUON_INLINE void dma16(const void* g, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "global_load_lds_dwordx4 %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(g), "s"(lds)
      : "memory");
}

template <int N>
MUON_INLINE void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Q operand stored K-major (QK engines): LDS rows are K indices of 256 bf16
// (512 bytes, 32 slots). The slot of chunk c of row k is c ^ swzk(k), which
// keeps the transposing fragment reads below free of bank conflicts for 32-
// and 64-bank LDS. It depends only on k % 4.
MUON_INLINE int lds_swizzle_k(int k) { return ((k & 1) ? 4 : 0) ^ ((k & 2) ? 10 : 0); }

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));

// ds_read_b64_tr_b16: within each group of 16 lanes, lane i receives element
// i % 4 of the 4 x 16-bit values at the address of lane 4e + i/4, for
// e = 0..3. If lane j of the group points at row k0 + j/4, columns
// n0 + 4(j%4) .. +3 of a K-major tile, lane i gets column n0 + i at rows
// k0 .. k0+3: the B-operand fragment layout of the MFMA.
MUON_INLINE v4i16 lds_read_tr(const unsigned char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4i16*)(const_cast<unsigned char*>(p)));
}

// Between lanes of one wave that hand each other data through LDS: what is
// written before is there for every lane's reads after it, and what is read
// before is not overwritten. The hardware keeps a wave's LDS accesses in order,
// so this is no instruction; it holds the compiler, which sees one lane's
// addresses only and may reorder those that differ.
MUON_INLINE void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Direct global -> LDS copy of 16 bytes per lane, addressed as a uniform
// 64-bit base plus a per-lane 32-bit byte offset (the saddr form of
// global_load_lds_dwordx4). Same M0 handling as dma16.
MUON_INLINE void dma16s(const void* base_, uint32_t voff, uint32_t lds) {
  // The base must live in SGPRs; read it from the first lane (it is
  // uniform). readfirstlane returns int: each half goes through uint32_t so
  // that the low half is zero-extended, not sign-extended, into 64 bits.
  const uint64_t b = (uint64_t)(uintptr_t)base_;
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint64_t base = ((uint64_t)hi << 32) | (uint64_t)lo;
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(voff), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds))
      : "memory");
}

// threadIdx.x behind an empty asm: address arithmetic derived from it stays
// where it is written. Without this the compiler hoists per-lane offsets (of
// the engines' fragment reads and DMA, and of the epilogues) out of the
// persistent tile loop as loop invariants, keeps dozens of them live across
// the GEMM, spills them, and reloads them one by one.
MUON_INLINE int fresh_tid() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

}  // namespace muon
