// gfx950 kernels of linear layers in 8-bit floating point: weights into e4m3 with
// one power of two per block of 128 x 128, and the product of such a weight with an
// e4m3 checkpoint, y = x W^T, or with W transposed dx = dy W.
//
// The weight is kept in both orientations, so both products read their operands
// along K. Scales are powers of two, which the 8-bit MFMA applies by itself. 8192 x
// 25600 x 5120 976 us either way (2200 TFLOP/s), 1024 x 8192 x 5120 57 (1500), in tiles of
// 128 x 128.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "product.h"

namespace muon {

template <class Z>
__global__ void __launch_bounds__(Z::NT, Z::WG) linear8_kernel(PrArgs) {
  __shared__ __align__(1024) unsigned char smem[Z::LDS];
  pr_run<Z, PrStoreOut>(smem);
}

__global__ void __launch_bounds__(256) linear8_join_kernel(PrArgs, int edge) { pr_join_of<PrStoreOut>(edge); }

template <int MODE>
static hipError_t launch_tiles(const PrArgs& args, hipStream_t s) {
  typedef PrCfg<256, 256, 128, 2, MODE, 1> Large;
  typedef PrCfg<128, 128, 128, 2, MODE, 2> Medium;
  typedef PrCfg<64, 64, 128, 4, MODE, 2> Small;
  const dim3 block(256);
  if (args.tile == kPrLarge) {
    if constexpr (MODE == kNT8) hipLaunchKernelGGL(linear8_kernel<Large>, dim3(pr_grid<Large>(args)), block, 0, s, args);
    else return hipErrorInvalidValue;  // not chosen for fp32
  } else if (args.tile == kPrMedium) hipLaunchKernelGGL(linear8_kernel<Medium>, dim3(pr_grid<Medium>(args)), block, 0, s, args);
  else hipLaunchKernelGGL(linear8_kernel<Small>, dim3(pr_grid<Small>(args)), block, 0, s, args);
  const hipError_t e = hipGetLastError();
  const int64_t join = pr_join_blocks(args, false);
  if (e != hipSuccess || join == 0) return e;
  hipLaunchKernelGGL(linear8_join_kernel, dim3((uint32_t)join), dim3(256), 0, s, args, kPrEdge[args.tile]);
  return hipGetLastError();
}

hipError_t launch_linear8(const PrArgs& args, hipStream_t s) {
  return args.f32 ? launch_tiles<kNT8X>(args, s) : launch_tiles<kNT8>(args, s);
}

// ------------------------------------------------------------ weights

// One 128 x 128 block per workgroup: thread t holds columns 8 (t % 16) .. +7 of rows
// t / 16 + 16 i, the block's largest magnitude is one reduction over the workgroup,
// and the transposed bytes leave through LDS. Bound by memory: every element is
// read once and written twice, a byte each (8192 x 5120 bf16 35.6 us, 4.7 TB/s).
constexpr int kW8Row = kBlock + 4;  // LDS row of the transposing copy: rows four apart in different banks

template <class T>
__global__ void __launch_bounds__(256) w8_save_kernel(const T* w, int64_t ldw, muon_w8 out) {
  __shared__ uint32_t tops[4];
  __shared__ __align__(16) unsigned char tile[kBlock * kW8Row];
  const int n = (int)out.n, k = (int)out.k, kb = (k + kBlock - 1) / kBlock, bn = blockIdx.x / kb, bk = blockIdx.x - bn * kb;
  const int n0 = bn * kBlock, k0 = bk * kBlock, tid = threadIdx.x, c = tid % 16 * 8, r0 = tid / 16;
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = n0 + r0 + 16 * i;
    load_run(w + (int64_t)min(row, n - 1) * ldw + min(k0 + c, k - 1), row < n ? k - (k0 + c) : 0, v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[i][e]) & 0x7fffffffu);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const bool fine = top < 0x7f800000u;
  const int ex = (int)(top >> 23), man = (int)(top & 0x7fffffu);
  const int E = fine ? max(ex - 8 + (man > 0x600000), kMinExp) : 255;  // 448 = 1.75 * 2^8
  const float inv = __uint_as_float((uint32_t)(254 - min(E, 253)) << 23);
  if (tid == 0) *((g_u8*)(static_cast<uint8_t*>(out.e) + (int64_t)bn * out.lde + bk)) = (uint8_t)E;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u32x2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = __builtin_amdgcn_cvt_pk_fp8_f32(v[i][4 * h] * inv, v[i][4 * h + 1] * inv, 0, false);
      o[h] = fine ? (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[i][4 * h + 2] * inv, v[i][4 * h + 3] * inv, t, true) : 0u;
    }
    const int r = r0 + 16 * i;
    if (n0 + r < n && k0 + c < (k + 15) / 16 * 16)
      *((g_u32x2*)(static_cast<uint8_t*>(out.q) + (int64_t)(n0 + r) * out.ldq + k0 + c)) = o;
    if (out.qt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) *reinterpret_cast<uint32_t*>(tile + r * kW8Row + c + 4 * h) = o[h];
    }
  }
  if (!out.qt) return;
  __syncthreads();
  // row of the transposed block: k index; a thread gathers 8 rows of one column
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int kk = r0 + 16 * i, rr = c;  // column kk of the block, its rows rr .. rr+7
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e >> 2] |= (uint32_t)tile[(rr + e) * kW8Row + kk] << (8 * (e & 3));
    if (k0 + kk < k && n0 + rr < (n + 15) / 16 * 16)
      *((g_u32x2*)(static_cast<uint8_t*>(out.qt) + (int64_t)(k0 + kk) * out.ldqt + n0 + rr)) = u32x2{o[0], o[1]};
  }
}

template <class T>
__global__ void __launch_bounds__(256) w8_load_kernel(muon_w8 in, T* w, int64_t ldw) {
  const int64_t runs = (in.k + 7) / 8, count = runs * in.n;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / runs, col = (i - row * runs) * 8;
    const u32x2 q = *((const g_u32x2*)(static_cast<const uint8_t*>(in.q) + row * in.ldq + col));
    const uint32_t E = *((const g_u8*)(static_cast<const uint8_t*>(in.e) + row / kBlock * in.lde + col / kBlock));
    float v[8];
    q8_decode(q, E, MUON_Q8_E4M3, v);
    store_run(w + row * ldw + col, (int)min((int64_t)8, in.k - col), v);
  }
}

hipError_t launch_w8_save(const void* w, int64_t ldw, int dtype, const muon_w8& out, hipStream_t s) {
  const dim3 grid((uint32_t)((out.k + kBlock - 1) / kBlock * ((out.n + kBlock - 1) / kBlock)));
  if (dtype == MUON_BF16) hipLaunchKernelGGL(w8_save_kernel<u16>, grid, dim3(256), 0, s, static_cast<const u16*>(w), ldw, out);
  else hipLaunchKernelGGL(w8_save_kernel<float>, grid, dim3(256), 0, s, static_cast<const float*>(w), ldw, out);
  return hipGetLastError();
}

hipError_t launch_w8_load(const muon_w8& in, void* w, int64_t ldw, int dtype, hipStream_t s) {
  const int64_t count = (in.k + 7) / 8 * in.n;
  const dim3 grid((uint32_t)((count + 255) / 256 < 16384 ? (count + 255) / 256 : 16384));
  if (dtype == MUON_BF16) hipLaunchKernelGGL(w8_load_kernel<u16>, grid, dim3(256), 0, s, in, static_cast<u16*>(w), ldw);
  else hipLaunchKernelGGL(w8_load_kernel<float>, grid, dim3(256), 0, s, in, static_cast<float*>(w), ldw);
  return hipGetLastError();
}

}  // namespace muon
