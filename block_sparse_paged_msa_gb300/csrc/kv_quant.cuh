// The pools' quantisers, shared by the cache writes: fp32 values to e4m3 codes
// and to NVFP4 codes and scales, every step one IEEE fp32 operation rounded to
// nearest even and every code saturating.  Not part of the ABI.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "msa_device.cuh"

namespace msa {

// Two values -> two e4m3 codes of x / scale (the first in the low byte).
__device__ __forceinline__ uint32_t e4m3x2_of(float a, float b, float scale) {
  const float2 f = make_float2(__fdiv_rn(a, scale), __fdiv_rn(b, scale));
  return (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

// Largest magnitude of eight values (NaN ignored: E2M1 has none).
__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// Eight values of a 16-element block of largest magnitude amax -> four bytes of
// E2M1 pairs (even element in the low nibble), and the block's E4M3 scale code,
// for tensor scale g.  A block whose scale code is 0 stores zero codes.
__device__ __forceinline__ uint32_t nvfp4_codes8(const float (&f)[8], float amax, float g,
                                                 uint8_t& scale) {
  const __nv_fp8_storage_t sc =
      __nv_cvt_float_to_fp8(__fdiv_rn(amax, __fmul_rn(6.f, g)), __NV_SATFINITE, __NV_E4M3);
  scale = (uint8_t)sc;
  const float d = __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(sc, __NV_E4M3))), g);
  if (d == 0.f) return 0u;
  uint32_t codes = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = make_float2(__fdiv_rn(f[2 * i], d), __fdiv_rn(f[2 * i + 1], d));
    codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(u, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  return codes;
}

// Eight bf16 (one 16-byte chunk) -> fp32.
__device__ __forceinline__ void bf16x8_to_f32(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
}

}  // namespace msa
