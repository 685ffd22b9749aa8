// Device helpers of the MX element formats (blocks of 32 values that share a
// power-of-two scale) and of lane exchanges, shared by the MX kernels.
#pragma once
#include "common.h"

namespace moe {

constexpr int kE4M3 = 1, kE2M1 = 2;  // MOE_MX_*

// The exponent p of a block's scale: the smallest p >= -126 with m <= M * 2^p,
// from the bits of m = the block's largest magnitude.  M = 1.75 * 2^8 (e4m3) or
// 1.5 * 2^2 (e2m1): m = f * 2^q with 1 <= f < 2 needs p = q - 8 (or q - 2), one
// more if f > 1.75 (or 1.5).
template <int FMT>
__device__ __forceinline__ int mx_exponent(uint32_t mbits) {
  const int q = (int)(mbits >> 23) - 127;
  const bool over = (mbits & 0x7FFFFFu) > (FMT == kE4M3 ? 0x600000u : 0x400000u);
  const int p = q - (FMT == kE4M3 ? 8 : 2) + (over ? 1 : 0);
  return p < -126 ? -126 : p;
}
__device__ __forceinline__ bool mx_not_finite(uint32_t mbits) { return mbits >= 0x7F800000u; }
// 2^-p for -126 <= p <= 126
__device__ __forceinline__ float mx_inverse(int p) { return __builtin_bit_cast(float, (uint32_t)(127 - p) << 23); }

// Four values, already divided by the scale, to their codes: 4 bytes of e4m3,
// or 2 bytes of e2m1 (the first value in the low nibble).  The conversions
// round to nearest even; with mx_exponent's scale nothing exceeds the largest
// element, so their saturation is never reached.
__device__ __forceinline__ uint32_t mx_pack4_e4m3(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return (uint32_t)v;
}
__device__ __forceinline__ uint32_t mx_pack4_e2m1(float a, float b, float c, float d) {
  uint32_t v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, 1.0f, 0);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, c, d, 1.0f, 1);
  return v;
}

// max over the 4 lanes of a quad (DPP quad permutes: no LDS traffic)
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  return v > b ? v : b;
}

}  // namespace moe
