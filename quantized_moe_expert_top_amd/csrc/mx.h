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
// 2^p for -126 <= p <= 126
__device__ __forceinline__ float mx_scale(int p) { return __builtin_bit_cast(float, (uint32_t)(p + 127) << 23); }

// Four values over the scale (a power of two: exact) to their codes: 4 bytes of
// e4m3, or 2 bytes of e2m1 (the first value in the low nibble).  The conversions
// round to nearest even; with mx_exponent's scale nothing exceeds the largest
// element, so their saturation is never reached.
template <int FMT>
__device__ __forceinline__ uint32_t mx_pack4(float a, float b, float c, float d, float scale) {
  if constexpr (FMT == kE4M3) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    s16x2 v = {0, 0};
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, a, b, scale, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, c, d, scale, true);
    return __builtin_bit_cast(uint32_t, v);
  } else {
    uint32_t v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, scale, 0);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, c, d, scale, 1);
  }
}

// Bits of the largest magnitude of n values; a NaN among them stays (IEEE
// maximum, two values per instruction).
template <int N>
__device__ __forceinline__ uint32_t absmax_bits(const float (&v)[N]) {
  float m = __builtin_fabsf(v[0]);
#pragma unroll
  for (int i = 1; i + 1 < N; i += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(v[i]), __builtin_fabsf(v[i + 1])), m);
  if (N % 2 == 0) m = __builtin_elementwise_maximum(__builtin_fabsf(v[N - 1]), m);
  return __builtin_bit_cast(uint32_t, m) & 0x7FFFFFFFu;
}

// fp16 pair, rounded to nearest even
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

// max over the 4 lanes of a quad (DPP quad permutes: no LDS traffic)
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  return v > b ? v : b;
}

// --------------------------------------------------------------- quantisation
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// 8 consecutive values as they are stored: 16 bytes (16-bit types) or 32.
template <int DT>
struct Raw8 {
  u32x4 d[DT == 1 ? 2 : 1];
};
// ONCE: data that nothing reads again (a streaming load)
template <int DT, bool ONCE = false>
__device__ __forceinline__ Raw8<DT> load8(const void* x, size_t i8) {
  Raw8<DT> r;
  const u32x4* p = static_cast<const u32x4*>(x) + i8 * (DT == 1 ? 2 : 1);
  r.d[0] = ONCE ? __builtin_nontemporal_load(p) : p[0];
  if constexpr (DT == 1) r.d[1] = ONCE ? __builtin_nontemporal_load(p + 1) : p[1];
  return r;
}
template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT>& r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = r.d[0][i];
    if constexpr (DT == 0) {
      v[2 * i] = bf16_lo(w);
      v[2 * i + 1] = bf16_hi(w);
    } else if constexpr (DT == 2) {
      v[2 * i] = f16_to_f32((uint16_t)(w & 0xFFFFu));
      v[2 * i + 1] = f16_to_f32((uint16_t)(w >> 16));
    } else {
      const uint32_t w1 = r.d[1][i];
      v[i] = __builtin_bit_cast(float, w);
      v[4 + i] = __builtin_bit_cast(float, w1);
    }
  }
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t pk_umax16(uint32_t a, uint32_t b) {
  const u16x2 m = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
  return __builtin_bit_cast(uint32_t, m);
}
// fp32 bits of the largest magnitude of the lane's 8 values
template <int DT>
__device__ __forceinline__ uint32_t absmax8(const Raw8<DT>& r) {
  if constexpr (DT == 1) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = r.d[0][i], b = r.d[1][i];
      m = umax(m, umax(a & 0x7FFFFFFFu, b & 0x7FFFFFFFu));
    }
    return m;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = r.d[0][i];
      m = pk_umax16(m, a & 0x7FFF7FFFu);
    }
    m = umax(m & 0xFFFFu, m >> 16);
    return DT == 0 ? m << 16 : __builtin_bit_cast(uint32_t, f16_to_f32((uint16_t)m));
  }
}
// Quantises the lane's 8 values (group i8 of the flat array) given its block's
// largest magnitude; the quad's first lane writes the scale byte.
template <int FMT>
__device__ __forceinline__ void store_mx8(const float (&v)[8], uint32_t mbits, size_t i8, uint8_t* __restrict__ codes,
                                          uint8_t* __restrict__ scales) {
  const int p = mx_exponent<FMT>(mbits);
  const bool bad = mx_not_finite(mbits);
  const float scale = mx_scale(p);
  const uint32_t lo = mx_pack4<FMT>(v[0], v[1], v[2], v[3], scale), hi = mx_pack4<FMT>(v[4], v[5], v[6], v[7], scale);
  if constexpr (FMT == kE4M3)
    reinterpret_cast<u32x2*>(codes)[i8] = u32x2{bad ? 0u : lo, bad ? 0u : hi};
  else
    reinterpret_cast<uint32_t*>(codes)[i8] = bad ? 0u : lo | (hi << 16);
  if ((threadIdx.x & 3) == 0) scales[i8 >> 2] = bad ? (uint8_t)255 : (uint8_t)(p + 127);
}

// One workgroup's share of a quantisation: NT * kQuantUnroll groups of 8 values,
// of n8 (a multiple of 4, so quads are whole).  All loads are issued before the
// first is used.  Two groups per thread and streaming loads: 16384 x 4096 bf16 to
// e4m3 33.8 us (6.0 TB/s read and written); 1, 4 and 8 groups 36 to 41 us, loads
// kept in the caches 36.4 us.
constexpr int kQuantUnroll = 2;
template <int DT, int FMT, int NT>
__device__ __forceinline__ void quantize_block(const void* __restrict__ x, size_t n8, uint8_t* __restrict__ codes,
                                               uint8_t* __restrict__ scales, size_t block) {
  const size_t base = block * (NT * kQuantUnroll) + threadIdx.x;
  Raw8<DT> r[kQuantUnroll];
#pragma unroll
  for (int j = 0; j < kQuantUnroll; ++j)
    if (base + j * NT < n8) r[j] = load8<DT, true>(x, base + j * NT);
#pragma unroll
  for (int j = 0; j < kQuantUnroll; ++j) {
    const size_t i8 = base + j * NT;
    if (i8 < n8) {
      float v[8];
      unpack8<DT>(r[j], v);
      store_mx8<FMT>(v, quad_umax(absmax8<DT>(r[j])), i8, codes, scales);
    }
  }
}

}  // namespace moe
