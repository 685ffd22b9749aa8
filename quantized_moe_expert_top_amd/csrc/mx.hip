// MX rows: quantisation, its inverse, and the residual RMS norm that writes
// them.  All three are one pass over memory; what bounds them is HBM.
//
// A block of 32 values belongs to 4 neighbouring lanes with 8 values each (one
// 16-byte load of a 16-bit type per lane, a wavefront reads 1 KB in a row); its
// largest magnitude is a maximum over the lane's 8 bit patterns and two DPP
// quad permutes.  Magnitudes are compared as integers: that orders them like
// the numbers and keeps infinities and NaN on top, where a float maximum would
// drop a NaN.
#include "mx.h"

namespace moe {

namespace {
constexpr int kThreads = 256;
constexpr int kUnroll = kQuantUnroll;
template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void quantize_mx_kernel(const void* __restrict__ x, size_t n8,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  quantize_block<DT, FMT, kThreads>(x, n8, codes, scales, blockIdx.x);
}

template <int DT>
__device__ __forceinline__ void store8(void* out, size_t i8, const float v[8]) {
  u32x4* p = static_cast<u32x4*>(out) + i8 * (DT == 1 ? 2 : 1);
  u32x4 o;
  if constexpr (DT == 1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = v[4 * h + i];
        o[i] = __builtin_bit_cast(uint32_t, f);
      }
      p[h] = o;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = DT == 0 ? pack_bf16x2(v[2 * i], v[2 * i + 1])
                     : pack_f16x2(v[2 * i], v[2 * i + 1]);
    p[0] = o;
  }
}

// Bound by HBM: 57344 rows of 4096 e2m1 to bf16 100 us, 5.9 TB/s read and written.
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int FMT, int DT>
__global__ __launch_bounds__(kThreads) void dequantize_mx_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales, size_t n8,
                                                                 void* __restrict__ out) {
  const size_t base = (size_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  uint32_t lo[kUnroll], hi[kUnroll], sb[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const size_t i8 = base + j * kThreads;
    lo[j] = hi[j] = sb[j] = 0;
    if (i8 < n8) {
      if constexpr (FMT == kE4M3) {
        const u32x2 c = reinterpret_cast<const u32x2*>(codes)[i8];
        lo[j] = c[0];
        hi[j] = c[1];
      } else {
        lo[j] = reinterpret_cast<const uint32_t*>(codes)[i8];
      }
      sb[j] = scales[i8 >> 2];
    }
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const size_t i8 = base + j * kThreads;
    if (i8 >= n8) continue;
    f32x2 e[4];
    if constexpr (FMT == kE4M3) {
      e[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo[j], false);
      e[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo[j], true);
      e[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi[j], false);
      e[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi[j], true);
    } else {
      e[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[j], 1.0f, 0);
      e[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[j], 1.0f, 1);
      e[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[j], 1.0f, 2);
      e[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[j], 1.0f, 3);
    }
    // byte 0 is 2^-127 (subnormal), 255 is not a number
    const uint32_t sbits = sb[j] == 0 ? 0x00400000u : sb[j] == 255 ? 0x7FC00000u : sb[j] << 23;
    const float s = __builtin_bit_cast(float, sbits);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = e[i][0] * s;
      v[2 * i + 1] = e[i][1] * s;
    }
    store8<DT>(out, i8, v);
  }
}

// ------------------------------------------------------------------- RMS norm
// TPR threads hold one row in registers (NV groups of 8 values each), so x and
// residual are read once: v = x + residual rounded to the row's type, the sum
// of squares in float64 (squares and their sum neither overflow nor lose small
// rows there), then n = v * weight * factor in float64 too: the product of two
// floats is exact in it, while in fp32 it can leave the range on either side
// although n does not, and the factor alone can.  n is rounded to nearest for an
// fp32 y; what is rounded again, to 16 bits or to an MX element, is rounded to odd
// first (an inexact n gets an odd last bit), so that the second rounding is that of
// the exact value and not of an fp32 number on the border.  Past the largest float
// n is infinite.  HBM bounds it: 8192 rows of 4096 with residual, sum, y and 8-bit
// blocks 54 us in bf16, 109 in fp32 (n in fp32 pairs, which is wrong at the ends of
// the range: 52.5 and 110; 16384 rows of 512 16.4 and 14.7, 64 rows of 4096 3.8 both).
template <int DT>
__device__ __forceinline__ float round_to(float f) {
  if constexpr (DT == 0) return bf16_to_f32(f32_to_bf16(f));
  if constexpr (DT == 2) return f16_to_f32(f32_to_f16(f));
  return f;
}

template <int DT, int FMT, int TPR, int NV>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void rmsnorm_mx_kernel(NormArgs a) {
#pragma clang fp contract(off)  // sums are rounded before they are rounded to 16 bits; rest is that of the rounded d
  constexpr int kRows = TPR > kThreads ? 1 : kThreads / TPR, kWaves = TPR / 64;
  __shared__ double part[kRows * kWaves];
  const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const size_t row = (size_t)blockIdx.x * kRows + sub;
  const bool live = row < (size_t)a.rows;
  const int n8 = a.H >> 3;
  const size_t r8 = row * n8;
  float v[NV][8];
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * TPR;
    const bool on = live && c < n8;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    if (on) {
      unpack8<DT>(load8<DT>(a.x, r8 + c), v[j]);
      if (a.residual) {
        float q[8];
        unpack8<DT>(load8<DT>(a.residual, r8 + c), q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = round_to<DT>(v[j][i] + q[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[j][i], (double)v[j][i], sum);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if constexpr (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += part[sub * kWaves + w];
  }
  const double f = 1.0 / sqrt(sum / a.H + (double)a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * TPR;
    if (!(live && c < n8)) continue;
    if (a.sum) store8<DT>(a.sum, r8 + c, v[j]);
    float w[8], nearest[8];
    unpack8<DT>(load8<DT>(a.weight, c), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = (double)v[j][i] * (double)w[i] * f + 0.0;  // (a zero is +0)
      const float n = (float)d;
      const double rest = __builtin_fabs(d) - __builtin_fabs((double)n);
      nearest[i] = n;
      // the neighbour on the side of the rest (infinities and NaN stay)
      const int b = __builtin_bit_cast(int, n), odd = b + (rest > 0.0 ? 1 : -1);
      v[j][i] = (__builtin_isfinite(rest) && rest != 0.0 && !(b & 1)) ? __builtin_bit_cast(float, odd) : n;
    }
    if (a.y) store8<DT>(a.y, r8 + c, DT == 1 ? nearest : v[j]);
    if constexpr (FMT != 0) store_mx8<FMT>(v[j], quad_umax(absmax_bits(v[j])), r8 + c, a.codes, a.scales);
  }
}

// ------------------------------------------------------------------- repack
// One thread per 16-byte lane record of the tiled codes, resp. per 4-byte lane
// record of the tiled scales.  K is padded to whole chunks of 256 with zeros
// under the scale 2^0.
__global__ __launch_bounds__(kThreads) void mx_repack_codes_kernel(const uint8_t* __restrict__ src, size_t n, int K,
                                                                   uint8_t* __restrict__ dst) {
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const int lane = (int)(i & 63);
  const size_t tk = i >> 6;  // (e, tile, step)
  const int steps = (K + 255) >> 8 << 2;
  const size_t row = tk / steps * 32 + (lane & 31);
  const size_t k0 = tk % steps * 64 + 32 * (lane >> 5);
  reinterpret_cast<u32x4*>(dst)[i] =
      k0 < (size_t)K ? *reinterpret_cast<const u32x4*>(src + row * (size_t)(K >> 1) + (k0 >> 1)) : u32x4{};
}
__global__ __launch_bounds__(kThreads) void mx_repack_scales_kernel(const uint8_t* __restrict__ src, size_t n, int K,
                                                                    uint8_t* __restrict__ dst) {
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const int lane = (int)(i & 63);
  const int chunks = (K + 255) >> 8, nb = K >> 5;
  const size_t row = (i >> 6) / chunks * 32 + (lane & 31);
  const int b0 = (int)((i >> 6) % chunks) * 8 + (lane >> 5);
  uint32_t v = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int b = b0 + 2 * s;
    v |= (uint32_t)(b < nb ? src[row * nb + b] : 127) << (8 * s);
  }
  reinterpret_cast<uint32_t*>(dst)[i] = v;
}

inline unsigned blocks_for(size_t n, size_t per) { return (unsigned)((n + per - 1) / per); }

template <int DT, int FMT>
void norm_rows(const NormArgs& a, hipStream_t s) {
  // Threads per row: the whole workgroup for a wide row (8 values per thread
  // and step), one wavefront for narrow ones.  Few rows leave the chip empty and
  // wait for one row's chain of additions: 8 values per thread.  Rows of 4096 /
  // 8192 bf16 in us, with more threads / fewer: 3.4 / 4.0 and 4.5 / 5.9 (64 rows),
  // 5.1 / 5.2 and 8.3 / 8.3 (512), 13.9 / 13.1 and 24.1 / 20.6 (2048); rows of
  // 16384 6.3 / 9.8 (64), 39.0 / 37.9 (2048), 161 / 182 (8192).
  const bool few = a.rows <= 512;
#define MOE_NORM(TPR, NV)                                                                                  \
  hipLaunchKernelGGL((rmsnorm_mx_kernel<DT, FMT, TPR, NV>),                                                \
                     dim3(blocks_for(a.rows, TPR > kThreads ? 1 : kThreads / TPR)),                        \
                     dim3(TPR > kThreads ? TPR : kThreads), 0, s, a)
  if (a.H <= 512) MOE_NORM(64, 1);
  else if (a.H <= 2048) MOE_NORM(256, 1);
  else if (a.H <= 4096 && few) MOE_NORM(512, 1);
  else if (a.H <= 4096) MOE_NORM(256, 2);
  else if (a.H <= 8192 && few) MOE_NORM(1024, 1);
  else if (a.H <= 8192) MOE_NORM(256, 4);
  else MOE_NORM(1024, 2);
#undef MOE_NORM
}
template <int DT>
void norm_fmt(const NormArgs& a, hipStream_t s) {
  if (a.fmt == kE4M3) norm_rows<DT, kE4M3>(a, s);
  else if (a.fmt == kE2M1) norm_rows<DT, kE2M1>(a, s);
  else norm_rows<DT, 0>(a, s);
}
}  // namespace

int launch_quantize_mx(const void* x, int x_dtype, int64_t rows, int K, int fmt, uint8_t* codes, uint8_t* scales,
                       void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t n8 = (size_t)rows * K / 8;
  const dim3 grid(blocks_for(n8, kThreads * kUnroll)), block(kThreads);
#define MOE_Q(DT)                                                                                              \
  if (fmt == kE4M3) hipLaunchKernelGGL((quantize_mx_kernel<DT, kE4M3>), grid, block, 0, s, x, n8, codes, scales); \
  else hipLaunchKernelGGL((quantize_mx_kernel<DT, kE2M1>), grid, block, 0, s, x, n8, codes, scales)
  if (x_dtype == 0) { MOE_Q(0); }
  else if (x_dtype == 1) { MOE_Q(1); }
  else { MOE_Q(2); }
#undef MOE_Q
  return (int)hipGetLastError();
}

int launch_dequantize_mx(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, int fmt, int out_dtype,
                         void* out, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t n8 = (size_t)rows * K / 8;
  const dim3 grid(blocks_for(n8, kThreads * kUnroll)), block(kThreads);
#define MOE_DQ(DT)                                                                                                \
  if (fmt == kE4M3) hipLaunchKernelGGL((dequantize_mx_kernel<kE4M3, DT>), grid, block, 0, s, codes, scales, n8, out); \
  else hipLaunchKernelGGL((dequantize_mx_kernel<kE2M1, DT>), grid, block, 0, s, codes, scales, n8, out)
  if (out_dtype == 0) { MOE_DQ(0); }
  else if (out_dtype == 1) { MOE_DQ(1); }
  else { MOE_DQ(2); }
#undef MOE_DQ
  return (int)hipGetLastError();
}

int launch_rmsnorm_mx(const NormArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.dtype == 0) norm_fmt<0>(a, s);
  else if (a.dtype == 1) norm_fmt<1>(a, s);
  else norm_fmt<2>(a, s);
  return (int)hipGetLastError();
}

int launch_mx_repack(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* tcodes,
                     uint8_t* tscales, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t tiles = (size_t)E * (N / 32);
  const size_t nc = tiles * ((K + 255) / 256) * 256, ns = tiles * ((K + 255) / 256) * 64;
  hipLaunchKernelGGL(mx_repack_codes_kernel, dim3(blocks_for(nc, kThreads)), dim3(kThreads), 0, s, codes, nc, K, tcodes);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return (int)e;
  hipLaunchKernelGGL(mx_repack_scales_kernel, dim3(blocks_for(ns, kThreads)), dim3(kThreads), 0, s, scales, ns, K, tscales);
  return (int)hipGetLastError();
}

}  // namespace moe
