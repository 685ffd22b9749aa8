// Grouped product of MX activation rows with the experts' MX weights (e2m1,
// blocks of 32 along K), on the scaled matrix instructions
// (v_mfma_scale_f32_32x32x64_f8f6f4): they multiply the elements, apply both
// blocks' power-of-two scales and accumulate in fp32.
//
// Operands of one instruction (32 channels x 32 tokens x 64 inputs; weights are
// the A operand, so an accumulator column is a token and a lane holds 16
// channels of one token):
//   lane l: channel / token l % 32, half h = l / 32
//   e2m1    16 bytes: inputs 32h .. 32h + 31
//   e4m3    32 bytes: inputs 16h .. 16h + 15, then 32 + 16h .. 32 + 16h + 15
//   scale   one byte of a register (op_sel): block h (inputs 32h .. 32h + 31)
//   result  register r of lane l: channel 8*(r/4) + 4*h + r%4, token l % 32
// (checked lane by lane against the formula for all four format pairs).
#include "mx.h"

namespace moe {

namespace {
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kEpiBf16 = 0, kEpiSwiglu = 1, kEpiF32 = 2, kEpiF16 = 3, kEpiSwigluE4M3 = 4, kEpiSwigluE2M1 = 5;
constexpr bool is_swiglu(int epi) { return epi == kEpiSwiglu || epi == kEpiSwigluE4M3 || epi == kEpiSwigluE2M1; }

struct MxK {  // kernel arguments
  const uint8_t* wc;
  const uint8_t* wsc;
  int N, K;
  const uint8_t* a;
  const uint8_t* as;
  uint32_t a_bytes, as_bytes;
  int A_rows;
  const int32_t* gather;
  int k;
  const int32_t* seg;
  int E, M_total;
  void* out;
  uint8_t* out_scales;
};

// The 8-register operand: an e2m1 operand fills the first 4.
__device__ __forceinline__ i32x8 operand(u32x4 lo) {
  const i32x4 v = __builtin_bit_cast(i32x4, lo);
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}
__device__ __forceinline__ i32x8 operand(u32x4 lo, u32x4 hi) {
  const i32x4 a = __builtin_bit_cast(i32x4, lo), b = __builtin_bit_cast(i32x4, hi);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// STEP (0, 1): weight scale in byte WB of ws, activation scale in byte 2 * STEP
// of as (shifted by the lane's half beforehand).
template <int AF, int WB, int AB>
__device__ __forceinline__ f32x16 mx_mfma(i32x8 w, i32x8 x, f32x16 c, uint32_t ws, uint32_t as) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 4, AF == kE4M3 ? 0 : 4, WB, (int)ws, AB, (int)as);
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Segment e's rows, clamped to the buffers.
__device__ __forceinline__ void segment(const MxK& p, int e, int& s0, int& s1) {
  s0 = min(max(p.seg[e], 0), p.M_total);
  s1 = min(max(p.seg[e + 1], s0), p.M_total);
}
__device__ __forceinline__ int source_row(const MxK& p, int row) {
  const int r = p.gather ? p.gather[row] / p.k : row;
  return min(max(r, 0), p.A_rows - 1);
}

// -------------------------------------------------------- few rows per expert
// A workgroup takes 64 output channels of one expert (SwiGLU: 32 gate and the
// matching 32 up channels) and the expert's rows, 32 at a time; its NW
// wavefronts split K and add their sums through LDS.  Weights and activations
// go from memory straight to the operand registers: each weight byte is read
// once per 32 rows.
template <int AF>
struct SmallBlock {  // operands of one K block of 128
  u32x4 w[2][2];     // [channel tile][step]
  u32x4 x[2][AF == kE4M3 ? 2 : 1];
  uint32_t ws[2], as;
};

template <int AF, int EPI, int NW>
__global__ __launch_bounds__(64 * NW) void mx_small_kernel(MxK p) {
  constexpr int D = 2;  // K blocks in flight
  __shared__ float red[NW][2][16][64];
  __shared__ uint32_t amx[4][32];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int e = blockIdx.y;
  int s0, s1;
  segment(p, e, s0, s1);
  if (s0 >= s1) return;

  const int NT = p.N >> 5, KB = p.K >> 7, KC = (p.K + 255) >> 8;
  const int t0 = is_swiglu(EPI) ? blockIdx.x : 2 * blockIdx.x;
  const int t1 = is_swiglu(EPI) ? NT / 2 + blockIdx.x : min(2 * (int)blockIdx.x + 1, NT - 1);
  const size_t tile_bytes = (size_t)p.K * 16;  // 32 channels of e2m1
  const rsrc_t wr0 = make_rsrc(p.wc + ((size_t)e * NT + t0) * tile_bytes, (uint32_t)tile_bytes);
  const rsrc_t wr1 = make_rsrc(p.wc + ((size_t)e * NT + t1) * tile_bytes, (uint32_t)tile_bytes);
  const rsrc_t sr0 = make_rsrc(p.wsc + ((size_t)e * NT + t0) * KC * 256, KC * 256);
  const rsrc_t sr1 = make_rsrc(p.wsc + ((size_t)e * NT + t1) * KC * 256, KC * 256);
  const rsrc_t ar = make_rsrc(p.a, p.a_bytes);
  const rsrc_t asr = make_rsrc(p.as, p.as_bytes);
  const int kb0 = KB * wv / NW, kb1 = KB * (wv + 1) / NW;
  constexpr int kXB = AF == kE4M3 ? 128 : 64;  // activation bytes of a K block

  for (int r0 = s0; r0 < s1; r0 += 32) {
    // a lane without a row loads the last one's: its column is never stored
    const int src = source_row(p, min(r0 + col, s1 - 1));
    const uint32_t x_off = (uint32_t)src * (uint32_t)(KB * kXB) + 16 * half;
    const uint32_t xs_off = (uint32_t)src * (uint32_t)(KB * 4);
    auto load = [&](int kb) {
      SmallBlock<AF> b;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        b.w[0][s] = buf_x4(wr0, 16 * lane, kb * 2048 + 1024 * s);
        b.w[1][s] = buf_x4(wr1, 16 * lane, kb * 2048 + 1024 * s);
        if constexpr (AF == kE4M3) {
          b.x[s][0] = buf_x4(ar, x_off, kb * kXB + 64 * s);
          b.x[s][1] = buf_x4(ar, x_off, kb * kXB + 64 * s + 32);
        } else {
          b.x[s][0] = buf_x4(ar, x_off, kb * kXB + 32 * s);
        }
      }
      b.ws[0] = buf_x1(sr0, 4 * lane, (kb >> 1) * 256) >> (16 * (kb & 1));
      b.ws[1] = buf_x1(sr1, 4 * lane, (kb >> 1) * 256) >> (16 * (kb & 1));
      b.as = buf_x1(asr, xs_off, kb * 4) >> (8 * half);
      return b;
    };
    f32x16 acc[2] = {};
    SmallBlock<AF> q[D];
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (kb0 + i < kb1) q[i] = load(kb0 + i);
    for (int kb = kb0; kb < kb1; kb += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        if (kb + i < kb1) {
          const SmallBlock<AF> b = q[i];
          if (kb + i + D < kb1) q[i] = load(kb + i + D);
          i32x8 x0, x1;
          if constexpr (AF == kE4M3) {
            x0 = operand(b.x[0][0], b.x[0][1]);
            x1 = operand(b.x[1][0], b.x[1][1]);
          } else {
            x0 = operand(b.x[0][0]);
            x1 = operand(b.x[1][0]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            acc[t] = mx_mfma<AF, 0, 0>(operand(b.w[t][0]), x0, acc[t], b.ws[t], b.as);
            acc[t] = mx_mfma<AF, 1, 2>(operand(b.w[t][1]), x1, acc[t], b.ws[t], b.as);
          }
        }
      }
    }

    // Sum over the wavefronts' K ranges, in order; thread (q4, lane) then holds
    // channels 8 * q4 + 4 * half + 0..3 of both tiles for token col.
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) red[wv][t][r][lane] = acc[t][r];
    __syncthreads();
    const int row = r0 + col;
    float v[2][4];
    if (wv < 4) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float s = 0.0f;
#pragma unroll
          for (int w = 0; w < NW; ++w) s += red[w][t][4 * wv + i][lane];
          v[t][i] = s;
        }
      const int ch = 8 * wv + 4 * half;
      if constexpr (is_swiglu(EPI)) {
        const int I = p.N / 2;
        float h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = silu_mul(v[0][i], v[1][i]);
        if constexpr (EPI == kEpiSwiglu) {
          if (row < s1) {
            const u32x2 o = {pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + (size_t)row * I + 32 * t0 + ch) = o;
          }
        } else {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b = __builtin_bit_cast(uint32_t, h[i]) & 0x7FFFFFFFu;
            m = m > b ? m : b;
          }
          const uint32_t o = __shfl_xor(m, 32, 64);
          if (half == 0) amx[wv][col] = m > o ? m : o;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[0][i] = h[i];
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int tile = 2 * blockIdx.x + t;
          if (row < s1 && tile < NT) {
            const size_t o = (size_t)row * p.N + 32 * tile + ch;
            if constexpr (EPI == kEpiF32) {
              *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + o) = f32x4{v[t][0], v[t][1], v[t][2], v[t][3]};
            } else {
              u32x2 b;
#pragma unroll
              for (int i = 0; i < 2; ++i)
                b[i] = EPI == kEpiBf16 ? pack_bf16x2(v[t][2 * i], v[t][2 * i + 1])
                                       : (uint32_t)f32_to_f16(v[t][2 * i]) | ((uint32_t)f32_to_f16(v[t][2 * i + 1]) << 16);
              *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + o) = b;
            }
          }
        }
      }
    }
    __syncthreads();
    if constexpr (EPI == kEpiSwigluE4M3 || EPI == kEpiSwigluE2M1) {
      if (wv < 4 && row < s1) {
        constexpr int F = EPI == kEpiSwigluE4M3 ? kE4M3 : kE2M1;
        const int I = p.N / 2, ch = 8 * wv + 4 * half;
        uint32_t m = amx[0][col];
#pragma unroll
        for (int w = 1; w < 4; ++w) m = m > amx[w][col] ? m : amx[w][col];
        const bool bad = mx_not_finite(m);
        const int pe = mx_exponent<F>(m);
        const float inv = mx_inverse(pe);
        float u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = bad ? 0.0f : v[0][i] * inv;
        const size_t o = (size_t)row * I + 32 * t0 + ch;
        if constexpr (F == kE4M3)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + o) = mx_pack4_e4m3(u[0], u[1], u[2], u[3]);
        else
          *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.out) + o / 2) = (uint16_t)mx_pack4_e2m1(u[0], u[1], u[2], u[3]);
        if (wv == 0 && half == 0) p.out_scales[(size_t)row * (I >> 5) + t0] = bad ? (uint8_t)255 : (uint8_t)(pe + 127);
      }
      __syncthreads();  // amx is written again for the next rows
    }
  }
}

template <int AF, int EPI>
int launch_small(const MxK& k, hipStream_t s) {
  const int NT = k.N / 32;
  const dim3 grid(is_swiglu(EPI) ? NT / 2 : (NT + 1) / 2, k.E);
  hipLaunchKernelGGL((mx_small_kernel<AF, EPI, 4>), grid, dim3(256), 0, s, k);
  return (int)hipGetLastError();
}
template <int AF>
int launch_fmt(const MxK& k, int epi, hipStream_t s) {
  switch (epi) {
    case kEpiBf16: return launch_small<AF, kEpiBf16>(k, s);
    case kEpiSwiglu: return launch_small<AF, kEpiSwiglu>(k, s);
    case kEpiF32: return launch_small<AF, kEpiF32>(k, s);
    case kEpiF16: return launch_small<AF, kEpiF16>(k, s);
    case kEpiSwigluE4M3: return launch_small<AF, kEpiSwigluE4M3>(k, s);
    default: return launch_small<AF, kEpiSwigluE2M1>(k, s);
  }
}
}  // namespace

int launch_mxgemm(const MxGemmArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t row_codes = a.a_fmt == kE4M3 ? a.K : a.K / 2;
  const MxK k{a.wcodes, a.wscales, a.N, a.K, a.a, a.as, (uint32_t)(a.A_rows * row_codes),
              (uint32_t)((size_t)a.A_rows * (a.K / 32)), a.A_rows, a.gather, a.gather ? a.k : 1, a.seg, a.E, a.M_total,
              a.out, a.out_scales};
  return a.a_fmt == kE4M3 ? launch_fmt<kE4M3>(k, a.epilogue, s) : launch_fmt<kE2M1>(k, a.epilogue, s);
}

}  // namespace moe
