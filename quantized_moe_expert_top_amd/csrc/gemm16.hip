// Grouped product of rows with the experts' 16-bit weights, and its gradients by
// the rows and by the weights, on v_mfma_f32_32x32x16 (bf16 or fp16 operands,
// fp32 sums).
#include "segments.h"

namespace moe {

namespace {
constexpr int kForward = 0, kRows = 1, kWeights = 2;                               // what a kernel computes
constexpr int kEpiBf16 = 0, kEpiSwiglu = 1, kEpiF32 = 2, kEpiF16 = 3, kEpiSwigluGrad = 6;  // MOE_EPI_*

struct GemmK {  // kernel arguments
  const uint16_t* w;
  const uint16_t* a;
  const uint16_t* dy;
  int E, N, K, A_rows, M_total;
  const int32_t* gather;
  PairDiv div;
  const int32_t* seg;
  const uint16_t* pre_in;
  uint16_t* pre_out;
  void* out;
};

__device__ __forceinline__ int source_row(const GemmK& p, int row) {
  const int r = p.gather ? p.div(p.gather[row]) : row;
  return min(max(r, 0), p.A_rows - 1);
}
__device__ __forceinline__ void store_one(void* out, size_t at, int epi, float v) {
  if (epi == kEpiF32) static_cast<float*>(out)[at] = v;
  else static_cast<uint16_t*>(out)[at] = epi == kEpiF16 ? f32_to_f16(v) : f32_to_bf16(v);
}

// 64 x 64 tiles, operands element by element through LDS.
template <bool F16, int MODE>
__global__ __launch_bounds__(256) void gemm16_kernel(GemmK p, int epi, int n_ab) {
  __shared__ __attribute__((aligned(16))) uint16_t P[64][40], Q[64][40];
  __shared__ float C[64][65];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, wa = wv & 1, wb = wv >> 1;
  const bool sw = epi == kEpiSwiglu;
  int e, ab, b0, s0 = 0, s1 = 0, red;
  if constexpr (MODE == kWeights) {
    e = blockIdx.z;
    ab = blockIdx.x;
    b0 = blockIdx.y * 64;
    if (p.M_total > 0) segment_rows(p.seg, e, p.M_total, s0, s1);
    red = s1 - s0;
  } else {
    int idx = blockIdx.x;
    RowTile t;
    if (!find_tile<64>(p.seg, p.E, p.M_total, n_ab, idx, t)) return;
    e = t.e;
    ab = idx % n_ab;
    b0 = t.r0 + idx / n_ab * 64;
    s1 = t.s1;
    red = MODE == kForward ? p.K : p.N;
  }
  const int I = p.N / 2;
  const uint16_t* const w = MODE == kWeights ? nullptr : p.w + (size_t)e * p.N * p.K;
  f32x16 acc = {};
  for (int k0 = 0; k0 < red; k0 += 32) {
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      uint16_t pv = 0, qv = 0;
      const int r = i >> 5, kk = k0 + (i & 31);
      if constexpr (MODE == kForward) {
        const int ch = sw ? (r < 32 ? 32 * ab + r : 32 * ab + r - 32) : 64 * ab + r;
        if (kk < red && ch < (sw ? I : p.N)) pv = w[(size_t)(sw && r >= 32 ? I + ch : ch) * p.K + kk];
        if (kk < red && b0 + r < s1) qv = p.a[(size_t)source_row(p, b0 + r) * p.K + kk];
      } else if constexpr (MODE == kRows) {
        if (kk < red && 64 * ab + r < p.K) pv = w[(size_t)kk * p.K + 64 * ab + r];
        if (kk < red && b0 + r < s1) qv = p.dy[(size_t)(b0 + r) * p.N + kk];
      } else if (kk < red) {
        if (64 * ab + r < p.K) pv = p.a[(size_t)source_row(p, s0 + kk) * p.K + 64 * ab + r];
        if (b0 + r < p.N) qv = p.dy[(size_t)(s0 + kk) * p.N + b0 + r];
      }
      P[r][i & 31] = pv;
      Q[r][i & 31] = qv;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int c = 16 * s + 8 * (lane >> 5);
      acc = mfma32t<F16>(*reinterpret_cast<const u32x4*>(&P[32 * wa + (lane & 31)][c]),
                         *reinterpret_cast<const u32x4*>(&Q[32 * wb + (lane & 31)][c]), acc);
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) C[32 * wb + (lane & 31)][32 * wa + acc_row(r, lane)] = acc[r];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int b = b0 + (i >> 6), a = i & 63;
    const float v = C[i >> 6][a];
    if constexpr (MODE == kForward) {
      if (b >= s1) continue;
      if (sw) {
        const int ch = 32 * ab + (a & 31);
        if (ch >= I) continue;
        if (p.pre_out) p.pre_out[(size_t)b * p.N + (a < 32 ? ch : I + ch)] = round16<F16>(v);
        if (a < 32)
          static_cast<uint16_t*>(p.out)[(size_t)b * I + ch] = round16<F16>(v / (1.0f + __expf(-v)) * C[i >> 6][32 + a]);
      } else if (64 * ab + a < p.N) {
        store_one(p.out, (size_t)b * p.N + 64 * ab + a, epi, v);
      }
    } else if constexpr (MODE == kRows) {
      const int ch = 64 * ab + a;
      if (b >= s1 || ch >= p.K) continue;
      if (epi == kEpiSwigluGrad) {
        const size_t at = (size_t)b * 2 * p.K + ch;
        const float g = widen16<F16>(p.pre_in[at]), u = widen16<F16>(p.pre_in[at + p.K]);
        const float s = 1.0f / (1.0f + __expf(-g));
        static_cast<uint16_t*>(p.out)[at] = round16<F16>(v * u * s * (1.0f + g * (1.0f - s)));
        static_cast<uint16_t*>(p.out)[at + p.K] = round16<F16>(v * g * s);
      } else {
        store_one(p.out, (size_t)b * p.K + ch, epi, v);
      }
    } else if (b < p.N && 64 * ab + a < p.K) {
      store_one(p.out, ((size_t)e * p.N + b) * p.K + 64 * ab + a, epi, v);
    }
  }
}

GemmK kernel_args(const Gemm16Args& a) {
  return GemmK{static_cast<const uint16_t*>(a.w), static_cast<const uint16_t*>(a.a), static_cast<const uint16_t*>(a.dy),
               a.E, a.N, a.K, a.A_rows, a.M_total, a.gather, pair_div(a.gather ? a.k : 1), a.seg,
               static_cast<const uint16_t*>(a.pre_in), static_cast<uint16_t*>(a.pre_out), a.out};
}
// Upper bound of the tiles of `rows` rows: one partial tile per segment that has rows.
int64_t row_tiles(int M_total, int E, int rows) { return (int64_t)M_total / rows + (E < M_total ? E : M_total); }

template <int MODE>
int launch_rowwise(const Gemm16Args& a, int n_ab, hipStream_t s) {
  const int64_t wgs = row_tiles(a.M_total, a.E, 64) * n_ab;
  if (wgs >= ((int64_t)1 << 23)) return (int)hipErrorInvalidConfiguration;
  if (a.dtype == 2) hipLaunchKernelGGL((gemm16_kernel<true, MODE>), dim3((unsigned)wgs), dim3(256), 0, s, kernel_args(a), a.epilogue, n_ab);
  else hipLaunchKernelGGL((gemm16_kernel<false, MODE>), dim3((unsigned)wgs), dim3(256), 0, s, kernel_args(a), a.epilogue, n_ab);
  return (int)hipGetLastError();
}
}  // namespace

int launch_gemm16(const Gemm16Args& a, void* stream) {
  const int n_ab = a.epilogue == kEpiSwiglu ? (a.N / 2 + 31) / 32 : (a.N + 63) / 64;
  return launch_rowwise<kForward>(a, n_ab, static_cast<hipStream_t>(stream));
}
int launch_gemm16_grad_rows(const Gemm16Args& a, void* stream) {
  return launch_rowwise<kRows>(a, (a.K + 63) / 64, static_cast<hipStream_t>(stream));
}
size_t gemm16_grad_weights_workspace_bytes(int E, int N, int K, int M_total, int kernel) { return 0; }
int launch_gemm16_grad_weights(const Gemm16Args& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((a.K + 63) / 64, (a.N + 63) / 64, a.E);
  if (grid.y > 65535) return (int)hipErrorInvalidConfiguration;
  if (a.dtype == 2) hipLaunchKernelGGL((gemm16_kernel<true, kWeights>), grid, dim3(256), 0, s, kernel_args(a), a.epilogue, 0);
  else hipLaunchKernelGGL((gemm16_kernel<false, kWeights>), grid, dim3(256), 0, s, kernel_args(a), a.epilogue, 0);
  return (int)hipGetLastError();
}

}  // namespace moe
