// Gradient of the gate-weighted combine and of the gates before it:
//   dy[pos(t, j)] = w[t][j] * dout[t],  dw[t][j] = <dout[t], y[pos(t, j)]>
//   dlogits[t][ids[t][j]] = w[t][j] * (dw[t][j] - sum_i w[t][i] dw[t][i])
// One workgroup per token: a thread keeps 8 values of dout per 2048 of the row,
// reads 8 of each expert's output and writes 8 of its gradient (16 bytes each),
// so every byte moves once.  The row sums are added in fp32 over a thread's
// values, the wavefront's lanes and the wavefronts, in that order; no atomics.
#include "segments.h"

namespace moe {

namespace {
constexpr int kThreads = 256;
constexpr int kSlots = 8;      // slots whose rows are loaded before the first is used
constexpr int kMaxSlots = 1024;

__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// YT: expert outputs in bf16 (0), fp32 (1) or fp16 (2).
template <int YT, bool F16>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGradArgs a) {
  __shared__ float part[kThreads / 64][kSlots];
  __shared__ float dws[kMaxSlots];
  __shared__ float dot;
  const int t = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int nvec = a.H >> 3, k = a.k;
  const int nv = a.n_valid ? min(*a.n_valid, a.T * k) : a.T * k;
  const u32x4* const dout = reinterpret_cast<const u32x4*>(a.dout + (size_t)t * a.H);
  for (int j0 = 0; j0 < k; j0 += kSlots) {
    int pos[kSlots];
    float w[kSlots], sum[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int j = j0 + i;
      const int p = j < k ? a.pos[(size_t)t * k + j] : -1;
      pos[i] = p >= 0 && p < nv ? p : -1;
      w[i] = j < k && a.w ? a.w[(size_t)t * k + j] : 1.0f;
      sum[i] = 0.0f;
    }
    for (int c = threadIdx.x; c < nvec; c += kThreads) {
      f32x4 v[kSlots][2];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        v[i][0] = v[i][1] = f32x4{};
        if (pos[i] < 0) continue;
        if constexpr (YT == 1) {
          const f32x4* row = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.y) + (size_t)pos[i] * a.H);
          v[i][0] = row[2 * c];
          v[i][1] = row[2 * c + 1];
        } else {
          const u32x4 b = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.y) + (size_t)pos[i] * a.H)[c];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[i][q >> 1][2 * (q & 1)] = widen16<YT == 2>((uint16_t)(b[q] & 0xFFFFu));
            v[i][q >> 1][2 * (q & 1) + 1] = widen16<YT == 2>((uint16_t)(b[q] >> 16));
          }
        }
      }
      const u32x4 db = dout[c];
      float d[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t x = db[q];
        d[2 * q] = bf16_lo(x);
        d[2 * q + 1] = bf16_hi(x);
      }
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (pos[i] < 0) continue;
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sum[i] = __builtin_fmaf(d[2 * q], v[i][q >> 1][2 * (q & 1)], sum[i]);
          sum[i] = __builtin_fmaf(d[2 * q + 1], v[i][q >> 1][2 * (q & 1) + 1], sum[i]);
          o[q] = pack16x2<F16>(w[i] * d[2 * q], w[i] * d[2 * q + 1]);
        }
        reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.dy) + (size_t)pos[i] * a.H)[c] = o;
      }
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const float s = lane_sum(sum[i]);
      if (lane == 0) part[wv][i] = s;
    }
    __syncthreads();
    if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < k) {
      const int j = j0 + threadIdx.x;
      float s = 0.0f;
      for (int x = 0; x < kThreads / 64; ++x) s += part[x][threadIdx.x];
      const int p = a.pos[(size_t)t * k + j];
      if (p < 0 || p >= nv) s = 0.0f;
      a.dw[(size_t)t * k + j] = s;
      dws[j] = s;
    }
    __syncthreads();
  }
  if (!a.dlogits) return;
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int j = 0; j < k; ++j) s = __builtin_fmaf(a.w[(size_t)t * k + j], dws[j], s);
    dot = s;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float g = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int p = a.pos[(size_t)t * k + j];
      if (a.ids[(size_t)t * k + j] == e && p >= 0 && p < nv) g += a.w[(size_t)t * k + j] * (dws[j] - dot);
    }
    a.dlogits[(size_t)t * a.E + e] = g;
  }
}

template <int YT>
int launch_typed(const CombineGradArgs& a, hipStream_t s) {
  if (a.dy_dtype == 2) hipLaunchKernelGGL((combine_grad_kernel<YT, true>), dim3(a.T), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((combine_grad_kernel<YT, false>), dim3(a.T), dim3(kThreads), 0, s, a);
  return (int)hipGetLastError();
}
}  // namespace

int launch_combine_grad(const CombineGradArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return a.y_dtype == 1 ? launch_typed<1>(a, s) : a.y_dtype == 2 ? launch_typed<2>(a, s) : launch_typed<0>(a, s);
}

}  // namespace moe
