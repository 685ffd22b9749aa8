// Gradient of the gate-weighted combine and of the gates before it:
//   dy[pos(t, j)] = w[t][j] * dout[t],  dw[t][j] = <dout[t], y[pos(t, j)]>
//   dlogits[t][ids[t][j]] = w[t][j] * (dw[t][j] - sum_i w[t][i] dw[t][i])
// One workgroup per token: a thread keeps 8 values of dout per 2048 of the row,
// reads 8 of each expert's output and writes 8 of its gradient (16 bytes each),
// so every byte moves once.  The row sums are added in fp32 over a thread's
// values, the wavefront's lanes and the wavefronts, in that order; no atomics.
// Bytes bound it: 8192 tokens x 8 of 2048, y in fp16, 570 MB in 108 us (5.3 TB/s, a
// copy's rate).  What brought it there from 177 us: streaming loads and stores (a row
// moves once), the slots' places read once through LDS and not by every thread, lane
// sums by exchanged halves.
#include "segments.h"

namespace moe {

namespace {
constexpr int kThreads = 256;
constexpr int kSlots = 8;      // slots whose rows are loaded before the first is used
constexpr int kMaxSlots = 1024;

// Sums of eight values over the wavefront's lanes: pairs of lanes exchange halves of
// their values, so that 10 exchanges do and not 48; lane l holds the sum of value l / 8.
__device__ __forceinline__ float lane_sums(const float (&v)[kSlots]) {
  const int lane = threadIdx.x & 63;
  float a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float mine = lane & 32 ? v[i + 4] : v[i], other = lane & 32 ? v[i] : v[i + 4];
    a[i] = mine + __shfl_xor(other, 32, 64);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float mine = lane & 16 ? a[i + 2] : a[i], other = lane & 16 ? a[i] : a[i + 2];
    b[i] = mine + __shfl_xor(other, 16, 64);
  }
  const float mine = lane & 8 ? b[1] : b[0], other = lane & 8 ? b[0] : b[1];
  c = mine + __shfl_xor(other, 8, 64);
#pragma unroll
  for (int off = 4; off; off >>= 1) c += __shfl_xor(c, off, 64);
  return c;
}

// YT: expert outputs in bf16 (0), fp32 (1) or fp16 (2).
template <int YT, bool F16>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGradArgs a) {
  __shared__ float part[kThreads / 64][kSlots];
  __shared__ float dws[kMaxSlots], ws[kMaxSlots];
  __shared__ int at[kMaxSlots], id[kMaxSlots];
  const int t = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int nvec = a.H >> 3, k = a.k;
  const u32x4* const dout = reinterpret_cast<const u32x4*>(a.dout + (size_t)t * a.H);
  const int c0 = threadIdx.x;
  u32x4 first = {};  // (on its way with the slots' places)
  if (c0 < nvec) first = __builtin_nontemporal_load(dout + c0);
  const int nv = a.n_valid ? min(*a.n_valid, a.T * k) : a.T * k;
  for (int j = threadIdx.x; j < k; j += kThreads) {
    const int p = a.pos[(size_t)t * k + j];
    at[j] = p >= 0 && p < nv ? p : -1;
    ws[j] = a.w ? a.w[(size_t)t * k + j] : 1.0f;
    id[j] = a.ids ? a.ids[(size_t)t * k + j] : -1;
  }
  __syncthreads();
  for (int j0 = 0; j0 < k; j0 += kSlots) {
    int pos[kSlots];
    float w[kSlots], sum[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      pos[i] = j0 + i < k ? __builtin_amdgcn_readfirstlane(at[j0 + i]) : -1;
      w[i] = j0 + i < k ? ws[j0 + i] : 0.0f;
      sum[i] = 0.0f;
    }
    for (int c = c0; c < nvec; c += kThreads) {
      f32x4 v[kSlots][YT == 1 ? 2 : 1];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (pos[i] < 0) continue;
        if constexpr (YT == 1) {
          const f32x4* row = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.y) + (size_t)pos[i] * a.H);
          v[i][0] = __builtin_nontemporal_load(row + 2 * c);
          v[i][1] = __builtin_nontemporal_load(row + 2 * c + 1);
        } else {
          v[i][0] = __builtin_bit_cast(f32x4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.y) + (size_t)pos[i] * a.H) + c));
        }
      }
      const u32x4 db = c == c0 ? first : dout[c];
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
          float y0, y1;
          if constexpr (YT == 1) {
            y0 = v[i][q >> 1][2 * (q & 1)];
            y1 = v[i][q >> 1][2 * (q & 1) + 1];
          } else {
            const uint32_t x = __builtin_bit_cast(u32x4, v[i][0])[q];
            y0 = widen16<YT == 2>((uint16_t)(x & 0xFFFFu));
            y1 = widen16<YT == 2>((uint16_t)(x >> 16));
          }
          sum[i] = __builtin_fmaf(d[2 * q], y0, sum[i]);
          sum[i] = __builtin_fmaf(d[2 * q + 1], y1, sum[i]);
          o[q] = pack16x2<F16>(w[i] * d[2 * q], w[i] * d[2 * q + 1]);
        }
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.dy) + (size_t)pos[i] * a.H) + c);
      }
    }
    const float total = lane_sums(sum);
    if ((lane & 7) == 0) part[wv][lane >> 3] = total;
    __syncthreads();
    if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < k) {
      const int j = j0 + threadIdx.x;
      float s = 0.0f;
#pragma unroll
      for (int x = 0; x < kThreads / 64; ++x) s += part[x][threadIdx.x];
      if (at[j] < 0) s = 0.0f;
      a.dw[(size_t)t * k + j] = s;
      dws[j] = s;
    }
    __syncthreads();
  }
  if (!a.dlogits) return;
  float dot = 0.0f;
  for (int j = 0; j < k; ++j)
    if (at[j] >= 0) dot = __builtin_fmaf(ws[j], dws[j], dot);  // (a weight that no row got may be anything)
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float g = 0.0f;
    for (int j = 0; j < k; ++j)
      if (id[j] == e && at[j] >= 0) g += ws[j] * (dws[j] - dot);
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
