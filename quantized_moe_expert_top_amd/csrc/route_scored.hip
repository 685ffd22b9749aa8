// Expert choice from scores of all experts: softmax or sigmoid, a choice bias,
// expert groups, top-k, renormalised and scaled weights.
//
// One wavefront per token; lane l owns experts l, l + 64, ... (NS per lane).
// Scores are float64: the choice depends on scores next to each other, and
// float64 makes it the same however they are summed.  Groups are contiguous, so
// their bests come from the wavefront's LDS copy of the choice scores, one lane
// per group; the group ranks are a count of better groups.  Then k wave-wide
// arg-max rounds over (score, -index).
#include <float.h>

#include "common.h"

namespace moe {

namespace {
constexpr int kWavesPerBlock = 4;
constexpr int kMaxE = 1024;

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ __forceinline__ double neg_inf() { return -__builtin_inf(); }

template <int NS>
__global__ __launch_bounds__(64 * kWavesPerBlock) void route_scored_kernel(ScoredArgs a) {
  __shared__ double lds[kWavesPerBlock][64 * NS];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kWavesPerBlock + wv;
  if (t >= a.T) return;
  double* const buf = lds[wv];
  const float* row = a.logits + (size_t)t * a.E;

  float x[NS], b[NS];
  float top = -__builtin_inff();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int e = lane + 64 * s;
    float v = e < a.E ? row[e] : -__builtin_inff();
    b[s] = (a.bias && e < a.E) ? a.bias[e] : 0.0f;
    v = v != v ? -__builtin_inff() : fminf(v, FLT_MAX);
    x[s] = v;
    top = fmaxf(top, v);
  }
  double score[NS], c[NS];
  if (a.score == 0) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    double sum = 0.0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      score[s] = x[s] == -__builtin_inff() ? 0.0 : exp((double)x[s] - (double)top);
      sum += score[s];
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
#pragma unroll
    for (int s = 0; s < NS; ++s) score[s] = sum > 0.0 ? score[s] / sum : 0.0;
  } else {
#pragma unroll
    for (int s = 0; s < NS; ++s) score[s] = 1.0 / (1.0 + exp(-(double)x[s]));
  }
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const double v = score[s] + (double)b[s];
    c[s] = (x[s] == -__builtin_inff() || v != v) ? neg_inf() : v;
  }

  if (a.n_group > 1) {
    const int size = a.E / a.n_group;
#pragma unroll
    for (int s = 0; s < NS; ++s) buf[lane + 64 * s] = c[s];
    wave_fence();
    double best = neg_inf(), second = neg_inf();
    if (lane < a.n_group)
      for (int i = 0; i < size; ++i) {
        const double v = buf[lane * size + i];
        if (v > best) {
          second = best;
          best = v;
        } else if (v > second) {
          second = v;
        }
      }
    if (a.group_top == 2 && second > neg_inf()) best += second;
    int before = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const double v = __shfl(best, g, 64);
      before += (v > best || (v == best && g < lane)) ? 1 : 0;
    }
    const uint64_t open = __ballot(lane < a.n_group && before < a.topk_group);
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (lane + 64 * s < a.E && !((open >> ((lane + 64 * s) / size)) & 1)) c[s] = neg_inf();
    wave_fence();
  }

  // k rounds; slot j's score goes to the wavefront's buffer
  const size_t o = (size_t)t * a.k;
  for (int j = 0; j < a.k; ++j) {
    double bv = neg_inf();
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (c[s] > bv) {
        bv = c[s];
        bi = lane + 64 * s;
      }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      const double ov = __shfl_xor(bv, off, 64);
      const int oi = __shfl_xor(bi, off, 64);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bi = oi;
      }
    }
    const bool none = bi == 0x7FFFFFFF;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (lane + 64 * s == bi) {
        c[s] = neg_inf();
        buf[j] = score[s];
      }
    if (lane == 0) {
      a.ids[o + j] = none ? -1 : bi;
      if (none) buf[j] = 0.0;
    }
  }
  wave_fence();
  double sum = 1.0;
  if (a.renorm) {
    sum = 0.0;
    for (int j = 0; j < a.k; ++j) sum += buf[j];
  }
  for (int j = lane; j < a.k; j += 64)
    a.w[o + j] = sum > 0.0 ? (float)(buf[j] / sum * (double)a.scale) : 0.0f;
}
}  // namespace

int launch_route_scored(const ScoredArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((a.T + kWavesPerBlock - 1) / kWavesPerBlock), block(64 * kWavesPerBlock);
  if (a.E <= 64) hipLaunchKernelGGL(route_scored_kernel<1>, grid, block, 0, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL(route_scored_kernel<2>, grid, block, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL(route_scored_kernel<4>, grid, block, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL(route_scored_kernel<8>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(route_scored_kernel<16>, grid, block, 0, s, a);
  return (int)hipGetLastError();
}

}  // namespace moe
