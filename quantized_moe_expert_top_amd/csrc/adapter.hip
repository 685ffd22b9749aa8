// Low-rank adapters of many requests added to a shared projection's output:
//   out[t] = y[t] + scale[a] * B_a (A_a x[t])
// A workgroup takes up to 32 tokens of one adapter and a range of the output
// channels.  First v = A_a x (K split over the four wavefronts, added through
// LDS), then B_a v in chunks of 64 channels per wavefront; both on
// v_mfma_f32_16x16x32 with the adapter as the first operand, so that a lane holds
// neighbouring channels of one token.  A lane's register of tile i stands for
// channel 16*(lane / 16) + 4*i + register of the chunk: 16 neighbouring channels
// over the chunk's four tiles, 32 bytes in a row.
// v goes to the second product as hi + lo, two 16-bit numbers, each multiplied
// and both added in fp32: one would round v to 8 bits (bf16), as much as the
// output's own rounding.
#include "segments.h"

namespace moe {

namespace {
constexpr int kTM = 32;  // tokens of a workgroup

struct AdapterK {
  AdapterArgs a;
  int n_chunk, per_wg;  // chunks of 64 channels, and of a workgroup
  int n_nb;             // workgroups per row tile
};

template <bool F16, int YT, int NR>  // NR: tiles of 16 of the rank
__global__ __launch_bounds__(256) void adapter_kernel(AdapterK p) {
  constexpr int RP = (16 * NR + 31) / 32 * 32;  // the rank, padded to whole steps
  const AdapterArgs& a = p.a;
  __shared__ float red[4][NR][2][4][64];
  __shared__ __attribute__((aligned(16))) uint16_t vh[kTM][RP + 8], vl[kTM][RP + 8];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  int idx = blockIdx.x;
  RowTile t;
  bool none = false;
  if (!find_tile<kTM>(a.seg, a.n, a.T, p.n_nb, idx, t)) {
    // tokens without an adapter come behind the others: copied, 32 a workgroup
    const int end = min(max(a.seg[a.n], 0), a.T);
    if (a.out == a.y || idx >= (a.T - end + kTM - 1) / kTM * p.n_nb) return;
    none = true;
    t.e = 0;
    t.r0 = end;
    t.s1 = a.T;
  }
  const int r0 = t.r0 + idx / p.n_nb * kTM, c0 = idx % p.n_nb * p.per_wg, c1 = min(c0 + p.per_wg, p.n_chunk);
  int tok[2];  // this lane's tokens of the two column tiles; past the end the last again, never stored
#pragma unroll
  for (int b = 0; b < 2; ++b) tok[b] = min(max(a.rows[min(r0 + 16 * b + col, t.s1 - 1)], 0), a.T - 1);

  if (!none) {
    const rsrc_t xr = make_rsrc(a.x, (uint32_t)((size_t)a.T * a.K * 2));
    const rsrc_t ar = make_rsrc(static_cast<const uint16_t*>(a.A) + (size_t)t.e * a.r * a.K, (uint32_t)((size_t)a.r * a.K * 2));
    f32x4 acc[NR][2] = {};
    for (int k0 = 32 * wv; k0 < a.K; k0 += 128) {
      const uint32_t k = k0 + 8 * q;
      const bool in = (int)k < a.K;
      u32x4 xv[2], av[NR];
#pragma unroll
      for (int b = 0; b < 2; ++b) xv[b] = buf_x4(xr, in ? ((uint32_t)tok[b] * a.K + k) * 2 : ~0u, 0);
#pragma unroll
      for (int i = 0; i < NR; ++i) av[i] = buf_x4(ar, in && 16 * i + col < a.r ? ((16 * i + col) * a.K + k) * 2 : ~0u, 0);
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[i][b] = mfma16t<F16>(av[i], xv[b], acc[i][b]);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wv][i][b][r][lane] = acc[i][b][r];
    __syncthreads();
    for (int i = threadIdx.x; i < kTM * RP; i += 256) {
      const int row = i / RP, c = i % RP;
      float v = 0.0f;
      if (c < 16 * NR)
#pragma unroll
        for (int w = 0; w < 4; ++w) v += red[w][c >> 4][row >> 4][c & 3][16 * ((c >> 2) & 3) + (row & 15)];
      const uint16_t hi = round16<F16>(v);
      vh[row][c] = hi;
      vl[row][c] = round16<F16>(v - widen16<F16>(hi));
    }
    __syncthreads();
  }
  const float scale = none ? 0.0f : a.scale ? a.scale[t.e] : 1.0f;
  const rsrc_t br = make_rsrc(static_cast<const uint16_t*>(a.B) + (size_t)t.e * a.N * a.r, (uint32_t)((size_t)a.N * a.r * 2));
  for (int c = c0 + wv; c < c1; c += 4) {
    f32x4 d[4][2] = {};
    if (!none) {
      for (int k0 = 0; k0 < a.r; k0 += 32) {
        const int k = k0 + 8 * q;
        u32x4 bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ch = 64 * c + 16 * (col >> 2) + 4 * i + (col & 3);
          bv[i] = buf_x4(br, k < a.r && ch < a.N ? ((uint32_t)ch * a.r + k) * 2 : ~0u, 0);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const u32x4 h = *reinterpret_cast<const u32x4*>(&vh[16 * b + col][k]);
          const u32x4 l = *reinterpret_cast<const u32x4*>(&vl[16 * b + col][k]);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i][b] = mfma16t<F16>(bv[i], h, mfma16t<F16>(bv[i], l, d[i][b]));
        }
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int ch = 64 * c + 16 * q;
      if (r0 + 16 * b + col >= t.s1) continue;
#pragma unroll
      for (int i = 0; i < 4; i += 2) {  // 8 channels at a time
        if (ch + 4 * i >= a.N) continue;
        const size_t at = (size_t)tok[b] * a.N + ch + 4 * i;
        if constexpr (YT == 1) {
          const f32x4* y = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.y) + at);
          f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f32x4 v = y[j];
            if (!none)
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(scale, d[i + j][b][r], v[r]);
            o[j] = v;
          }
        } else {
          u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.y) + at);
          if (!none) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t x = v[j];
              const float lo = widen16<YT == 2>((uint16_t)(x & 0xFFFFu)), hi = widen16<YT == 2>((uint16_t)(x >> 16));
              v[j] = pack16x2<YT == 2>(__builtin_fmaf(scale, d[i + j / 2][b][2 * (j & 1)], lo),
                                       __builtin_fmaf(scale, d[i + j / 2][b][2 * (j & 1) + 1], hi));
            }
          }
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + at) = v;
        }
      }
    }
  }
}

template <bool F16, int YT>
int launch_rank(const AdapterK& p, unsigned wgs, hipStream_t s) {
  if (p.a.r <= 16) hipLaunchKernelGGL((adapter_kernel<F16, YT, 1>), dim3(wgs), dim3(256), 0, s, p);
  else if (p.a.r <= 32) hipLaunchKernelGGL((adapter_kernel<F16, YT, 2>), dim3(wgs), dim3(256), 0, s, p);
  else if (p.a.r <= 64) hipLaunchKernelGGL((adapter_kernel<F16, YT, 4>), dim3(wgs), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((adapter_kernel<F16, YT, 8>), dim3(wgs), dim3(256), 0, s, p);
  return (int)hipGetLastError();
}
template <bool F16>
int launch_typed(const AdapterK& p, unsigned wgs, hipStream_t s) {
  return p.a.y_dtype == 1 ? launch_rank<F16, 1>(p, wgs, s) : p.a.y_dtype == 2 ? launch_rank<F16, 2>(p, wgs, s)
                                                                              : launch_rank<F16, 0>(p, wgs, s);
}
}  // namespace

int launch_adapter_add(const AdapterArgs& a, void* stream) {
  AdapterK p{a, (a.N + 63) / 64, 0, 0};
  // tiles: one partial per adapter that has tokens, and one of the tokens without
  const int64_t tiles = (int64_t)a.T / kTM + (a.n < a.T ? a.n : a.T) + 1;
  const int64_t want = tiles >= 512 ? 1 : (512 + tiles - 1) / tiles;
  const int n_nb = (int)(want < (p.n_chunk + 3) / 4 ? want : (p.n_chunk + 3) / 4);
  p.per_wg = (p.n_chunk + n_nb - 1) / n_nb;
  p.n_nb = (p.n_chunk + p.per_wg - 1) / p.per_wg;
  const int64_t wgs = tiles * p.n_nb;
  if (wgs >= ((int64_t)1 << 23)) return (int)hipErrorInvalidConfiguration;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return a.dtype == 2 ? launch_typed<true>(p, (unsigned)wgs, s) : launch_typed<false>(p, (unsigned)wgs, s);
}

}  // namespace moe
