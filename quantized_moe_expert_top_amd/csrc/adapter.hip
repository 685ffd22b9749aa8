// Low-rank adapters of many requests added to a shared projection's output:
//   out[t] = y[t] + scale[a] * B_a (A_a x[t])
// A workgroup takes up to 32 tokens of one adapter and a range of the output
// channels.  First v = A_a x (K split over the four wavefronts, added through
// LDS), then B_a v in chunks of 64 channels per wavefront; both on
// v_mfma_f32_16x16x32 with the adapter as the first operand, so that a lane holds
// neighbouring channels of one token.  A lane's register of tile i stands for
// channel 16*(lane / 16) + 4*i + register of the chunk: 16 neighbouring channels
// over the chunk's four tiles, 32 bytes in a row.
// v keeps fp32's 24 bits and range: it goes to the second product as three bf16
// numbers, B's fp16 numbers as two, all exact, and their products are added in fp32
// (bf16 products for either type: fp16 parts of v would end at 65504 and at 2^-24).
// Three parts cost bf16 nothing that shows, two of B cost fp16: 4096 tokens, 4096 to 14336,
// ranks 16, 32, 64 and 128, us: 57, 74, 151, 246 in bf16, 64, 76, 161, 316 in fp16.
// Bytes bound long batches: y in, out, x and the adapters.  4096 tokens, 4096 to
// 14336, rank 32, 16 adapters, y and out in bf16, us: 74 (288 MB, 3.9 TB/s; a copy of
// them 55), of which the first product, that all workgroups start with, 16; with 32 tokens a workgroup 129, with single steps of the first product (a
// line of x fetched by two wavefronts) and one chunk under way 78; rank 16 57, with one
// chunk under way 82.  Latency bounds few tokens: a chain of dependent accesses, 10.4 us
// for 32 tokens of 16 adapters of rank 16, 4096 to 4096, 6 of them the first product's.
#include "segments.h"

namespace moe {

namespace {
constexpr int kWorkgroups = 256;
// Tiles of 16 tokens of a workgroup.
constexpr int token_tiles(int nr) { return nr <= 2 ? 1 : 2; }
// v = high + rest, high a bf16 number of v's sign that is nearer to zero.  Exact: rest has
// 8 bits fewer than v (three parts hold fp32's 24 bits, two fp16's 11).  Neither part is zero
// unless v is, so that an infinity which meets v meets numbers of v's sign; an infinite v has
// the largest number for high and is itself the rest.  (Below 2^-100 a last part may be subnormal
// and count for nothing: 2^-126 absolute.)
struct Parts {
  float high, rest;
};
__device__ __forceinline__ Parts cut_bf16(float v) {
  // the next fp32 number towards zero (v - v * 2^-24, rounded), without its last 16 bits
  const float below = __builtin_amdgcn_fmed3f(v, -0x1.fffffep127f, 0x1.fffffep127f) * 0x1.fffffep-1f;
  const float high = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, below) & 0xFFFF0000u);
  return {high, v - high};
}
// Two floats that are bf16 numbers (their last 16 bits zero), as a pair.
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}
// Eight of B's numbers as bf16 ones: themselves, or for fp16 high parts and rests of the numbers
// times 2^-15, for which the sums make up.  Parts as of cut_bf16, in 8 instructions a pair where
// that takes 12 (4096 tokens, 4096 to 14336, us: rank 16 66, rank 128 330): finite numbers are
// below 2 then, the top bit of their exponent is 0, and an infinite one's is masked off.
constexpr float kScaleB = 0x1p-15f;
__device__ __forceinline__ Parts cut_f16(_Float16 v) {
  const float below = __builtin_fmaf((float)v, kScaleB * 0x1.fffffep-1f, 0.0f);
  const float high = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, below) & 0xBFFF0000u);
  return {high, __builtin_fmaf((float)v, kScaleB, -high)};
}
template <bool F16>
__device__ __forceinline__ void split_b(u32x4 b, u32x4 (&to)[F16 ? 2 : 1]) {
  if constexpr (F16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
      const uint32_t x = b[q];
      const f16x2 v = __builtin_bit_cast(f16x2, x);
      const Parts l = cut_f16(v[0]), h = cut_f16(v[1]);
      to[0][q] = pair_bf16(l.high, h.high);
      to[1][q] = pair_bf16(l.rest, h.rest);
    }
  } else {
    to[0] = b;
  }
}

// Wavefronts of a workgroup: the sums that they exchange take 2 KB of LDS each and tile of 16 ranks.
constexpr int waves(int nr) { return nr <= 4 ? 8 : 4; }

struct AdapterK {
  AdapterArgs a;
  int n_chunk, per_wg;  // chunks of 64 channels, and of a workgroup
  int n_nb;             // workgroups per row tile
};

template <bool F16, int YT, int NR>  // NR: tiles of 16 of the rank
__global__ __launch_bounds__(64 * waves(NR), NR <= 2 ? 4 : 2) void adapter_kernel(AdapterK p) {
  constexpr int W = waves(NR), RP = (16 * NR + 31) / 32 * 32;  // the rank, padded to whole steps
  constexpr int NB = token_tiles(NR), kTM = 16 * NB;           // tokens
  constexpr int U = 2;                                         // steps of the first product loaded at a time
  const AdapterArgs& a = p.a;
  // the first product's sums; then a wavefront's 16 x 64 results of the second
  constexpr int RED = W * NR * NB * 64 > W * 256 ? W * NR * NB * 64 : W * 256;
  __shared__ f32x4 lds[RED];
  auto red = [&](int w, int i, int b) { return lds + ((w * NR + i) * NB + b) * 64; };
  __shared__ __attribute__((aligned(16))) uint16_t parts[3][kTM][RP + 8];  // of v
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  int idx = blockIdx.x;
  RowTile t;
  bool none = false;
  if (!find_tile<kTM>(a.seg, a.n, a.T, p.n_nb, idx, t)) {
    // tokens without an adapter come behind the others: copied a tile a workgroup
    const int end = min(max(a.seg[a.n], 0), a.T);
    if (a.out == a.y || idx >= (a.T - end + kTM - 1) / kTM * p.n_nb) return;
    none = true;
    t.e = 0;
    t.r0 = end;
    t.s1 = a.T;
  }
  const int r0 = t.r0 + idx / p.n_nb * kTM, c0 = idx % p.n_nb * p.per_wg, c1 = min(c0 + p.per_wg, p.n_chunk);
  int tok[NB];  // this lane's tokens in the first product; past the end the last again, never stored
#pragma unroll
  for (int b = 0; b < NB; ++b) tok[b] = min(max(a.rows[min(r0 + 16 * b + col, t.s1 - 1)], 0), a.T - 1);

  // Second product, in chunks of 64 channels.  It leaves a lane four channels of a token
  // and goes through 4 KB of LDS a wavefront and 16 tokens, so that y is read and out
  // written 128 bytes and more in a row: 16 bytes a lane, LR lanes a row, RI rows at a time.
  constexpr int V = YT == 1 ? 4 : 8, LR = 64 / V, RI = 64 / LR, IT = kTM / RI;
  int row_tok[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) row_tok[i] = min(max(a.rows[min(r0 + RI * i + lane / LR, t.s1 - 1)], 0), a.T - 1);
  const rsrc_t br = scalar_rsrc(static_cast<const uint16_t*>(a.B) + (size_t)t.e * a.N * a.r, (uint32_t)((size_t)a.N * a.r * 2));
  constexpr int ES = YT == 1 ? 4 : 2;
  struct Chunk {
    u32x4 b[RP / 32][4];
    u32x4 y[IT];
  };
  auto fetch = [&](int c) {
    Chunk k;
#pragma unroll
    for (int s = 0; s < RP / 32; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 32 * s + 8 * quad, ch = 64 * c + 16 * i + col;
        k.b[s][i] = buf_x4(br, !none && at < a.r && ch < a.N ? ((uint32_t)ch * (uint32_t)a.r + at) * 2 : ~0u, 0);
      }
    const int ch = min(64 * c + V * (lane % LR), a.N - V);
#pragma unroll
    for (int i = 0; i < IT; ++i)
      k.y[i] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.y) + ((size_t)row_tok[i] * a.N + ch) * ES);
    return k;
  };
  constexpr int D = NR <= 4 ? 2 : 1;  // chunks under way, while the first product is worked out too
  Chunk ring[D];
#pragma unroll
  for (int u = 0; u < D; ++u)
    if (u == 0 || c0 + wv + W * u < c1) ring[u] = fetch(c0 + wv + W * u);

  if (!none) {
    // First product: wavefront wv takes pairs wv, wv + W, ... of steps of 32 inputs, a
    // line of 128 bytes of every row (single steps: a line fetched by two wavefronts).
    const rsrc_t xr = scalar_rsrc(a.x, (uint32_t)((size_t)a.T * a.K * 2));
    const rsrc_t ar = scalar_rsrc(static_cast<const uint16_t*>(a.A) + (size_t)t.e * a.r * a.K, (uint32_t)((size_t)a.r * a.K * 2));
    struct Step {
      u32x4 x[NB], w[NR];
    };
    auto load = [&](int k0) {
      Step s;
      const uint32_t k = k0 + 8 * quad;
      const bool in = (int)k < a.K;
#pragma unroll
      for (int b = 0; b < NB; ++b) s.x[b] = buf_x4(xr, in ? ((uint32_t)tok[b] * (uint32_t)a.K + k) * 2 : ~0u, 0);
#pragma unroll
      for (int i = 0; i < NR; ++i) s.w[i] = buf_x4(ar, in && 16 * i + col < a.r ? ((uint32_t)(16 * i + col) * (uint32_t)a.K + k) * 2 : ~0u, 0);
      return s;
    };
    f32x4 acc[NR][NB] = {};
    Step s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (in the order of their use, which the loop's waits count on: 77 us without, 73 so)
      s[u] = load(64 * (wv + W * (u >> 1)) + 32 * (u & 1));
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int k0 = 64 * wv; k0 < a.K; k0 += 32 * W * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[i][b] = mfma16t<F16>(s[u].w[i], s[u].x[b], acc[i][b]);
        // (a load moved in front of the products gets other registers, and copies that wait for it)
        __builtin_amdgcn_sched_barrier(0);
        s[u] = load(k0 + 32 * W * U + 64 * W * (u >> 1) + 32 * (u & 1));  // (past the end: nothing)
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) red(wv, i, b)[lane] = acc[i][b];
    __syncthreads();
    for (int o = threadIdx.x; o < kTM * (RP / 4); o += 64 * W) {  // four ranks of a token
      const int row = o % kTM, c = o / kTM;
      f32x4 v = {};
      if (4 * c < a.r)  // (a padding rank: 0, also where x is infinite and 0 * x is not)
#pragma unroll
        for (int w = 0; w < W; ++w) v += red(w, c >> 2, row >> 4)[16 * (c & 3) + (row & 15)];
      f32x4 part[3];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Parts first = cut_bf16(v[i]), second = cut_bf16(first.rest);
        part[0][i] = first.high;
        part[1][i] = second.high;
        part[2][i] = second.rest;
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<u32x2*>(&parts[k][row][4 * c]) = u32x2{pair_bf16(part[k][0], part[k][1]), pair_bf16(part[k][2], part[k][3])};
    }
    __syncthreads();
  }
  const float scale = none ? 0.0f : a.scale ? a.scale[t.e] : 1.0f;
  auto chunk = [&](const Chunk& k, int c) {
    f32x4 d[4][NB] = {};
    if (!none) {
#pragma unroll
      for (int s = 0; s < RP / 32; ++s) {
        u32x4 v[3][NB];
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
          for (int b = 0; b < NB; ++b) v[q][b] = *reinterpret_cast<const u32x4*>(&parts[q][16 * b + col][32 * s + 8 * quad]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          constexpr int BP = F16 ? 2 : 1;
          u32x4 w[BP];
          split_b<F16>(k.b[s][i], w);
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int x = BP - 1; x >= 0; --x)
#pragma unroll
              for (int b = 0; b < NB; ++b) d[i][b] = mfma16t<false>(w[x], v[q][b], d[i][b]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // [16 tokens][64 channels] fp32, chunk k of 16 bytes of row r at place k ^ r
      f32x4* const at = lds + wv * 256;
#pragma unroll
      for (int i = 0; i < 4; ++i) at[col * 16 + ((4 * i + quad) ^ col)] = d[i][b];
#pragma unroll
      for (int i = b * (16 / RI); i < (b + 1) * (16 / RI); ++i) {
        const int r = RI * i - 16 * b + lane / LR, ch = 64 * c + V * (lane % LR);
        f32x4 v[V / 4];
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          v[q] = at[r * 16 + ((V / 4 * (lane % LR) + q) ^ r)];
          if constexpr (F16) v[q] *= 1.0f / kScaleB;
        }
        u32x4 o = k.y[i];
        if (!none) {
          if constexpr (YT == 1) {
            f32x4 y = __builtin_bit_cast(f32x4, o);
#pragma unroll
            for (int q = 0; q < 4; ++q) y[q] = __builtin_fmaf(scale, v[0][q], y[q]);
            o = __builtin_bit_cast(u32x4, y);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t x = o[q];
              const float lo = widen16<YT == 2>((uint16_t)(x & 0xFFFFu)), hi = widen16<YT == 2>((uint16_t)(x >> 16));
              o[q] = pack16x2<YT == 2>(__builtin_fmaf(scale, v[q >> 1][2 * (q & 1)], lo), __builtin_fmaf(scale, v[q >> 1][2 * (q & 1) + 1], hi));
            }
          }
        }
        if (r0 + RI * i + lane / LR < t.s1 && ch < a.N)
          *reinterpret_cast<u32x4*>(static_cast<char*>(a.out) + ((size_t)row_tok[i] * a.N + ch) * ES) = o;
      }
    }
  };
  int c = c0 + wv;
  for (; c + W * (2 * D - 1) < c1; c += W * D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      chunk(ring[u], c + W * u);
      __builtin_amdgcn_sched_barrier(0);
      ring[u] = fetch(c + W * (D + u));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // The last 2 D - 1 at most, apart: branches around the loop's loads would cost its waits
  // their counts (4096 tokens: 4 %), loads of chunks that nobody uses 32 tokens 8 %.
#pragma unroll
  for (int u = 0; u < 2 * D - 1; ++u) {
    if (c + W * u >= c1) return;
    chunk(ring[u % D], c + W * u);
    if (u + D < 2 * D - 1 && c + W * (u + D) < c1) ring[u] = fetch(c + W * (u + D));
  }
}

template <bool F16, int YT, int NR>
int launch_kernel(AdapterK p, hipStream_t s) {
  // One partial tile per adapter that has tokens, and one of the tokens without; the
  // channels are split over workgroups, each with the first product of its own, until the
  // chip is full.
  const int64_t tiles = (int64_t)p.a.T / (16 * token_tiles(NR)) + (p.a.n < p.a.T ? p.a.n : p.a.T) + 1;
  const int64_t want = (kWorkgroups + tiles - 1) / tiles, most = (p.n_chunk + waves(NR) - 1) / waves(NR);
  const int n_nb = (int)(want < most ? want : most);
  p.per_wg = (p.n_chunk + n_nb - 1) / n_nb;
  p.n_nb = (p.n_chunk + p.per_wg - 1) / p.per_wg;
  // (fewer than 2^21 workgroups: T < 2^24, and more than one a tile only up to 512 of them)
  hipLaunchKernelGGL((adapter_kernel<F16, YT, NR>), dim3((unsigned)(tiles * p.n_nb)), dim3(64 * waves(NR)), 0, s, p);
  return (int)hipGetLastError();
}
template <bool F16, int YT>
int launch_rank(const AdapterK& p, hipStream_t s) {
  return p.a.r <= 16 ? launch_kernel<F16, YT, 1>(p, s) : p.a.r <= 32 ? launch_kernel<F16, YT, 2>(p, s)
         : p.a.r <= 64 ? launch_kernel<F16, YT, 4>(p, s) : launch_kernel<F16, YT, 8>(p, s);
}
template <bool F16>
int launch_typed(const AdapterK& p, hipStream_t s) {
  return p.a.y_dtype == 1 ? launch_rank<F16, 1>(p, s) : p.a.y_dtype == 2 ? launch_rank<F16, 2>(p, s) : launch_rank<F16, 0>(p, s);
}
}  // namespace

int launch_adapter_add(const AdapterArgs& a, void* stream) {
  const AdapterK p{a, (a.N + 63) / 64, 0, 0};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return a.dtype == 2 ? launch_typed<true>(p, s) : launch_typed<false>(p, s);
}

}  // namespace moe
