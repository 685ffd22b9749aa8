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

// ------------------------------------------------------------ tiles of 256 x 256
// out[b][a] = sum_k P[a][k] Q[b][k]: a runs along the output's rows (contiguous),
// b over them.
//   forward  a: channels (SwiGLU: 128 gate and the matching 128 up channels), b: rows, k: inputs
//   rows     a: inputs, b: rows, k: channels
//   weights  a: inputs, b: channels, k: the segment's rows
// P and Q go through two LDS stages of 64 k, filled by LDS-DMA.  An operand whose
// k lie next to each other in memory ("direct") is kept [256][64], one whose a or
// b do [64][256], read back transposed (ds_read_b64_tr_b16).
typedef short s16x4 __attribute__((ext_vector_type(4)));
constexpr int kStage = 65536;   // bytes: P, then Q
constexpr uint32_t kOut = ~0u;  // a buffer offset past any buffer: reads zero

// [256][64] of 16 bits in 16-byte chunks, 8 a row: chunk c of row r at place c ^ swz(r).
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

struct Tile {
  int e, ab, b0, s0, s1;  // expert, a block, first b; the segment's rows (weights: the sum's)
};

template <bool F16, int MODE, bool GATHER, bool GLU, int NB>
__device__ __forceinline__ void tile_body(const GemmK& p, const Tile& c, int epi, char* sA, char* sB) {
  constexpr bool PT = MODE != kForward, QT = MODE == kWeights;  // transposed operands
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wa = wv & 3, wb = wv >> 2, half = lane >> 5, col = lane & 31;
  const int I = p.N / 2;
  const int red = MODE == kForward ? p.K : MODE == kRows ? p.N : c.s1 - c.s0;
  const int na = MODE == kForward ? p.N : p.K;  // a's extent (and a transposed P's row length)

  // This lane's part of the wavefront's DMAs: 4 of P, NB of Q (4 transposed).
  constexpr int QD = QT ? 4 : NB;
  uint32_t po[4], qo[QD];
  int pk[2], qk[2];  // direct operands: first k of the lane's chunk, DMAs of even and odd number
  const uint16_t* pbase;  // of step 0
  const uint16_t* qbase;
  uint32_t pbytes = 0, qbytes = 0;
  int src[4];
  auto pair_row = [&](int i, int step) {  // gathered P: grouped row of DMA i's lane
    return min(c.s0 + 64 * step + 2 * (4 * wv + i) + (lane >> 5), c.s1 - 1);
  };
  if constexpr (PT) {
    const int k2 = lane >> 5, s16 = lane & 31;  // row of the DMA's two, 16-byte place in it
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 2 * (4 * wv + i) + k2;
      const int ch = 256 * c.ab + 8 * ((((s16 >> 1) ^ (k & 3)) << 1) + (s16 & 1));
      po[i] = ch < na ? (GATHER ? (uint32_t)ch : (uint32_t)k * (uint32_t)na + ch) * 2 : kOut;
    }
    pbase = MODE == kRows ? p.w + (size_t)c.e * p.N * p.K : GATHER ? p.a : p.a + (size_t)c.s0 * p.K;
    if constexpr (GATHER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) src[i] = red > 0 ? p.gather[pair_row(i, 0)] : 0;
      pbytes = (uint32_t)((size_t)p.A_rows * p.K * 2);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = 4 * wv + i, r = 8 * idx + (lane >> 3), ck = (lane & 7) ^ swz(r);
      if (i < 2) pk[i] = 8 * ck;
      int ch, end = p.N;
      if constexpr (GLU) {
        // rows 64w .. 64w + 31 are gate channels of wavefront column w, 64w + 32 .. 64w + 63 their up channels
        const int x = 128 * c.ab + 32 * (r >> 6) + (r & 31);
        ch = r & 32 ? I + x : x;
        end = r & 32 ? p.N : I;
      } else {
        ch = 256 * c.ab + r;
      }
      po[i] = ch < end ? ((uint32_t)ch * (uint32_t)p.K + 8 * ck) * 2 : kOut;
    }
    pbase = p.w + (size_t)c.e * p.N * p.K;
    pbytes = (uint32_t)((size_t)p.N * p.K * 2);
  }
  if constexpr (QT) {
    const int k2 = lane >> 5, s16 = lane & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 2 * (4 * wv + i) + k2;
      const int ch = c.b0 + 8 * ((((s16 >> 1) ^ (k & 3)) << 1) + (s16 & 1));
      qo[i] = ch < p.N ? ((uint32_t)k * (uint32_t)p.N + ch) * 2 : kOut;
    }
    qbase = p.dy + (size_t)c.s0 * p.N;
  } else {
    const int ld = MODE == kForward ? p.K : p.N;
    const bool gather = MODE == kForward && p.gather;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int idx = NB * wv + i, r = 8 * idx + (lane >> 3), ck = (lane & 7) ^ swz(r);
      if (i < 2) qk[i] = 8 * ck;
      const int row = c.b0 + r;
      uint32_t from = r;
      if (gather) from = source_row(p, min(row, c.s1 - 1));
      qo[i] = row < c.s1 ? (from * (uint32_t)ld + 8 * ck) * 2 : kOut;
    }
    qbase = MODE == kForward ? (gather ? p.a : p.a + (size_t)c.b0 * ld) : p.dy + (size_t)c.b0 * ld;
    qbytes = gather ? (uint32_t)((size_t)p.A_rows * ld * 2) : (uint32_t)((size_t)min(c.s1 - c.b0, 256) * ld * 2);
  }
  const int n = (red + 63) >> 6;

  // DMAs of step st into a stage; past the sum's end zeros.
  auto issue = [&](char* stage, int st) {
    const int left = red - 64 * st;  // k of this step and later ones
    // (as a scalar: the compiler clamps on the vector side, and would loop over the lanes for the descriptor)
    const uint32_t rows = (uint32_t)__builtin_amdgcn_readfirstlane(max(min(left, 64), 0));
    const uint32_t adv = (uint32_t)min(st, n - 1) * 128u;
    if constexpr (PT) {
      if constexpr (GATHER) {
        const rsrc_t pr = make_rsrc(pbase, pbytes);
        uint32_t off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = min(max(p.div(src[i]), 0), p.A_rows - 1);
          const int k = 2 * (4 * wv + i) + (lane >> 5);
          off[i] = k < left && po[i] != kOut ? (uint32_t)row * (uint32_t)(2 * p.K) + po[i] : kOut;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) src[i] = p.gather[pair_row(i, st + 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(pr, (__attribute__((address_space(3))) void*)(stage + (4 * wv + i) * 1024), 16, off[i], 0, 0, 0);
      } else {
        const uint32_t row = 2u * (uint32_t)na;  // bytes
        const rsrc_t pr = make_rsrc(pbase + (size_t)(64 * st) * na, rows * row);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(pr, (__attribute__((address_space(3))) void*)(stage + (4 * wv + i) * 1024), 16, po[i], 0, 0, 0);
      }
    } else {
      const rsrc_t pr = make_rsrc(pbase, pbytes);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(pr, (__attribute__((address_space(3))) void*)(stage + (4 * wv + i) * 1024), 16,
                                                 pk[i & 1] < left ? po[i] : kOut, adv, 0, 0);
    }
    if constexpr (QT) {
      const rsrc_t qr = make_rsrc(qbase + (size_t)(64 * st) * p.N, rows * (2u * (uint32_t)p.N));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(qr, (__attribute__((address_space(3))) void*)(stage + 32768 + (4 * wv + i) * 1024), 16, qo[i], 0, 0, 0);
    } else {
      const rsrc_t qr = make_rsrc(qbase, qbytes);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(qr, (__attribute__((address_space(3))) void*)(stage + 32768 + (NB * wv + i) * 1024), 16,
                                                 qk[i & 1] < left ? qo[i] : kOut, adv, 0, 0);
    }
  };

  // Fragments of 16 k: 2 of P (32 a each), NB of Q.
  struct Frags {
    u32x4 p[2], q[NB];
  };
  auto read_direct = [&](const char* at, int row, int s) {
    return *reinterpret_cast<const u32x4*>(at + row * 128 + (((2 * s + half) ^ swz(row)) << 4));
  };
  auto read_trans = [&](const char* at, int x0, int s) {  // 16 columns from x0, 16 from x0 + 64
    const int j = (lane >> 2) & 3, u = (x0 >> 4) + 4 * ((lane >> 4) & 1);
    const char* from = at + (16 * s + 8 * half + j) * 512 + ((u ^ j) << 5) + ((lane & 3) << 3);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(from));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(from + 2048));
    const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
    return u32x4{l[0], l[1], h[0], h[1]};
  };
  auto read = [&](const char* stage, int s) {
    Frags f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      f.p[t] = PT ? read_trans(stage, 128 * (wa >> 1) + 32 * (wa & 1) + 16 * t, s) : read_direct(stage, 64 * wa + 32 * t + col, s);
#pragma unroll
    for (int j = 0; j < NB; ++j)
      f.q[j] = QT ? read_trans(stage + 32768, 128 * (j >> 1) + 32 * (j & 1) + 16 * wb, s) : read_direct(stage + 32768, 64 * j + 32 * wb + col, s);
    return f;
  };
  f32x16 acc[2][NB] = {};
  auto mul = [&](const Frags& f) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[t][j] = mfma32t<F16>(f.p[t], f.q[j], acc[t][j]);
    __builtin_amdgcn_s_setprio(0);
  };
  // Every wavefront's reads of a stage are done and the other stage's DMAs landed.
  auto ready = [&] {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt 0, lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  if (n > 0) {
    issue(sA, 0);
    ready();
    issue(sB, 1);
    Frags f = read(sA, 0), g;
    for (int st = 0; st < n; st += 2) {
      g = read(sA, 1);
      mul(f);
      f = read(sA, 2);
      mul(g);
      g = read(sA, 3);
      mul(f);
      ready();
      issue(sA, st + 2);
      f = read(sB, 0);
      mul(g);
      g = read(sB, 1);
      mul(f);
      f = read(sB, 2);
      mul(g);
      g = read(sB, 3);
      mul(f);
      ready();
      issue(sB, st + 3);
      f = read(sA, 0);
      mul(g);
    }
    ready();
  }

  // Epilogue: a wavefront's 32 b x 64 a at a time through 8 KB of LDS, so that
  // neighbouring lanes store 128 bytes and more in a row.  Lane (half, col) holds
  // b = col and of tile t a = 32t + 8g + 4*half + 0..3 in registers 4g ...
  char* const eb = sA + wv * 8192;
  const int a0 = GLU && MODE == kForward ? 128 * c.ab + 32 * wa : PT ? 256 * c.ab + 128 * (wa >> 1) + 32 * (wa & 1) : 256 * c.ab + 64 * wa;
  // channel of place x of the wavefront's 64
  auto a_of = [&](int x) { return a0 + (PT ? (x & 31) + 64 * (x >> 5) : x); };
  // the places of 8 channels (fp32: 4) of tile t, register group g
  auto chunk16 = [&](int t, int g) { return PT ? 4 * (g >> 1) + 2 * t + (g & 1) : 4 * t + g; };
  auto put16 = [&](int ck, float v0, float v1, float v2, float v3, bool f16) {  // 8 chunks a row
    const u32x2 d = f16 ? u32x2{pack16x2<true>(v0, v1), pack16x2<true>(v2, v3)} : u32x2{pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)};
    *reinterpret_cast<u32x2*>(eb + col * 128 + ((ck ^ (col & 7)) << 4) + 8 * half) = d;
  };
  auto get16 = [&](int r, int ck) { return *reinterpret_cast<const u32x4*>(eb + r * 128 + ((ck ^ (r & 7)) << 4)); };
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int b = c.b0 + (QT ? 128 * (j >> 1) + 32 * (j & 1) + 16 * wb : 64 * j + 32 * wb);  // of the 32's first row
    auto b_of = [&](int r) { return b + (QT ? (r & 15) + 64 * (r >> 4) : r); };
    const int bend = MODE == kWeights ? p.N : c.s1;
    const size_t out0 = MODE == kWeights ? (size_t)c.e * p.N : 0;
    if constexpr (GLU && MODE == kForward) {
      if (p.pre_out) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            put16(4 * t + g, acc[t][j][4 * g], acc[t][j][4 * g + 1], acc[t][j][4 * g + 2], acc[t][j][4 * g + 3], F16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 3), ck = lane & 7, ch = a0 + 8 * (ck & 3);
          const u32x4 v = get16(r, ck);
          if (b_of(r) < bend && ch < I)
            *reinterpret_cast<u32x4*>(p.pre_out + (size_t)b_of(r) * p.N + (ck >> 2 ? I : 0) + ch) = v;
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = acc[0][j][4 * g + i];
          h[i] = x * __builtin_amdgcn_rcpf(1.0f + __expf(-x)) * acc[1][j][4 * g + i];
        }
        put16(g, h[0], h[1], h[2], h[3], F16);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * i + (lane >> 2), ck = lane & 3;
        const u32x4 v = get16(r, ck);
        if (b_of(r) < bend && a0 + 8 * ck < I)
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + (size_t)b_of(r) * I + a0 + 8 * ck) = v;
      }
    } else if (GLU || epi == kEpiF32) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int ck = 2 * chunk16(t, g) + half;  // 16 chunks a row
          *reinterpret_cast<f32x4*>(eb + col * 256 + ((ck ^ (col & 15)) << 4)) =
              f32x4{acc[t][j][4 * g], acc[t][j][4 * g + 1], acc[t][j][4 * g + 2], acc[t][j][4 * g + 3]};
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 4), ck = lane & 15, ch = a_of(4 * ck);
        const f32x4 v = *reinterpret_cast<const f32x4*>(eb + r * 256 + ((ck ^ (r & 15)) << 4));
        if (b_of(r) >= bend || ch >= na) continue;
        if constexpr (GLU) {
          const size_t at = (size_t)b_of(r) * 2 * p.K + ch;
          const u32x2 gv = *reinterpret_cast<const u32x2*>(p.pre_in + at), uv = *reinterpret_cast<const u32x2*>(p.pre_in + at + p.K);
          float dg[4], du[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t gw = gv[q >> 1], uw = uv[q >> 1];
            const float g = widen16<F16>((uint16_t)(q & 1 ? gw >> 16 : gw & 0xFFFFu));
            const float u = widen16<F16>((uint16_t)(q & 1 ? uw >> 16 : uw & 0xFFFFu));
            const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
            dg[q] = v[q] * u * s * (1.0f + g * (1.0f - s));
            du[q] = v[q] * g * s;
          }
          uint16_t* const o = static_cast<uint16_t*>(p.out) + at;
          *reinterpret_cast<u32x2*>(o) = u32x2{pack16x2<F16>(dg[0], dg[1]), pack16x2<F16>(dg[2], dg[3])};
          *reinterpret_cast<u32x2*>(o + p.K) = u32x2{pack16x2<F16>(du[0], du[1]), pack16x2<F16>(du[2], du[3])};
        } else {
          *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + (out0 + b_of(r)) * na + ch) = v;
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          put16(chunk16(t, g), acc[t][j][4 * g], acc[t][j][4 * g + 1], acc[t][j][4 * g + 2], acc[t][j][4 * g + 3], epi == kEpiF16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 3), ck = lane & 7, ch = a_of(8 * ck);
        const u32x4 v = get16(r, ck);
        if (b_of(r) < bend && ch < na)
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + (out0 + b_of(r)) * na + ch) = v;
      }
    }
  }
}

// Tiles in an order that neighbours share operands in an XCD's L2: workgroups are
// dealt to the 8 XCDs in turn, each takes a contiguous range; within a segment in
// groups of 8 row tiles by a block.
__device__ __forceinline__ bool xcd_index(int wgs, int& idx) {
  const int per = (wgs + 7) >> 3;
  idx = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  return ((int)blockIdx.x >> 3) < per && idx < wgs;
}
__device__ __forceinline__ void grouped_order(int idx, int tiles, int n_ab, int& tile, int& ab) {
  const int g = idx / (8 * n_ab), gm = min(8, tiles - 8 * g), in = idx - g * 8 * n_ab;
  ab = in / gm;
  tile = 8 * g + in % gm;
}

template <bool F16, int MODE, bool GATHER, bool GLU>
__global__ __launch_bounds__(512, 2) void tile256_kernel(GemmK p, int epi, int n_ab, int n_bb) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __attribute__((aligned(1024))) char sA[kStage], sB[kStage];
  Tile c;
  int idx, tile;
  if constexpr (MODE == kWeights) {
    if (!xcd_index(p.E * n_ab * n_bb, idx)) return;
    c.e = idx / (n_ab * n_bb);
    grouped_order(idx % (n_ab * n_bb), n_bb, n_ab, tile, c.ab);
    c.b0 = 256 * tile;
    c.s0 = c.s1 = 0;
    if (p.M_total > 0) segment_rows(p.seg, c.e, p.M_total, c.s0, c.s1);
    tile_body<F16, MODE, GATHER, GLU, 4>(p, c, epi, sA, sB);
  } else {
    if (!xcd_index(count_tiles<256>(p.seg, p.E, p.M_total) * n_ab, idx)) return;
    RowTile t;
    if (!find_tile<256>(p.seg, p.E, p.M_total, n_ab, idx, t)) return;
    grouped_order(idx, t.tiles, n_ab, tile, c.ab);
    c.e = t.e;
    c.b0 = t.r0 + 256 * tile;
    c.s0 = t.r0;
    c.s1 = t.s1;
    const int left = c.s1 - c.b0;
    if (left <= 64) tile_body<F16, MODE, GATHER, GLU, 1>(p, c, epi, sA, sB);
    else if (left <= 128) tile_body<F16, MODE, GATHER, GLU, 2>(p, c, epi, sA, sB);
    else if (left <= 192) tile_body<F16, MODE, GATHER, GLU, 3>(p, c, epi, sA, sB);
    else tile_body<F16, MODE, GATHER, GLU, 4>(p, c, epi, sA, sB);
  }
#endif
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

template <bool F16, int MODE, bool GATHER, bool GLU>
int launch256(const Gemm16Args& a, hipStream_t s) {
  const int na = MODE == kForward ? (GLU ? a.N : a.N) : a.K, n_ab = (na + 255) / 256, n_bb = (a.N + 255) / 256;
  const int64_t wgs = ((MODE == kWeights ? (int64_t)a.E * n_bb : row_tiles(a.M_total, a.E, 256)) * n_ab + 7) / 8 * 8;
  if (wgs >= ((int64_t)1 << 22)) return (int)hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((tile256_kernel<F16, MODE, GATHER, GLU>), dim3((unsigned)wgs), dim3(512), 0, s, kernel_args(a), a.epilogue, n_ab, n_bb);
  return (int)hipGetLastError();
}
template <int MODE, bool GATHER, bool GLU>
int launch256t(const Gemm16Args& a, void* s) {
  return a.dtype == 2 ? launch256<true, MODE, GATHER, GLU>(a, static_cast<hipStream_t>(s)) : launch256<false, MODE, GATHER, GLU>(a, static_cast<hipStream_t>(s));
}
}  // namespace

int launch_gemm16(const Gemm16Args& a, void* stream) {
  if (a.kernel == 9 || a.kernel == 0)
    return a.epilogue == kEpiSwiglu ? launch256t<kForward, false, true>(a, stream) : launch256t<kForward, false, false>(a, stream);
  const int n_ab = a.epilogue == kEpiSwiglu ? (a.N / 2 + 31) / 32 : (a.N + 63) / 64;
  return launch_rowwise<kForward>(a, n_ab, static_cast<hipStream_t>(stream));
}
int launch_gemm16_grad_rows(const Gemm16Args& a, void* stream) {
  if (a.kernel == 9 || a.kernel == 0)
    return a.epilogue == kEpiSwigluGrad ? launch256t<kRows, false, true>(a, stream) : launch256t<kRows, false, false>(a, stream);
  return launch_rowwise<kRows>(a, (a.K + 63) / 64, static_cast<hipStream_t>(stream));
}
size_t gemm16_grad_weights_workspace_bytes(int E, int N, int K, int M_total, int kernel) { return 0; }
int launch_gemm16_grad_weights(const Gemm16Args& a, void* stream) {
  if (a.kernel == 9 || a.kernel == 0)
    return a.gather ? launch256t<kWeights, true, false>(a, stream) : launch256t<kWeights, false, false>(a, stream);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((a.K + 63) / 64, (a.N + 63) / 64, a.E);
  if (grid.y > 65535) return (int)hipErrorInvalidConfiguration;
  if (a.dtype == 2) hipLaunchKernelGGL((gemm16_kernel<true, kWeights>), grid, dim3(256), 0, s, kernel_args(a), a.epilogue, 0);
  else hipLaunchKernelGGL((gemm16_kernel<false, kWeights>), grid, dim3(256), 0, s, kernel_args(a), a.epilogue, 0);
  return (int)hipGetLastError();
}

}  // namespace moe
