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
// The instruction aligns its 64 products before it adds them: measured over
// random and adversarial operands, its result is off by at most 2^-11 of the
// largest product with e4m3 rows and 2^-20 with e2m1 rows; the sums over K are
// kept in fp32.  Registers alone, random operands: 3.5 to 3.8 PF with e4m3 rows,
// 6.5 PF with e2m1 rows (the power limit; 5.1 and 9.6 PF on zeros).
#include <type_traits>

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
  uint32_t k_mul;  // pair / k = (pair * k_mul) >> (31 + k_shift), 0 <= pair < 2^31
  int k_shift;
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
// Weight scale in byte WB of ws, activation scale in byte AB of as (shifted by the
// lane's half beforehand).
template <int AF, int WB, int AB>
__device__ __forceinline__ f32x16 mx_mfma(i32x8 w, i32x8 x, f32x16 c, uint32_t ws, uint32_t as) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 4, AF == kE4M3 ? 0 : 4, WB, (int)ws, AB, (int)as);
}

// Fast exponential and reciprocal, as in the library's other SwiGLU epilogues.  The
// exponential's argument is off by 1.5 |g| 2^-24 (log2 e and the product rounded),
// it, the sum, the reciprocal and the products by 7 * 2^-24 together, relative: below
// 2^-21 for g >= 0, where the sum damps the first term, (1.5 |g| + 7) 2^-24 for g < 0
// (2^-19 at -16); below -88 the exponential is infinite and the result 0, as in
// float32 arithmetic.  What follows rounds to bf16 (2^-9) or an MX element (2^-4 or
// more).
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Segment e's rows, clamped to the buffers.
__device__ __forceinline__ void segment(const MxK& p, int e, int& s0, int& s1) {
  s0 = min(max(p.seg[e], 0), p.M_total);
  s1 = min(max(p.seg[e + 1], s0), p.M_total);
}
__device__ __forceinline__ int pair_token(const MxK& p, int pair) {
  return (int)(((uint64_t)(uint32_t)pair * p.k_mul) >> (31 + p.k_shift));
}
__device__ __forceinline__ int source_row(const MxK& p, int row) {
  const int r = p.gather ? pair_token(p, p.gather[row]) : row;
  return min(max(r, 0), p.A_rows - 1);
}

// -------------------------------------------------------- few rows per expert
// A workgroup takes 64 output channels of one expert (SwiGLU: 32 gate and the
// matching 32 up channels) and 32 of the expert's rows (every gridDim.z-th
// group of 32); its NW wavefronts split K and add their sums through LDS.  Weights
// and activations go from memory straight to the operand registers: each weight
// byte is read once per 32 rows.  Bound by the weights' bytes (8 experts of 4096 x
// 14336, 32 rows in all: 249 MB in 47 us, 5.3 TB/s) and, with few workgroups, by the
// latency of a wavefront's K / 4 range: 8.1 us for 8 experts of 2048 x 2048.
template <int AF>
struct SmallBlock {  // operands of one K block of 128
  u32x4 w[2][2];     // [channel tile][step]
  u32x4 x[2][AF == kE4M3 ? 2 : 1];
  uint32_t ws[2], as;
};

template <int AF, int EPI>
__global__ __launch_bounds__(256, 3) void mx_small_kernel(MxK p) {
  constexpr int NW = 4;  // 8 wavefronts were slower where the chip has work (8 experts, 64 rows, 2048 x 2048: 15 for 12 us)
  constexpr int D = 2;   // K blocks in flight
  __shared__ float red[NW][2][16][64];
  __shared__ uint32_t amx[4][32];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int e = blockIdx.y;
  int s0, s1;
  segment(p, e, s0, s1);
  if (s0 + 32 * (int)blockIdx.z >= s1) return;

  const int NT = p.N >> 5, KB = p.K >> 7, KC = (p.K + 255) >> 8;
  const int t0 = is_swiglu(EPI) ? blockIdx.x : 2 * blockIdx.x;
  const int t1 = is_swiglu(EPI) ? NT / 2 + blockIdx.x : min(2 * (int)blockIdx.x + 1, NT - 1);
  const size_t tile_bytes = (size_t)KC * 4096;  // 32 channels of e2m1, K in whole chunks of 256
  const rsrc_t wr0 = make_rsrc(p.wc + ((size_t)e * NT + t0) * tile_bytes, (uint32_t)tile_bytes);
  const rsrc_t wr1 = make_rsrc(p.wc + ((size_t)e * NT + t1) * tile_bytes, (uint32_t)tile_bytes);
  const rsrc_t sr0 = make_rsrc(p.wsc + ((size_t)e * NT + t0) * KC * 256, KC * 256);
  const rsrc_t sr1 = make_rsrc(p.wsc + ((size_t)e * NT + t1) * KC * 256, KC * 256);
  const rsrc_t ar = make_rsrc(p.a, p.a_bytes);
  const rsrc_t asr = make_rsrc(p.as, p.as_bytes);
  const int kb0 = KB * wv / NW, kb1 = KB * (wv + 1) / NW;
  constexpr int kXB = AF == kE4M3 ? 128 : 64;  // activation bytes of a K block

  for (int r0 = s0 + 32 * (int)blockIdx.z; r0 < s1; r0 += 32 * (int)gridDim.z) {
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
          const SmallBlock<AF>& b = q[i];
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
          if (kb + i + D < kb1) q[i] = load(kb + i + D);
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
    {
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
          const uint32_t m = absmax_bits(h);
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
                                       : pack_f16x2(v[t][2 * i], v[t][2 * i + 1]);
              *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + o) = b;
            }
          }
        }
      }
    }
    __syncthreads();
    if constexpr (EPI == kEpiSwigluE4M3 || EPI == kEpiSwigluE2M1) {
      if (row < s1) {
        constexpr int F = EPI == kEpiSwigluE4M3 ? kE4M3 : kE2M1;
        const int I = p.N / 2, ch = 8 * wv + 4 * half;
        uint32_t m = amx[0][col];
#pragma unroll
        for (int w = 1; w < 4; ++w) m = m > amx[w][col] ? m : amx[w][col];
        const bool bad = mx_not_finite(m);
        const int pe = mx_exponent<F>(m);
        const uint32_t d = bad ? 0u : mx_pack4<F>(v[0][0], v[0][1], v[0][2], v[0][3], mx_scale(pe));
        const size_t o = (size_t)row * I + 32 * t0 + ch;
        if constexpr (F == kE4M3)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + o) = d;
        else
          *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.out) + o / 2) = (uint16_t)d;
        if (wv == 0 && half == 0) p.out_scales[(size_t)row * (I >> 5) + t0] = bad ? (uint8_t)255 : (uint8_t)(pe + 127);
      }
      __syncthreads();  // amx is written again for the next rows
    }
  }
}

// ------------------------------------------------------- many rows per expert
// A workgroup of 4 wavefronts takes TM rows of one expert and 8 channel tiles
// (256 channels; SwiGLU: 128 gate and the matching 128 up channels), a
// wavefront all TM rows and 2 of the tiles (a gate and its up tile).  Rows and
// their scales go through two LDS stages of 256 inputs (128 of e4m3 rows in
// 128-row tiles) filled by LDS-DMA and shared by the wavefronts; weights, which
// only one wavefront uses, straight into its registers.  Workgroups share a CU (2 of
// 128 rows, 3 of 64), so one multiplies while another waits at its barrier.
//
// Measured with weights from memory (sets of 1 GB and more in turn), 65536 rows over
// 64 experts of 2048 x 2048, SwiGLU to MX rows: e4m3 rows 227 us, 2.4 PF (the clock
// under this load bounds it: registers alone reach 3.5); e2m1 rows 164 us, 3.4 PF
// (the loads' way through the caches).  512 tokens x 2 of 8 experts, 4096 x 14336,
// e2m1 rows: 74 to 78 us, of which 53 are the weights' bytes.
// Variants below were compared with the same weights call after call, which stay in
// the 256 MB cache where they fit, and are faster by that.
// Stages of 256 e2m1 inputs for 128: 158 -> 147 us (above; loads are under way twice
// as long).  Of 256 e4m3 inputs: 64-row tiles 914 -> 853 us (8192 rows over 8 experts
// of 28672 x 4096), 19.4 -> 15.4 (192 rows each, 16 of 448 x 4096; one register of
// the SwiGLU and fp32 kernels is spilled over the loop); 128-row tiles, short of
// registers with them, 218 -> 223 and 46 -> 50 (above, 1280 x 8).
//
// Each XCD (workgroups are dealt to the 8 of them in turn) takes a contiguous
// range of tiles, so that the weights and rows its CUs share stay in its L2.
//
// Rows in LDS: 16-byte chunks, chunk c of row r at place c ^ swizzle(r), so that
// the lanes of a fragment read (32 rows, one chunk) fall on different banks,
// whether 8 or 16 of them are served at once.  A DMA writes 64 chunks in a row,
// so the lanes fetch them in swizzled order.
template <int XC>
__device__ __forceinline__ int swizzle(int row) {
  return XC == 16 ? ((row >> 1) & 7) | ((row & 1) << 3) : (row & 7) ^ ((row >> 3) & 1);
}
// 16-byte chunks of a row in a stage of the TM-row kernel.
constexpr int stage_chunks(int af, int tm) { return af == kE4M3 && tm == 64 ? 16 : 8; }

// Tiles (row tile, channel block) are numbered expert by expert, within an
// expert in groups of 8 row tiles by channel block.
struct Tile {
  int e, r0, s1, nb;
};
// Inclusive sum over the wavefront's lanes (DPP: shifts within rows of 16, then
// row broadcasts).
__device__ __forceinline__ int wave_scan(int v) {
#define MOE_STEP(CTRL, RMASK) v += __builtin_amdgcn_update_dpp(0, v, CTRL, RMASK, 0xF, false);
  MOE_STEP(0x111, 0xF) MOE_STEP(0x112, 0xF) MOE_STEP(0x114, 0xF) MOE_STEP(0x118, 0xF)
  MOE_STEP(0x142, 0xA) MOE_STEP(0x143, 0xC)
#undef MOE_STEP
  return v;
}
template <int TM>
__device__ __forceinline__ int row_tiles(const MxK& p, int e, int& s0, int& s1) {
  s0 = s1 = 0;
  if (e < p.E) segment(p, e, s0, s1);
  return (s1 - s0 + TM - 1) / TM;
}
// This workgroup's tile (false: none).  64 segments at a time, one per lane; with
// more the first pass counts the tiles and a second one finds it.
template <int TM>
__device__ __forceinline__ bool own_tile(const MxK& p, int n_nb, Tile& t) {
  const int lane = threadIdx.x & 63;
  int s0, s1;
  int n = row_tiles<TM>(p, lane, s0, s1);
  int end = wave_scan(n), total = __builtin_amdgcn_readlane(end, 63);
  for (int e0 = 64; e0 < p.E; e0 += 64) {
    int a, b;
    total += __builtin_amdgcn_readlane(wave_scan(row_tiles<TM>(p, e0 + lane, a, b)), 63);
  }
  const int wgs = total * n_nb, per = (wgs + 7) >> 3;
  int idx = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (((int)blockIdx.x >> 3) >= per || idx >= wgs) return false;
  int e0 = 0;
  while (true) {
    const int sum = __builtin_amdgcn_readlane(end, 63) * n_nb;
    if (idx < sum || e0 + 64 >= p.E) break;
    idx -= sum;
    e0 += 64;
    n = row_tiles<TM>(p, e0 + lane, s0, s1);
    end = wave_scan(n);
  }
  const int src = __builtin_ctzll(__ballot(idx < end * n_nb));
  const int tiles = __builtin_amdgcn_readlane(n, src);
  const int j = idx - (__builtin_amdgcn_readlane(end, src) - tiles) * n_nb;
  const int g = j / (8 * n_nb), gm = min(8, tiles - 8 * g);
  const int in = j - g * 8 * n_nb;
  t.e = e0 + src;
  t.nb = in / gm;
  t.r0 = __builtin_amdgcn_readlane(s0, src) + (8 * g + in % gm) * TM;
  t.s1 = __builtin_amdgcn_readlane(s1, src);
  return true;
}

// Exchanges halves of the wavefront: afterwards a holds (a's low half, b's low
// half) and b (a's high half, b's high half) in lanes (0..31, 32..63).
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// One tile of 32 channels x 32 tokens as the accumulator holds it (register
// 4g + i: channel 8g + 4*half + i) to row `row` of a 16-bit output, 8 channels
// (16 bytes) per lane and store.
__device__ __forceinline__ void store_tile16(const uint32_t lohi[8], uint16_t* at, int half, bool on) {
#pragma unroll
  for (int g = 0; g < 4; g += 2) {
    uint32_t a0 = lohi[2 * g], a1 = lohi[2 * g + 1], b0 = lohi[2 * g + 2], b1 = lohi[2 * g + 3];
    swap_halves(a0, b0);
    swap_halves(a1, b1);
    if (on) *reinterpret_cast<u32x4*>(at + 8 * g + 8 * half) = u32x4{a0, a1, b0, b1};
  }
}

constexpr int kEpiChunks = 256;  // 16-byte chunks of LDS per wavefront in the epilogue
// XC: 16-byte chunks of a row in a stage.
template <int AF, int EPI, int TM, int KS, int XC>
__device__ __forceinline__ void mx_tile_body(const MxK& p, const Tile& c, u32x4* x0, u32x4* x1, uint32_t* s0, uint32_t* s1,
                                             f32x4* red) {
  constexpr int SS = XC / (AF == kE4M3 ? 4 : 2);  // steps of 64 inputs in a stage
  constexpr int RT = TM / 32;                // row tiles
  constexpr int XI = TM * XC / 256;          // row DMAs per wavefront and stage
  constexpr int RW = TM == 64 ? 16 : 32;     // rows whose scales a wavefront fetches
  const int lane = threadIdx.x & 63, all = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wv = all & 3, grp = KS == 1 ? 0 : all >> 2;
  const int half = lane >> 5, col = lane & 31;
  const int NT = p.N >> 5, KB = p.K >> 7, KC = (p.K + 255) >> 8;

  // this group's chunks of 256 inputs
  const int per_group = (KC + KS - 1) / KS, c0 = grp * per_group, n = KS == 1 ? KC : min(per_group, KC - c0);
  u32x4* const eb = x0 + all * kEpiChunks;  // for the epilogue, when the stages are done with
  x0 += grp * (TM * XC);
  x1 += grp * (TM * XC);
  s0 += grp * 256;
  s1 += grp * 256;

  // this wavefront's tiles; past the last channel: tile 0, loaded and never stored
  bool valid[2];
  int tile[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int t = is_swiglu(EPI) ? 4 * c.nb + wv : 8 * c.nb + 2 * wv + u;
    valid[u] = t < (is_swiglu(EPI) ? NT / 2 : NT);
    tile[u] = (valid[u] ? t : 0) + (is_swiglu(EPI) && u ? NT / 2 : 0);
  }
  const rsrc_t ar = make_rsrc(p.a, p.a_bytes);
  const rsrc_t asr = make_rsrc(p.as, p.as_bytes);
  const rsrc_t wr = make_rsrc(p.wc + (size_t)c.e * NT * KC * 4096, (uint32_t)((size_t)NT * KC * 4096));
  const rsrc_t wsr = make_rsrc(p.wsc + (size_t)c.e * NT * KC * 256, (uint32_t)((size_t)NT * KC * 256));
  const uint32_t wo[2] = {(uint32_t)tile[0] * (uint32_t)(KC * 4096), (uint32_t)tile[1] * (uint32_t)(KC * 4096)};
  // Weights of 4 steps (256 inputs, "chunk" kc), [tile][step]; a step's are loaded
  // again as soon as it is multiplied: 3 steps ahead of their use, 2 loads each.
  u32x4 w[2][4];
  auto load_weights = [&](int kc, int j) {
#pragma unroll
    for (int u = 0; u < 2; ++u) w[u][j] = buf_x4(wr, 16 * lane, wo[u] + (c0 + kc) * 4096 + 1024 * j);
  };
  struct Scales {  // of a chunk's weights
    uint32_t w[2];
  };
  auto load_scales = [&](int kc) {
    Scales s;
#pragma unroll
    for (int u = 0; u < 2; ++u) s.w[u] = buf_x1(wsr, 4 * lane, wo[u] / 16 + (c0 + kc) * 256);
    return s;
  };
  // the weights' way does not wait for the rows' addresses
  Scales sc = load_scales(0);
#pragma unroll
  for (int j = 0; j < SS; ++j) load_weights(0, j);
  // grouped rows of this lane's DMAs, then the row whose scales it fetches; past
  // the segment's end the last row again (its column is never stored)
  int src[XI + 1];
#pragma unroll
  for (int i = 0; i < XI; ++i) src[i] = min(c.r0 + ((wv * XI + i) * 64 + lane) / XC, c.s1 - 1);
  src[XI] = min(c.r0 + RW * wv + (lane & (RW - 1)), c.s1 - 1);
  if (p.gather) {
#pragma unroll
    for (int i = 0; i < XI + 1; ++i) src[i] = p.gather[src[i]];
#pragma unroll
    for (int i = 0; i < XI + 1; ++i) src[i] = pair_token(p, src[i]);
  }
#pragma unroll
  for (int i = 0; i < XI + 1; ++i) src[i] = min(max(src[i], 0), p.A_rows - 1);
  uint32_t xo[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int at = (wv * XI + i) * 64 + lane;
    xo[i] = (uint32_t)src[i] * (uint32_t)(KB * (AF == kE4M3 ? 128 : 64)) + 16 * ((at % XC) ^ swizzle<XC>(at / XC));
  }
  uint32_t xso = (uint32_t)src[XI] * (uint32_t)(KB * 4);
  // A stage of 256 inputs is two blocks: the lanes of the second fetch the first
  // again where K ends between the two (the weights there are zeros)
  const bool high = ((lane % XC) ^ swizzle<XC>(lane / XC)) >= XC / 2, high_s = (lane / RW) & 1;
  if (SS == 4 && high_s) xso += 4;

  // XI + 1 loads of the group's stage st, rows and scales
  const int st0 = SS == 2 ? 2 * c0 : c0, last = (SS == 2 ? KB : KC) - 1;
  auto issue = [&](u32x4* xs, uint32_t* ss, int rel) {
    const int st = min(st0 + rel, last);
    const bool half_stage = SS == 4 && 2 * st + 1 == KB;
    const uint32_t back = half_stage && high ? XC * 8 : 0, back_s = half_stage && high_s ? 4 : 0;
#pragma unroll
    for (int i = 0; i < XI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, xs + (wv * XI + i) * 64, 16, xo[i] - back, st * (XC * 16), 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(asr, ss + wv * 64, 4, xso - back_s, st * (2 * SS), 0, 0);
  };
  struct Frag {  // 32 rows' values in a step (64 inputs)
    u32x4 x[AF == kE4M3 ? 2 : 1];
  };
  auto read = [&](const u32x4* xs, int S, int t) {
    Frag f;
    const int row = 32 * t + col, z = swizzle<XC>(row);
    if constexpr (AF == kE4M3) {
      f.x[0] = xs[row * XC + ((4 * S + half) ^ z)];
      f.x[1] = xs[row * XC + ((4 * S + 2 + half) ^ z)];
    } else {
      f.x[0] = xs[row * XC + ((2 * S + half) ^ z)];
    }
    return f;
  };
  struct RowScales {  // of a stage
    uint32_t x[RT][SS / 2];
  };
  auto read_scales = [&](const uint32_t* ss) {
    RowScales s;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = 32 * t + col;
#pragma unroll
      for (int h = 0; h < SS / 2; ++h) s.x[t][h] = ss[row / RW * 64 + RW * h + row % RW] >> (8 * half);
    }
    return s;
  };
  f32x16 acc[RT][2];
  Frag f[RT];
  // Step j of a chunk: multiplies f and replaces it, row tile by row tile, with
  // the next step's fragments (of stage xs; not after the last).  128-row tiles at
  // raised priority, which also keeps the compiler from moving loads into it (with
  // weights from memory: 512 tokens x 2 of 8 experts, 4096 x 14336, e2m1 rows 86 -> 78
  // us, 65536 rows 170 -> 164, e4m3 rows the same); 64-row tiles take 5 % longer with
  // it.
  auto step = [&](auto j_tag, const Scales& sc, const RowScales& xsc, auto first_tag, const u32x4* xs, auto next_tag) {
    constexpr int J = decltype(j_tag)::value, S = J % SS;
    if constexpr (TM == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      i32x8 xf;
      if constexpr (AF == kE4M3) xf = operand(f[t].x[0], f[t].x[1]);
      else xf = operand(f[t].x[0]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x16 c0 = decltype(first_tag)::value ? f32x16{} : acc[t][u];
        acc[t][u] = mx_mfma<AF, J, 2 * (J & 1)>(operand(w[u][J]), xf, c0, sc.w[u], xsc.x[t][S / 2]);
      }
      if constexpr (decltype(next_tag)::value) f[t] = read(xs, (S + 1) % SS, t);
    }
    if constexpr (TM == 128) __builtin_amdgcn_s_setprio(0);
  };
  const std::integral_constant<int, 0> zero{};
  const std::integral_constant<int, 1> one{};
  const std::integral_constant<int, 2> two{};
  const std::integral_constant<int, 3> three{};
  // Everyone's fragments of the current block have arrived, and the next block's
  // rows.  Loads complete in order: `left` newer ones, weights and their scales
  // loaded since those rows were issued, may be on their way.  At least that many
  // are (in the one-stage loop 6 of weights and 2 of scales before its first wait,
  // 10 before the others; 6 or more of weights in the two-stage loop); the
  // scheduling barriers keep them between the two.  Waiting for them too cost 3 to
  // 30 %.
  auto ready = [&](auto left_tag) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070 | decltype(left_tag)::value);  // vmcnt `left`, lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  const std::integral_constant<int, 2 * SS> weights_may_fly{};

  // At stage i's barrier nobody reads it any more and stage i + 1's rows have
  // landed: stage i + 2's are issued into the free one, then stage i's last step
  // and all but the last of stage i + 1 multiply.  No branch in the loop (a branch
  // around a load makes the compiler wait for every load in flight, an exit in
  // the middle copies the accumulators): the weights are padded with zeros to a
  // whole chunk, whose missing half multiplies them with the other half's rows.
  issue(x0, s0, 0);
  ready(zero);
  if constexpr (SS == 2) {  // two stages in a chunk
    issue(x1, s1, 1);
    __builtin_amdgcn_sched_barrier(0);
    load_weights(0, 2);
    load_weights(0, 3);
#pragma unroll
    for (int t = 0; t < RT; ++t) f[t] = read(x0, 0, t);
    RowScales xa = read_scales(s0), xb;
    step(zero, sc, xa, one, x0, one);
    int kc = 0;
    for (; kc + 1 < n; ++kc) {
      load_weights(kc + 1, 0);
      ready(weights_may_fly);
      issue(x0, s0, 2 * kc + 2);
      const Scales next = load_scales(kc + 1);
      xb = read_scales(s1);
      __builtin_amdgcn_sched_barrier(0);
      step(one, sc, xa, zero, x1, one);
      load_weights(kc + 1, 1);
      step(two, sc, xb, zero, x1, one);
      load_weights(kc + 1, 2);
      ready(weights_may_fly);
      issue(x1, s1, 2 * kc + 3);
      xa = read_scales(s0);
      __builtin_amdgcn_sched_barrier(0);
      step(three, sc, xb, zero, x0, one);
      load_weights(kc + 1, 3);
      sc = next;
      step(zero, sc, xa, zero, x0, one);
    }
    ready(zero);
    xb = read_scales(s1);
    step(one, sc, xa, zero, x1, one);
    step(two, sc, xb, zero, x1, one);
    step(three, sc, xb, zero, x1, zero);
  } else {  // one
    const int k1 = min(1, n - 1);
    issue(x1, s1, k1);
    __builtin_amdgcn_sched_barrier(0);  // the loop's first wait counts the scales' loads too
    Scales next = load_scales(k1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < RT; ++t) f[t] = read(x0, 0, t);
    RowScales xa = read_scales(s0), xb;
    step(zero, sc, xa, one, x0, one);
    load_weights(k1, 0);
    step(one, sc, xa, zero, x0, one);
    load_weights(k1, 1);
    step(two, sc, xa, zero, x0, one);
    load_weights(k1, 2);
    int kc = 0;
    for (; kc + 2 < n; kc += 2) {
      ready(weights_may_fly);
      issue(x0, s0, kc + 2);
      xb = read_scales(s1);
      __builtin_amdgcn_sched_barrier(0);
      step(three, sc, xa, zero, x1, one);
      load_weights(kc + 1, 3);
      sc = next;
      next = load_scales(kc + 2);
      step(zero, sc, xb, zero, x1, one);
      load_weights(kc + 2, 0);
      step(one, sc, xb, zero, x1, one);
      load_weights(kc + 2, 1);
      step(two, sc, xb, zero, x1, one);
      load_weights(kc + 2, 2);
      ready(weights_may_fly);
      const int k3 = min(kc + 3, n - 1);
      issue(x1, s1, k3);
      xa = read_scales(s0);
      __builtin_amdgcn_sched_barrier(0);
      step(three, sc, xb, zero, x0, one);
      load_weights(kc + 2, 3);
      sc = next;
      next = load_scales(k3);
      step(zero, sc, xa, zero, x0, one);
      load_weights(k3, 0);
      step(one, sc, xa, zero, x0, one);
      load_weights(k3, 1);
      step(two, sc, xa, zero, x0, one);
      load_weights(k3, 2);
    }
    ready(zero);
    xb = read_scales(s1);
    step(three, sc, xa, zero, x1, one);
    if (kc + 1 < n) {
      load_weights(kc + 1, 3);
      step(zero, next, xb, zero, x1, one);
      step(one, next, xb, zero, x1, one);
      step(two, next, xb, zero, x1, one);
      step(three, next, xb, zero, x1, zero);
    }
  }

  int first = 0;  // the row tile of acc[0]
  if constexpr (KS == 2) {
    // A group with a chunk less waits at as many barriers (the loop takes chunks in
    // twos); then the groups exchange sums, each keeps half the rows.
    static_assert(SS == 4, "barriers counts the one-stage loop's");
    auto barriers = [](int chunks) { return (chunks + 1) / 2 * 2; };
    for (int i = barriers(n); i < barriers(per_group); ++i) __builtin_amdgcn_s_barrier();
    constexpr int Q = RT / 2 * 4;  // 16-byte quarters of the sums that a lane gives away at a time
    f32x4* const out = red + (size_t)all * Q * 64 + lane;
    const f32x4* const in = red + (size_t)(all ^ 4) * Q * 64 + lane;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int t = 0; t < RT / 2; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f32x4 v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = grp ? acc[t][u][4 * g + i] : acc[RT / 2 + t][u][4 * g + i];
          out[(t * 4 + g) * 64] = v;
        }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < RT / 2; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 v = in[(t * 4 + g) * 64];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][u][4 * g + i] = (grp ? acc[RT / 2 + t][u][4 * g + i] : acc[t][u][4 * g + i]) + v[i];
        }
      if (u == 0) __syncthreads();
    }
    first = grp * (RT / 2);
  }
#pragma unroll
  for (int t = 0; t < RT / KS; ++t) {
    const int row = c.r0 + 32 * (first + t) + col;
    const bool on = row < c.s1;
    if constexpr (is_swiglu(EPI)) {
      const int I = p.N / 2;
      {
        const int ht = tile[0];
        float h[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) h[r] = silu_mul(acc[t][0][r], acc[t][1][r]);
        if constexpr (EPI == kEpiSwiglu) {
          uint32_t d[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = pack_bf16x2(h[2 * i], h[2 * i + 1]);
          store_tile16(d, static_cast<uint16_t*>(p.out) + (size_t)row * I + 32 * ht, half, on && valid[0]);
        } else {
          constexpr int F = EPI == kEpiSwigluE4M3 ? kE4M3 : kE2M1;
          uint32_t m = absmax_bits(h), mo = m;
          swap_halves(m, mo);
          m = m > mo ? m : mo;
          const bool bad = mx_not_finite(m);
          const int pe = mx_exponent<F>(m);
          const float scale = mx_scale(pe);
          uint32_t d[4];
#pragma unroll
          for (int g = 0; g < 4; ++g)
            d[g] = bad ? 0u : mx_pack4<F>(h[4 * g], h[4 * g + 1], h[4 * g + 2], h[4 * g + 3], scale);
          // lane half h gets channels 16h .. 16h + 15 of its token
          swap_halves(d[0], d[2]);
          swap_halves(d[1], d[3]);
          if (on && valid[0]) {
            const size_t o = (size_t)row * I + 32 * ht + 16 * half;
            if constexpr (F == kE4M3)
              *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p.out) + o) = u32x4{d[0], d[2], d[1], d[3]};
            else
              *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(p.out) + o / 2) = u32x2{d[0] | (d[2] << 16), d[1] | (d[3] << 16)};
            if (half == 0) p.out_scales[(size_t)row * (I >> 5) + ht] = bad ? (uint8_t)255 : (uint8_t)(pe + 127);
          }
        }
      }} else if constexpr (EPI == kEpiF32) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // A use of the sums outside the branch (no instruction): without it the
        // compiler moves the last matrix instructions, which take operands from
        // all lanes, into the branch that only lanes with a row enter.
        asm volatile("" : "+v"(acc[t][u]));
        if (on && valid[u]) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + (size_t)row * p.N + 32 * tile[u] + 8 * g + 4 * half) =
                f32x4{acc[t][u][4 * g], acc[t][u][4 * g + 1], acc[t][u][4 * g + 2], acc[t][u][4 * g + 3]};
        }
      }
    } else {
      // Through 4 KB of LDS, so that 8 neighbouring lanes store 128 bytes in a row:
      // 16-byte chunk k of row r (4 chunks a tile) at place k ^ (r & 7), row by row.
      // (32 bytes in a row per store: 65536 rows of 2048 channels, 1024 inputs 164 us
      // for 154 with e4m3 rows, 139 for 128 with e2m1 rows.)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float v[4] = {acc[t][u][4 * g], acc[t][u][4 * g + 1], acc[t][u][4 * g + 2], acc[t][u][4 * g + 3]};
          const u32x2 d = EPI == kEpiBf16 ? u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}
                                          : u32x2{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
          reinterpret_cast<u32x2*>(eb)[2 * (8 * col + ((4 * u + g) ^ (col & 7))) + half] = d;
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 3), k = lane & 7, at = c.r0 + 32 * (first + t) + r;
        const u32x4 v = eb[8 * r + (k ^ (r & 7))];
        if (at < c.s1 && valid[k >> 2])
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + (size_t)at * p.N + 32 * tile[0] + 8 * k) = v;
      }
    }
  }
}

// (The LDS stages are declared here: with generic lambdas in the kernel template
// itself the host's launch stub is not emitted; and only the device's pass sees
// the body, as the host's cannot instantiate several.)
//
// Without bodies for fewer rows a last tile of a few rows cost a whole one: 160
// rows per expert, 16 experts of 4096 x 4096: 54 -> 48 us with e4m3 rows, 42 -> 36
// with e2m1 rows; 100 to 420 rows per expert 4 % on average.
template <int AF, int EPI, int TM>
__global__ __launch_bounds__(256, TM == 128 ? 2 : 3) void mx_tile_kernel(MxK p, int n_nb) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int XC = stage_chunks(AF, TM), X = TM * XC, X0 = X > 4 * kEpiChunks ? X : 4 * kEpiChunks;
  __shared__ u32x4 x0[X0], x1[X];
  __shared__ uint32_t s0[256], s1[256];
  Tile c;
  if (!own_tile<TM>(p, n_nb, c)) return;
  // a segment's last rows: as few row tiles as hold them
  const int left = c.s1 - c.r0;
  if (left <= 32) mx_tile_body<AF, EPI, 32, 1, XC>(p, c, x0, x1, s0, s1, nullptr);
  else if (TM == 64 || left <= 64) mx_tile_body<AF, EPI, 64, 1, XC>(p, c, x0, x1, s0, s1, nullptr);
  else if (left <= 96) mx_tile_body<AF, EPI, 96, 1, XC>(p, c, x0, x1, s0, s1, nullptr);
  else mx_tile_body<AF, EPI, TM, 1, XC>(p, c, x0, x1, s0, s1, nullptr);
#endif
}
// Two groups of four wavefronts, each with stages of its own, take half of K each
// (K > 256): alone on its CU, a workgroup of e2m1 rows waits for loads most of the
// time.
template <int AF, int EPI>
__global__ __launch_bounds__(512, 2) void mx_tile_split_kernel(MxK p, int n_nb) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int XC = stage_chunks(AF, 64);
  __shared__ u32x4 x0[8 * kEpiChunks], x1[2 * 64 * XC];
  __shared__ uint32_t s0[512], s1[512];
  __shared__ f32x4 red[8 * 4 * 64];
  Tile c;
  if (!own_tile<64>(p, n_nb, c)) return;
  mx_tile_body<AF, EPI, 64, 2, XC>(p, c, x0, x1, s0, s1, red);
#endif
}

template <int AF, int EPI>
int launch_small(const MxK& k, hipStream_t s) {
  const int NT = k.N / 32;
  // one workgroup per 32 rows up to twice the mean rows of an expert; fuller
  // experts' workgroups go round
  const int gz = (k.M_total / k.E - 1) / 16 + 1;
  const dim3 grid(is_swiglu(EPI) ? NT / 2 : (NT + 1) / 2, k.E, gz < 1 ? 1 : gz > 64 ? 64 : gz);
  hipLaunchKernelGGL((mx_small_kernel<AF, EPI>), grid, dim3(256), 0, s, k);
  return (int)hipGetLastError();
}
template <int AF, int EPI, int TM>
int launch_tile(const MxK& k, bool split, hipStream_t s) {
  const int NT = k.N / 32;
  const int n_nb = is_swiglu(EPI) ? (NT / 2 + 3) / 4 : (NT + 7) / 8;
  // upper bound of the row tiles: one partial tile per segment that has rows
  const int64_t tiles = (int64_t)k.M_total / TM + (k.E < k.M_total ? k.E : k.M_total);
  const int64_t wgs = (tiles * n_nb + 7) / 8 * 8;
  if (wgs >= ((int64_t)1 << 23)) return (int)hipErrorInvalidConfiguration;  // 2^32 threads in 512s
  if constexpr (TM == 64 && AF == kE2M1) {
    if (split) {
      hipLaunchKernelGGL((mx_tile_split_kernel<AF, EPI>), dim3((unsigned)wgs), dim3(512), 0, s, k, n_nb);
      return (int)hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_tile_kernel<AF, EPI, TM>), dim3((unsigned)wgs), dim3(256), 0, s, k, n_nb);
  return (int)hipGetLastError();
}
template <int AF, int EPI>
int launch_path(const MxK& k, int path, hipStream_t s) {
  if (path == 64 || path == kMxSplit) return launch_tile<AF, EPI, 64>(k, path == kMxSplit, s);
  if (path == 128) return launch_tile<AF, EPI, 128>(k, false, s);
  return launch_small<AF, EPI>(k, s);
}
template <int AF>
int launch_fmt(const MxK& k, int epi, int path, hipStream_t s) {
  switch (epi) {
    case kEpiBf16: return launch_path<AF, kEpiBf16>(k, path, s);
    case kEpiSwiglu: return launch_path<AF, kEpiSwiglu>(k, path, s);
    case kEpiF32: return launch_path<AF, kEpiF32>(k, path, s);
    case kEpiF16: return launch_path<AF, kEpiF16>(k, path, s);
    case kEpiSwigluE4M3: return launch_path<AF, kEpiSwigluE4M3>(k, path, s);
    default: return launch_path<AF, kEpiSwigluE2M1>(k, path, s);
  }
}
}  // namespace

int launch_mxgemm(const MxGemmArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t row_codes = a.a_fmt == kE4M3 ? a.K : a.K / 2;
  const int div = a.gather ? a.k : 1;
  int sh = 0;
  while (((int64_t)1 << sh) < div) ++sh;
  const MxK k{a.wcodes, a.wscales, a.N, a.K, a.a, a.as, (uint32_t)(a.A_rows * row_codes),
              (uint32_t)((size_t)a.A_rows * (a.K / 32)), a.A_rows, a.gather, (uint32_t)((((uint64_t)1 << (31 + sh)) + div - 1) / div), sh, a.seg, a.E, a.M_total,
              a.out, a.out_scales};
  const int path = mxgemm_path(a.M_total, a.E, a.N, a.K, a.a_fmt == kE2M1, a.kernel);
  return a.a_fmt == kE4M3 ? launch_fmt<kE4M3>(k, a.epilogue, path, s) : launch_fmt<kE2M1>(k, a.epilogue, path, s);
}

}  // namespace moe
