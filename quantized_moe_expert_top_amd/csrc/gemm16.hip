// Grouped product of rows with the experts' 16-bit weights, and its gradients by
// the rows and by the weights, on v_mfma_f32_16x16x32 (bf16 or fp16 operands,
// fp32 sums): the matrix units run at the power limit, and random operands cost less
// in this shape than in 32 x 32 x 16 (from registers alone 1978 and 1695 TFLOP/s; the
// tiles below at first, 8192^3: 760 and 831 us).
// Measured (bf16, random operands): 8192^3 749 us (1468 TFLOP/s), by the rows 755, by
// the weights 762.  64 experts of 2048 x 2048, 65536 rows gathered, SwiGLU and what
// enters it 527 us (1044); by the weights 535.  The rest goes to stores: all
// workgroups' tiles end at about the same time and wait for the memory (a quarter of
// them storing costs nearly nothing), and to segments' partial last tiles.
#include <type_traits>
#include <utility>

#include "offsets.h"
#include "segments.h"

namespace moe {

namespace {
constexpr int kForward = 0, kRows = 1, kWeights = 2;                          // what a kernel computes
constexpr int kEpiSwiglu = 1, kEpiF32 = 2, kEpiF16 = 3, kEpiSwigluGrad = 6;  // MOE_EPI_* (0: bf16)

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
  int splits;  // weights: parts of a segment's rows, each with fp32 sums of its own (out: [splits][E][N][K])
};

// ----------------------------------------- tiles of 256 x 256, 128 x 128, 128 x 256
// out[b][a] = sum_k P[a][k] Q[b][k]: a runs along the output's rows (contiguous),
// b over them.
//   forward  a: channels (SwiGLU: 128 gate and the matching 128 up channels), b: rows, k: inputs
//   rows     a: inputs, b: rows, k: channels
//   weights  a: inputs, b: channels, k: the segment's rows
// P and Q go through two (or three) LDS stages of 64 k, filled by LDS-DMA.  An operand whose
// k lie next to each other in memory ("direct") is kept [256][64], one whose a or
// b do [64][256], read back transposed (ds_read_b64_tr_b16).
// A wavefront of 256 x 256 reads 12 KB of LDS for 32 products (64 a x 128 b: half of its
// registers hold sums), of 128 x 128 8 KB for 16; but two workgroups of those a CU cover
// each other's ends of tiles, and short segments fill them.  The choice: gemm16_path.
typedef short s16x4 __attribute__((ext_vector_type(4)));
constexpr int kCUs = 256;
constexpr uint32_t kLastGather = kGatherBytes;  // kOut's part for a gathered row, also with a column added
constexpr uint32_t kDrop = 0x80000000u;  // past any output tile, also with a row added: not stored

// [256][64] of 16 bits in 16-byte chunks, 8 a row: chunk c of row r at place c ^ swz(r).  A read
// of 16 rows' 4 chunks takes lanes 0-3, 12-15, 20-23 and 24-27 at a time, 4-11, 16-19 and 28-31,
// and the same of the upper half: with this order each group covers all 64 banks (with bit 3 of
// the row mixed in too, as 16 lanes in a row would want it, every bank came twice: 8192^3 760 us
// and not 749).
__device__ __forceinline__ int swz(int row) { return row & 7; }

// [64][256] of 16 bits in 32-byte units, 16 a row: unit u of row k at place u ^ tswz(k): the
// four rows of a transposing read's 16 lanes and the eight of 32 lanes fall on different banks.
__device__ __forceinline__ int tswz(int k) { return (k & 3) | ((k >> 1) & 4); }

// The same for [32][64] of 16 bits, four units a row.
__device__ __forceinline__ int tswz4(int k) { return ((k >> 1) & 1) | ((k >> 2) & 2); }

// Fast exponential and reciprocal, as in the library's other SwiGLU epilogues (2^-19
// relative down to gates of -16, 0 below -88).
__device__ __forceinline__ float silu(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }
// Gradient of silu(g) * u from d, by g and u (16-bit numbers).
template <bool F16>
__device__ __forceinline__ float2 swiglu_grad(float d, uint16_t g16, uint16_t u16) {
  const float g = widen16<F16>(g16), u = widen16<F16>(u16), s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
  return {d * u * s * (1.0f + g * (1.0f - s)), d * g * s};
}
template <typename F, int... X>
__device__ __forceinline__ void for_each(F&& f, std::integer_sequence<int, X...>) {
  (f(std::integral_constant<int, X>{}), ...);
}

struct Tile {
  int e, ab, b0, s0, s1;  // expert, a block, first b; the segment's rows (weights: the sum's)
  int part;               // weights: which of the splits
};

// Tiles in an order that neighbours share operands in an XCD's L2: within a
// segment in groups of 8 row tiles by a block.
__device__ __forceinline__ void grouped_order(int idx, int tiles, int n_ab, int& tile, int& ab) {
  const int g = idx / (8 * n_ab), gm = min(8, tiles - 8 * g), in = idx - g * 8 * n_ab;
  ab = in / gm;
  tile = 8 * g + in % gm;
}

// A workgroup (256 a: 8 wavefronts, alone on its CU; 128: 4) takes tile after tile, a
// wavefront 64 a and up to 128 b of each.  The last NS steps of a tile issue the first ones of the
// next, so that only the first tile waits for its loads, and a tile's stores go
// out under the next one's products.
template <int T, int TB, int NS, bool F16, int MODE, bool GATHER, bool GLU>
__device__ __forceinline__ void tile_loop(const GemmK& p, int epi, int n_ab, int n_bb, char* const (&pS)[NS], char* const (&qS)[NS], char* sE) {
  constexpr bool PT = MODE != kForward, QT = MODE == kWeights;  // transposed operands
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  constexpr int WA = T / 64;      // wavefronts along a; two along b
  constexpr int QD = 4 * TB / T;  // DMAs of Q a wavefront and step (of P 4)
  static_assert(!QT || TB == T, "");
  const int wa = wv & (WA - 1), wb = wv / WA, col = lane & 15, quad = lane >> 4;
  const int I = p.N / 2;
  const int na = MODE == kForward ? p.N : p.K;  // a's extent (and a transposed P's row length)

  // Which tiles: workgroups are dealt to the 8 XCDs in turn, each XCD takes a
  // contiguous range.  The first 64 segments stay in registers, one per lane.
  int seg_n = 0, seg_end = 0, seg0 = 0, seg1 = 0, total;
  if constexpr (MODE == kWeights) {
    total = p.E * p.splits * n_ab * n_bb;
  } else {
    seg_n = segment_tiles<TB>(p.seg, p.E, p.M_total, lane, seg0, seg1);
    seg_end = lane_scan(seg_n);
    total = (p.E <= 64 ? __builtin_amdgcn_readlane(seg_end, 63) : count_tiles<TB>(p.seg, p.E, p.M_total)) * n_ab;
  }
  const int per = (total + 7) >> 3, xcd = (int)blockIdx.x & 7;
  int idx = xcd * per + ((int)blockIdx.x >> 3);
  const int idx_end = min(total, (xcd + 1) * per), idx_step = (int)gridDim.x >> 3;
  if (idx >= idx_end) return;
  auto locate = [&](int at) {
    Tile c;
    int tile;
    if constexpr (MODE == kWeights) {
      const int ep = at / (n_ab * n_bb);
      grouped_order(at - ep * (n_ab * n_bb), n_bb, n_ab, tile, c.ab);
      c.e = ep / p.splits;
      c.part = ep - c.e * p.splits;
      c.b0 = T * tile;
      c.s0 = c.s1 = 0;
      if (p.M_total > 0) segment_rows(p.seg, c.e, p.M_total, c.s0, c.s1);
      if (p.splits > 1) {  // whole steps of 64 rows
        const int64_t steps = (c.s1 - c.s0 + 63) >> 6;
        const int from = (int)(steps * c.part / p.splits) * 64, to = (int)(steps * (c.part + 1) / p.splits) * 64;
        c.s1 = min(c.s1, c.s0 + to);
        c.s0 = min(c.s1, c.s0 + from);
      }
    } else {
      RowTile t;
      if (p.E <= 64) {
        t.e = __builtin_ctzll(__ballot(at < seg_end * n_ab));
        t.tiles = __builtin_amdgcn_readlane(seg_n, t.e);
        t.r0 = __builtin_amdgcn_readlane(seg0, t.e);
        t.s1 = __builtin_amdgcn_readlane(seg1, t.e);
        at -= (__builtin_amdgcn_readlane(seg_end, t.e) - t.tiles) * n_ab;
      } else {
        find_tile<TB>(p.seg, p.E, p.M_total, n_ab, at, t);
      }
      grouped_order(at, t.tiles, n_ab, tile, c.ab);
      c.e = t.e;
      c.b0 = t.r0 + TB * tile;
      c.s0 = t.r0;
      c.s1 = t.s1;
    }
    return c;
  };

  // The DMAs of a tile: a wavefront fetches 4 KB of P and QD of Q a step, 1 KB each;
  // DMAs i and i + 2 (direct operands: i and i + 1) differ by a fixed number of bytes (not
  // where rows are gathered).
  // Rows past an operand's end lie past the descriptor's bytes and read zero.
  constexpr int QO = GATHER && MODE == kForward ? QD : QT ? 2 : 1;
  uint32_t po[PT ? 2 : 1], qo[QO];        // byte offsets of this lane's 16 bytes, or kOut
  int ck8 = 0;                            // direct operands: first k of the lane's chunk
  const uint16_t *pbase = p.w, *qbase = p.w;
  uint32_t pbytes = 0, qbytes = 0;
  int red = 0, ls0 = 0, ls1 = 0;
  int src = 0;                            // weights: the pair of the next step's row 8 wv + lane % 8
  // A copy of the lane's number that the compiler knows nothing about: what a tile
  // needs once is computed there, and not kept in registers over the products.
  auto lane_here = [&] {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };
  // Transposed operands: a row of a stage is T columns, a DMA RK rows; DMA i fetches k
  // = dr + RK i.  Two DMAs whose rows are 4 apart have the same places (tswz).
  constexpr int RK = 512 / T, LR = T / 8;  // (lanes of a row)
  const int dr = 4 * RK * wv + lane / LR;
  constexpr auto twin = [](int i) { return T == 256 ? i & 1 : i >> 1; };    // which of the two kinds
  constexpr auto second = [](int i) { return T == 256 ? i >> 1 : i & 1; };  // whether the later one
  // The pair of one of the wavefront's gathered rows: of forward's 8 QD b row lane % (8 QD), of
  // weights' 4 RK k of a step row lane % (4 RK).
  auto pair_of = [&](const Tile& c, int step) {
    if constexpr (!GATHER) return 0;
    const int l = lane_here();
    return p.gather[max(min(MODE == kForward ? c.b0 + 8 * QD * wv + (l & (8 * QD - 1)) : c.s0 + 64 * step + 4 * RK * wv + (l & (4 * RK - 1)), c.s1 - 1), 0)];
  };
  auto token = [&](int pair) { return (uint32_t)min(max(p.div(pair), 0), p.A_rows - 1); };
  auto trans_ch = [&](int lane, int k) {  // first of the 8 columns that this lane fetches of row k
    const int s16 = lane & (LR - 1);
    return 8 * ((((s16 >> 1) ^ tswz(k)) << 1) + (s16 & 1));
  };
  auto setup = [&](const Tile& c, bool on, int pair) {
    const int lane = lane_here(), dr = 4 * RK * wv + lane / LR, br = 32 * wv + (lane >> 3), bq = 8 * QD * wv + (lane >> 3), ck = (lane & 7) ^ swz(br);
    red = !on ? 0 : MODE == kForward ? p.K : MODE == kRows ? p.N : c.s1 - c.s0;
    ls0 = c.s0;
    ls1 = c.s1;
    if constexpr (PT) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = dr + (T == 256 ? 2 : 8) * i, ch = T * c.ab + trans_ch(lane, k);
        po[i] = ch < na ? (GATHER ? (uint32_t)ch : (uint32_t)k * (uint32_t)na + ch) * 2 : kOut;
      }
      pbase = MODE == kRows ? p.w + (size_t)c.e * p.N * p.K : GATHER ? p.a : p.a + (size_t)c.s0 * p.K;
      if constexpr (GATHER) {
        src = pair;
        pbytes = (uint32_t)((size_t)p.A_rows * p.K * 2);
      }
    } else {
      // SwiGLU: rows 64w .. 64w + 31 are gate channels of wavefront column w, 64w + 32 .. 64w + 63
      // their up channels (past the last gate channel: up ones, never stored)
      const int ch = GLU ? T / 2 * c.ab + 32 * (wv >> 1) + (lane >> 3) + (wv & 1 ? I : 0) : T * c.ab + br;
      po[0] = row_offset(ch, p.N, p.K, 8 * ck);
      pbase = p.w + (size_t)c.e * p.N * p.K;
      pbytes = (uint32_t)((size_t)p.N * p.K * 2);
    }
    if constexpr (QT) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = dr + (T == 256 ? 2 : 8) * i, ch = c.b0 + trans_ch(lane, k);
        qo[i] = ch < p.N ? ((uint32_t)k * (uint32_t)p.N + ch) * 2 : kOut;
      }
      qbase = p.dy + (size_t)c.s0 * p.N;
    } else {
      const int ld = MODE == kForward ? p.K : p.N;
      ck8 = 8 * ck;
#pragma unroll
      for (int i = 0; i < QO; ++i) {
        const int r = bq + 8 * i;
        const uint32_t from = GATHER ? (uint32_t)__shfl((int)token(pair), 8 * i + (lane >> 3), 64) : r;
        qo[i] = (from * (uint32_t)ld + 8 * ck) * 2;
        if (GATHER && c.b0 + r >= c.s1) qo[i] = kOut;
      }
      qbase = MODE == kForward ? (GATHER ? p.a : p.a + (size_t)c.b0 * ld) : p.dy + (size_t)c.b0 * ld;
      qbytes = GATHER ? (uint32_t)((size_t)p.A_rows * ld * 2) : (uint32_t)((size_t)min(c.s1 - c.b0, TB) * ld * 2);
    }
  };

  // DMAs of step st into a stage; past the sum's end zeros.
  auto dma = [&](rsrc_t r, char* to, uint32_t off, uint32_t adv) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, off, adv, 0, 0);
  };
  auto issue = [&](char* ps, char* qs, int st) {
    const int left = red - 64 * st;  // k of this step and later ones
    const uint32_t rows = (uint32_t)max(min(left, 64), 0);
    const uint32_t adv = left > 0 ? (uint32_t)st * 128u : 0u;
    char* const pd = ps + wv * 4096;
    char* const qd = qs + wv * (1024 * QD);
    if constexpr (PT && GATHER) {
      const rsrc_t pr = scalar_rsrc(pbase, pbytes);
      // row 4 RK wv + lane % (4 RK)'s offset, past the segment one that no column brings back (kLastGather)
      const int l = lane_here();
      uint32_t from = token(src) * (uint32_t)(2 * p.K);
      asm volatile("" : "+v"(from));  // (a select, not a branch around the loads)
      if (4 * RK * wv + (l & (4 * RK - 1)) >= left) from = kLastGather;
      src = pair_of(Tile{0, 0, 0, ls0, ls1, 0}, st + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t at;
        if constexpr (T == 256) {
          const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)from, 2 * i), hi = (uint32_t)__builtin_amdgcn_readlane((int)from, 2 * i + 1);
          at = l & 32 ? hi : lo;
        } else {
          at = (uint32_t)__shfl((int)from, 4 * i + (l >> 4), 64);
        }
        dma(pr, pd + 1024 * i, offset_sum(po[twin(i)], at), 0);
      }
    } else if constexpr (PT) {
      const rsrc_t pr = scalar_rsrc(pbase + (size_t)(64 * st) * na, rows * (2u * (uint32_t)na));
#pragma unroll
      for (int i = 0; i < 4; ++i) dma(pr, pd + 1024 * i, po[twin(i)], second(i) ? 8u * (uint32_t)na : 0u);
    } else {
      const rsrc_t pr = scalar_rsrc(pbase, pbytes);
      const uint32_t at = ck8 < left ? po[0] : kOut;
#pragma unroll
      for (int i = 0; i < 4; ++i) dma(pr, pd + 1024 * i, at, adv + (uint32_t)i * 16u * (uint32_t)p.K);
    }
    if constexpr (QT) {
      const rsrc_t qr = scalar_rsrc(qbase + (size_t)(64 * st) * p.N, rows * (2u * (uint32_t)p.N));
#pragma unroll
      for (int i = 0; i < 4; ++i) dma(qr, qd + 1024 * i, qo[twin(i)], second(i) ? 8u * (uint32_t)p.N : 0u);
    } else {
      const rsrc_t qr = scalar_rsrc(qbase, qbytes);
      const int ld = MODE == kForward ? p.K : p.N;
#pragma unroll
      for (int i = 0; i < QD; ++i)
        dma(qr, qd + 1024 * i, ck8 < left ? qo[QO == QD ? i : 0] : kOut, QO == QD ? adv : adv + (uint32_t)i * 16u * (uint32_t)ld);
    }
  };

  // Fragments of 16 rows (of a or b) x 32 k (half s of a stage), for 16 x 16 x 32:
  // lane (quad, col) holds row col, k = 8 quad .. 8 quad + 7.  The lane's place of the
  // first fragment; others differ in bits that no other term has (x, s) or by constants.
  const int dk = 8 * quad + ((lane >> 2) & 3);  // transposed: the lane reads 8 bytes of row dk (and dk + 4)
  constexpr int RB = 2 * T;  // bytes of a transposed row
  uint32_t pat = PT ? dk * RB + (((4 * wa) ^ tswz(dk)) << 5) + ((lane & 3) << 3) : wa * 8192 + col * 128 + ((quad ^ swz(col)) << 4);
  uint32_t qat = QT ? dk * RB + (((2 * wb) ^ tswz(dk)) << 5) + ((lane & 3) << 3) : wb * 4096 + col * 128 + ((quad ^ swz(col)) << 4);
  auto read_at = [&](const char* stage, uint32_t at, auto trans_tag) {
    if constexpr (decltype(trans_tag)::value) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(stage + at));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(stage + at + 4 * RB));
      const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
      return u32x4{l[0], l[1], h[0], h[1]};
    } else {
      return *reinterpret_cast<const u32x4*>(stage + at);
    }
  };
  auto read_p = [&](const char* ps, uint32_t at, int t, int s) {  // a = 64 wa + 16 t + col
    return PT ? read_at(ps + 32 * RB * s, at ^ (t << 5), std::integral_constant<bool, PT>{})
              : read_at(ps + 2048 * t, at ^ (s << 6), std::integral_constant<bool, PT>{});
  };
  // the wavefront's b: 32 rows of every 64, b = 64 (j / 2) + 32 wb + 16 (j % 2) + col
  auto read_q = [&](const char* qs, uint32_t at, int j, int s) {
    return QT ? read_at(qs + 32 * RB * s + 256 * (j >> 2), at ^ ((4 * ((j >> 1) & 1) + (j & 1)) << 5), std::integral_constant<bool, QT>{})
              : read_at(qs + 8192 * (j >> 1) + 2048 * (j & 1), at ^ (s << 6), std::integral_constant<bool, QT>{});
  };
  // Every wavefront's reads of a stage are done and the next stage's DMAs landed; those of
  // the stages behind it, 4 + QD each, may be on their way (vmcnt, whose upper two bits lie
  // apart; anything else in flight only makes it wait longer).
  auto ready = [&] {
    constexpr int fly = (4 + QD) * (NS - 2);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070 | (fly & 15) | (fly >> 4) << 14);  // lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  Tile cur = locate(idx), nxt;
  bool more;
  // One tile with b in NB x 64.
  auto body = [&](auto nb_tag) {
    constexpr int NB = decltype(nb_tag)::value;
    constexpr int J = 2 * NB;            // b tiles of 16
    constexpr int D = J < 4 ? J : 4;     // Q fragments read ahead
    f32x4 acc[4][J] = {};
    u32x4 pf[2][4], qf[D];
    // One stage: 2 J slots of 4 products (one Q fragment with 4 of P), each followed by
    // the reads for later ones.  All of the stage's reads are done D slots before its
    // end: there the wavefronts meet, the stage is filled again, and the last slots'
    // products cover the first reads of the other stage.
    auto stage = [&](const char* ps, const char* qs, const char* pn, const char* qn, auto meet) {
      // (opaque: the places of the other fragments are worked out here, not kept in registers)
      asm volatile("" : "+v"(pat), "+v"(qat));
      auto slot = [&](auto x_tag) {
        constexpr int X = decltype(x_tag)::value, S = X / J, JJ = X % J, Y = X + D;
        if constexpr (X == 2 * J - D) meet();
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t][JJ] = mfma16t<F16>(pf[S][t], qf[X % D], acc[t][JJ]);
        qf[X % D] = Y < 2 * J ? read_q(qs, qat, Y % J, Y / J) : read_q(qn, qat, Y % J, 0);
        if constexpr (X < D) {  // the second half's P
#pragma unroll
          for (int t = X * 4 / D; t < (X + 1) * 4 / D; ++t) pf[1][t] = read_p(ps, pat, t, 1);
        }
        if constexpr (X >= 2 * J - D && X < 2 * J - D + 2) {  // the other stage's
#pragma unroll
          for (int t = 2 * (X - 2 * J + D); t < 2 * (X - 2 * J + D) + 2; ++t) pf[0][t] = read_p(pn, pat, t, 0);
        }
        if constexpr (X & 1) __builtin_amdgcn_sched_barrier(0);
      };
      for_each(slot, std::make_integer_sequence<int, 2 * J>{});
    };
    const int next_pair = pair_of(nxt, 0);
    // a multiple of NS steps: past the sum's end they multiply zeros
    const int n = max((red + 64 * NS - 1) / (64 * NS) * NS, NS);
#pragma unroll
    for (int t = 0; t < 4; ++t) pf[0][t] = read_p(pS[0], pat, t, 0);
#pragma unroll
    for (int x = 0; x < D; ++x) qf[x] = read_q(qS[0], qat, x, 0);
    for (int st = NS; st < n; st += NS) {
      for_each([&](auto u_tag) {
        constexpr int U = decltype(u_tag)::value, V = (U + 1) % NS;
        stage(pS[U], qS[U], pS[V], qS[V], [&] {
          ready();
          issue(pS[U], qS[U], st + U);
        });
      }, std::make_integer_sequence<int, NS>{});
    }
    for_each([&](auto u_tag) {
      constexpr int U = decltype(u_tag)::value, V = (U + 1) % NS;
      stage(pS[U], qS[U], pS[V], qS[V], [&] {
        ready();
        if constexpr (U == 0) setup(nxt, more, next_pair);
        issue(pS[U], qS[U], U);
      });
    }, std::make_integer_sequence<int, NS>{});

    // Epilogue: a wavefront's 32 b x 64 a (fp32: 32) at a time through 4 KB of LDS, so
    // that neighbouring lanes store 64 bytes and more in a row.  Of tile (t, x)
    // lane (quad, col) holds a = a0 + 16t + 4*quad + 0..3 and b = 16x + col.
    // Rows past the end lie past the descriptor's bytes, channels get kDrop: every
    // lane stores, and the stores are counted.
    char* const eb = sE + wv * 4096;
    const int lane = lane_here(), quad = lane >> 4, col = lane & 15;
    const int a0 = GLU && MODE == kForward ? T / 2 * cur.ab + 32 * wa : T * cur.ab + 64 * wa;
    const int rows = min((MODE == kWeights ? p.N : cur.s1) - cur.b0, TB);
    const size_t row0 = (MODE == kWeights ? ((size_t)cur.part * p.E + cur.e) * p.N : 0) + cur.b0;
    auto chunk = [&](int r, int ck) { return eb + r * 128 + ((ck ^ swz(r)) << 4); };  // 8 chunks of 16 bytes a row
    auto put16 = [&](int t, int x, const f32x4& v, bool f16) {
      *reinterpret_cast<u32x2*>(chunk(16 * x + col, 2 * t + (quad >> 1)) + 8 * (quad & 1)) =
          f16 ? u32x2{pack16x2<true>(v[0], v[1]), pack16x2<true>(v[2], v[3])} : u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };
    auto put32 = [&](int t, int x, const f32x4& v) { *reinterpret_cast<f32x4*>(chunk(16 * x + col, 4 * t + quad)) = v; };
    auto get = [&](int r, int ck) { return *reinterpret_cast<const u32x4*>(chunk(r, ck)); };
    auto get32 = [&](int r, int ck) { return *reinterpret_cast<const f32x4*>(chunk(r, ck)); };
    auto row_of = [&](int j, int x) { return 64 * j + 32 * wb + x; };  // of the j-th 32's row x, from cur.b0
    auto store = [&](rsrc_t r, u32x4 v, uint32_t off, int row, uint32_t ld, auto stream_tag) {
      typedef unsigned int b128 __attribute__((ext_vector_type(4)));
      // The row's offset is added here: with a scalar register as the instruction's
      // offset the compiler sees no hazard in overwriting the data in the next
      // instruction, but gfx950 then stores some of the new values.
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(b128, v), r, off + (uint32_t)row * ld, 0, decltype(stream_tag)::value ? 2 : 0);
    };
    // Whole lines of 128 bytes go past the caches (65536 rows of 2048 channels, us with and without:
    // 87 / 122 with 256 inputs, 134 / 168 with 512, 265 / 267 with 1024), halves of lines, which
    // the L2 joins, do not (SwiGLU with what enters it 546 / 529).
    const std::true_type whole_lines{};
    const std::false_type half_lines{};
    if constexpr (GLU && MODE == kForward) {
      const uint32_t ldo = 2u * (uint32_t)I, ldp = 2u * (uint32_t)p.N;
      const rsrc_t ro = scalar_rsrc(static_cast<uint16_t*>(p.out) + row0 * I, (uint32_t)rows * ldo);
      const int ch = a0 + 8 * (lane & 3);
      const uint32_t oo = ch < I ? (uint32_t)(lane >> 2) * ldo + 2 * ch : kDrop;
      const uint32_t op = ch < I ? (uint32_t)(lane >> 3) * ldp + 2 * (ch + (lane & 4 ? I : 0)) : kDrop;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (p.pre_out) {
          const rsrc_t rp = scalar_rsrc(p.pre_out + row0 * p.N, (uint32_t)rows * ldp);
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) put16(t, x, acc[t][2 * j + x], F16);
#pragma unroll
          for (int i = 0; i < 4; ++i) store(rp, get(8 * i + (lane >> 3), lane & 7), op, row_of(j, 8 * i), ldp, half_lines);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const f32x4 &g = acc[t][2 * j + x], &u = acc[t + 2][2 * j + x];
            f32x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = silu(g[i]) * u[i];
            put16(t, x, h, F16);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) store(ro, get(16 * i + (lane >> 2), lane & 3), oo, row_of(j, 16 * i), ldo, half_lines);
      }
    } else if constexpr (GLU) {
      const uint32_t ld = 4u * (uint32_t)p.K;
      const rsrc_t ro = scalar_rsrc(static_cast<uint16_t*>(p.out) + row0 * 2 * p.K, (uint32_t)rows * ld);
      const rsrc_t rp = scalar_rsrc(p.pre_in + row0 * 2 * p.K, (uint32_t)rows * ld);
      const int x = 8 * (lane & 3);
      // 8 channels of 16 rows a load: gate and up, for both tiles and row halves of one j
      struct Pre {
        u32x4 g[2][2], u[2][2];
      };
      uint32_t off[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int ch = a0 + 32 * t + x;
        off[t] = ch < p.K ? (uint32_t)(lane >> 2) * ld + 2 * ch : kDrop;
      }
      auto fetch = [&](int j) {
        Pre v;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            v.g[t][i] = buf_x4(rp, off[t], (uint32_t)row_of(j, 16 * i) * ld);
            v.u[t][i] = buf_x4(rp, off[t] + ld / 2, (uint32_t)row_of(j, 16 * i) * ld);
          }
        return v;
      };
      Pre pre = fetch(0), ahead;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (j + 1 < NB) ahead = fetch(j + 1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int h = 0; h < 4; ++h) put32(h >> 1, h & 1, acc[2 * t + (h >> 1)][2 * j + (h & 1)]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 16 * i + (lane >> 2);
            u32x4 dg, du;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const f32x4 d = get32(r, 2 * (lane & 3) + q);
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const uint32_t gw = pre.g[t][i][2 * q + w], uw = pre.u[t][i][2 * q + w];
                float og[2], ou[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float2 o = swiglu_grad<F16>(d[2 * w + z], (uint16_t)(z ? gw >> 16 : gw & 0xFFFFu), (uint16_t)(z ? uw >> 16 : uw & 0xFFFFu));
                  og[z] = o.x;
                  ou[z] = o.y;
                }
                dg[2 * q + w] = pack16x2<F16>(og[0], og[1]);
                du[2 * q + w] = pack16x2<F16>(ou[0], ou[1]);
              }
            }
            store(ro, dg, off[t], row_of(j, 16 * i), ld, half_lines);
            store(ro, du, off[t] + ld / 2, row_of(j, 16 * i), ld, half_lines);
          }
        }
        pre = ahead;
      }
    } else if (epi == kEpiF32) {
      const uint32_t ld = 4u * (uint32_t)na;
      const rsrc_t ro = scalar_rsrc(static_cast<float*>(p.out) + row0 * na, (uint32_t)rows * ld);
      const int x = 4 * (lane & 7);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int ch = a0 + 32 * t + x;
        const uint32_t off = ch < na ? (uint32_t)(lane >> 3) * ld + 4 * ch : kDrop;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
#pragma unroll
          for (int h = 0; h < 4; ++h) put32(h >> 1, h & 1, acc[2 * t + (h >> 1)][2 * j + (h & 1)]);
#pragma unroll
          for (int i = 0; i < 4; ++i) store(ro, get(8 * i + (lane >> 3), lane & 7), off, row_of(j, 8 * i), ld, whole_lines);
        }
      }
    } else {
      const uint32_t ld = 2u * (uint32_t)na;
      const rsrc_t ro = scalar_rsrc(static_cast<uint16_t*>(p.out) + row0 * na, (uint32_t)rows * ld);
      const int x = 8 * (lane & 7), ch = a0 + x;
      const uint32_t off = ch < na ? (uint32_t)(lane >> 3) * ld + 2 * ch : kDrop;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) put16(t, x, acc[t][2 * j + x], epi == kEpiF16);
#pragma unroll
        for (int i = 0; i < 4; ++i) store(ro, get(8 * i + (lane >> 3), lane & 7), off, row_of(j, 8 * i), ld, whole_lines);
      }
    }
  };

  setup(cur, true, pair_of(cur, 0));
#pragma unroll
  for (int u = 0; u < NS; ++u) issue(pS[u], qS[u], u);
  ready();
  while (true) {
    idx += idx_step;
    more = idx < idx_end;
    nxt = more ? locate(idx) : cur;
    const int left = MODE == kWeights ? T : cur.s1 - cur.b0;
    if constexpr (TB == 256) {
      if (left <= 64) body(std::integral_constant<int, 1>{});
      else if (left <= 128) body(std::integral_constant<int, 2>{});
      else if (left <= 192) body(std::integral_constant<int, 3>{});
      else body(std::integral_constant<int, 4>{});
    } else {
      if (left <= 64) body(std::integral_constant<int, 1>{});
      else body(std::integral_constant<int, 2>{});
    }
    if (!more) break;
    cur = nxt;
  }
}

template <int T, bool F16, int MODE, bool GATHER, bool GLU>
__global__ __launch_bounds__(2 * T, 2) void tile_kernel(GemmK p, int epi, int n_ab, int n_bb) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __attribute__((aligned(1024))) char p0[128 * T], p1[128 * T], q0[128 * T], q1[128 * T], sE[T / 32 * 4096];
  char *const ps[2] = {p0, p1}, *const qs[2] = {q0, q1};
  tile_loop<T, T, 2, F16, MODE, GATHER, GLU>(p, epi, n_ab, n_bb, ps, qs, sE);
#endif
}

// Few tiles: one workgroup a CU, three stages.  Tiles of 128 x 128, or of 128 a x 256 rows
// where those of 128 rows would take two rounds, those of 256 one, and no segment has
// more than 192 (a tile's time goes with its rows): 8 experts of 4096 x 14336 with 110 to 150
// rows each 217 us, with two workgroups a CU 287 and 128-row tiles; by the rows of
// 28672 x 4096, 20 to 430 rows each, 567 with 128-row tiles, with 256-row ones 788.
template <bool F16, int MODE, bool GATHER, bool GLU>
__global__ __launch_bounds__(256, 1) void deep_kernel(GemmK p, int epi, int n_ab) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __attribute__((aligned(1024))) char p0[16384], p1[16384], p2[16384], q0[32768], q1[32768], q2[32768], sE[16384];
  char *const ps[3] = {p0, p1, p2}, *const qs[3] = {q0, q1, q2};
  bool even = true;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    int s0, s1;
    segment_tiles<128>(p.seg, p.E, p.M_total, e0 + (threadIdx.x & 63), s0, s1);
    even = even && __ballot(s1 - s0 > 192) == 0;
  }
  if (even && count_tiles<128>(p.seg, p.E, p.M_total) * n_ab > kCUs && count_tiles<256>(p.seg, p.E, p.M_total) * n_ab <= kCUs)
    tile_loop<128, 256, 3, F16, MODE, GATHER, GLU>(p, epi, n_ab, 0, ps, qs, sE);
  else
    tile_loop<128, 128, 3, F16, MODE, GATHER, GLU>(p, epi, n_ab, 0, ps, qs, sE);
#endif
}

// -------------------------------------------------------- few rows per expert
// A workgroup takes up to 32 rows of one expert and 32 channels (SwiGLU: 16 gate and
// their 16 up channels; gradient by the rows: 64 inputs).  Its four wavefronts take
// every fourth step of the sum and add their sums through LDS; each keeps four
// stages of weights of its own (4 KB: 32 channels x 64 inputs, or 32 channels x 64
// inputs transposed), filled by LDS-DMA three steps ahead, and the rows' part in
// registers: no barrier before the end.  The weights' bytes bound it: one row for each
// of 8 experts of 2048 x 2048 13 us (5.2 TB/s), SwiGLU 15, by the rows 12; 16 rows of one expert of
// 4096 x 4096 13 us, where tiles of 128 leave most CUs empty (32).
template <bool F16, int MODE, bool GATHER, bool GLU>
__device__ __forceinline__ void small_body(const GemmK& p, int epi, int n_cb, char* r0, char* r1, char* r2, char* r3) {
  constexpr int AT = MODE == kForward ? 2 : 4;       // a tiles of 16
  constexpr int ST = MODE == kForward ? 64 : 32;     // k of a step
  constexpr int SUB = ST / 32, NS = 4, OPS = 4 + 2 * SUB;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4, I = p.N / 2;
  int idx = blockIdx.x;
  RowTile t;
  if (!find_tile<32>(p.seg, p.E, p.M_total, n_cb, idx, t)) return;
  const int cb = idx % n_cb, b0 = t.r0 + idx / n_cb * 32, s1 = t.s1;
  const int red = MODE == kForward ? p.K : p.N, na = MODE == kForward ? p.N : p.K;
  const uint16_t* const w = p.w + (size_t)t.e * p.N * p.K;

  // this lane's part of a step's four DMAs, and its rows
  uint32_t po[4];
  int ck = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 3);
    if constexpr (MODE == kForward) {
      const int c = (lane & 7) ^ swz(r);
      ck = 8 * c;  // (the same in every DMA)
      const int ch = GLU ? (i < 2 ? 16 * cb + r : I + 16 * cb + r - 16) : 32 * cb + r;
      po[i] = row_offset(ch, p.N, p.K, 8 * c);
    } else {
      const int ch = 64 * cb + 8 * (((((lane >> 1) & 3) ^ tswz4(r)) << 1) + (lane & 1));
      po[i] = ch < p.K ? ((uint32_t)r * (uint32_t)p.K + ch) * 2 : kOut;
    }
  }
  uint32_t qo[2][SUB];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = 16 * x + col;
    uint32_t from = r;
    if constexpr (GATHER) from = (uint32_t)min(max(p.div(p.gather[min(b0 + r, s1 - 1)]), 0), p.A_rows - 1);
    const uint32_t first = b0 + r < s1 ? (from * (uint32_t)red + 8 * quad) * 2 : kOut;
#pragma unroll
    for (int u = 0; u < SUB; ++u) qo[x][u] = offset_sum(first, 64 * u);
  }
  const uint16_t* const rows = MODE == kForward ? p.a : p.dy;
  const rsrc_t qr = scalar_rsrc(GATHER ? rows : rows + (size_t)b0 * red,
                                GATHER ? (uint32_t)((size_t)p.A_rows * red * 2) : (uint32_t)((size_t)min(s1 - b0, 32) * red * 2));
  char* const ring[NS] = {r0 + wv * 4096, r1 + wv * 4096, r2 + wv * 4096, r3 + wv * 4096};
  u32x4 q[NS][2][SUB];
  auto load = [&](auto slot_tag, int step) {
    constexpr int S = decltype(slot_tag)::value;
    const int k0 = ST * (4 * step + wv), left = red - k0;
    const uint32_t adv = left > 0 ? 2u * (uint32_t)k0 : 0u;
    if constexpr (MODE == kForward) {
      const rsrc_t pr = scalar_rsrc(w, (uint32_t)((size_t)p.N * p.K * 2));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(pr, (__attribute__((address_space(3))) void*)(ring[S] + 1024 * i), 16,
                                                 ck < left ? po[i] : kOut, adv, 0, 0);
    } else {
      const rsrc_t pr = scalar_rsrc(w + (size_t)(left > 0 ? k0 : 0) * p.K, (uint32_t)max(min(left, 32), 0) * (2u * (uint32_t)p.K));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(pr, (__attribute__((address_space(3))) void*)(ring[S] + 1024 * i), 16, po[i], 0, 0, 0);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int u = 0; u < SUB; ++u) q[S][x][u] = buf_x4(qr, 32 * u + 8 * quad < left ? qo[x][u] : kOut, adv);
  };
  f32x4 acc[AT][2] = {};
  auto multiply = [&](auto slot_tag) {
    constexpr int S = decltype(slot_tag)::value;
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      u32x4 a[AT];
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        if constexpr (MODE == kForward) {
          a[i] = *reinterpret_cast<const u32x4*>(ring[S] + (16 * i + col) * 128 + (((4 * u + quad) ^ swz(col)) << 4));
        } else {
          const int k = 8 * quad + ((lane >> 2) & 3);
          const char* at = ring[S] + k * 128 + ((i ^ tswz4(k)) << 5) + ((lane & 3) << 3);
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
          // (rows k + 4 .. k + 7: bit 1 of the place flips with neither)
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 512));
          const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
          a[i] = u32x4{l[0], l[1], h[0], h[1]};
        }
      }
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) acc[i][x] = mfma16t<F16>(a[i], q[S][x][u], acc[i][x]);
    }
  };
  // Steps of a wavefront, a multiple of four: past the sum's end zeros.
  const int n = ((red + 4 * ST - 1) / (4 * ST) + NS - 1) / NS * NS;
  load(std::integral_constant<int, 0>{}, 0);
  load(std::integral_constant<int, 1>{}, 1);
  load(std::integral_constant<int, 2>{}, 2);
  auto turn = [&](auto slot_tag, int step) {
    constexpr int S = decltype(slot_tag)::value;
    __builtin_amdgcn_sched_barrier(0);
    load(std::integral_constant<int, (S + 3) % NS>{}, step + 3);
    __builtin_amdgcn_sched_barrier(0);
    // three newer steps may be on their way (vmcnt, whose upper two bits lie apart)
    __builtin_amdgcn_s_waitcnt(0x0F70 | (3 * OPS & 15) | (3 * OPS >> 4) << 14);
    __builtin_amdgcn_sched_barrier(0);
    multiply(slot_tag);
  };
  for (int step = 0; step < n; step += NS) {
    turn(std::integral_constant<int, 0>{}, step);
    turn(std::integral_constant<int, 1>{}, step + 1);
    turn(std::integral_constant<int, 2>{}, step + 2);
    turn(std::integral_constant<int, 3>{}, step + 3);
  }
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0070);  // the last loads too: the stages hold the sums next
  // a tile's sums of wavefront w at 4 KB of stage i / 2
  auto sums = [&](int i, int x, int w) { return reinterpret_cast<f32x4*>((i < 2 ? r0 : r1) + w * 4096) + (2 * (i & 1) + x) * 64; };
#pragma unroll
  for (int i = 0; i < AT; ++i)
#pragma unroll
    for (int x = 0; x < 2; ++x) sums(i, x, wv)[lane] = acc[i][x];
  __syncthreads();
  auto total = [&](int i, int x, int l) {
    f32x4 v = sums(i, x, 0)[l];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += sums(i, x, w)[l];
    return v;
  };
  auto narrow = [&](const f32x4& v, bool f16) {
    return f16 ? u32x2{pack16x2<true>(v[0], v[1]), pack16x2<true>(v[2], v[3])} : u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  };
  // Four channels of a row per thread, neighbouring threads the row's next ones.
  constexpr int TILES = GLU && MODE == kForward ? 1 : AT;
  for (int o = threadIdx.x; o < TILES * 128; o += 256) {
    const int i = o / 4 % TILES, r = o / (4 * TILES), qd = o & 3;
    const int row = b0 + r, x = r >> 4, l = 16 * qd + (r & 15);
    if (row >= s1) continue;
    if constexpr (GLU && MODE == kForward) {
      const int ch = 16 * cb + 4 * qd;
      if (ch >= I) continue;
      const f32x4 g = total(0, x, l), u = total(1, x, l);
      if (p.pre_out) {
        uint16_t* const pre = p.pre_out + (size_t)row * p.N + ch;
        *reinterpret_cast<u32x2*>(pre) = narrow(g, F16);
        *reinterpret_cast<u32x2*>(pre + I) = narrow(u, F16);
      }
      f32x4 h;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = silu(g[j]) * u[j];
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + (size_t)row * I + ch) = narrow(h, F16);
    } else {
      const int ch = 16 * AT * cb + 16 * i + 4 * qd;
      if (ch >= na) continue;
      const f32x4 v = total(i, x, l);
      if constexpr (GLU) {
        const size_t at = (size_t)row * 2 * p.K + ch;
        const u32x2 gv = *reinterpret_cast<const u32x2*>(p.pre_in + at), uv = *reinterpret_cast<const u32x2*>(p.pre_in + at + p.K);
        f32x4 dg, du;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t gw = gv[j >> 1], uw = uv[j >> 1];
          const float2 d = swiglu_grad<F16>(v[j], (uint16_t)(j & 1 ? gw >> 16 : gw & 0xFFFFu), (uint16_t)(j & 1 ? uw >> 16 : uw & 0xFFFFu));
          dg[j] = d.x;
          du[j] = d.y;
        }
        uint16_t* const d = static_cast<uint16_t*>(p.out) + at;
        *reinterpret_cast<u32x2*>(d) = narrow(dg, F16);
        *reinterpret_cast<u32x2*>(d + p.K) = narrow(du, F16);
      } else if (epi == kEpiF32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + (size_t)row * na + ch) = v;
      } else {
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + (size_t)row * na + ch) = narrow(v, epi == kEpiF16);
      }
    }
  }
}
template <bool F16, int MODE, bool GATHER, bool GLU>
__global__ __launch_bounds__(256, 2) void small_kernel(GemmK p, int epi, int n_cb) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __attribute__((aligned(1024))) char r0[16384], r1[16384], r2[16384], r3[16384];
  small_body<F16, MODE, GATHER, GLU>(p, epi, n_cb, r0, r1, r2, r3);
#endif
}

// The weights' gradient from the splits' sums, added in order: with it 8192 rows of one
// expert of 64 x 64 take 16 us and not 159, of 2048 x 2048 76 and not 163.
__global__ __launch_bounds__(256) void splits_kernel(const f32x4* __restrict__ sums, int splits, size_t n4, int epi, void* __restrict__ out) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (size_t)gridDim.x * 256) {
    f32x4 v = sums[i];
    for (int k = 1; k < splits; ++k) v += sums[i + (size_t)k * n4];
    if (epi == kEpiF32) static_cast<f32x4*>(out)[i] = v;
    else
      static_cast<u32x2*>(out)[i] = epi == kEpiF16 ? u32x2{pack16x2<true>(v[0], v[1]), pack16x2<true>(v[2], v[3])}
                                                   : u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

GemmK kernel_args(const Gemm16Args& a) {
  return GemmK{static_cast<const uint16_t*>(a.w), static_cast<const uint16_t*>(a.a), static_cast<const uint16_t*>(a.dy),
               a.E, a.N, a.K, a.A_rows, a.M_total, a.gather, pair_div(a.gather ? a.k : 1), a.seg,
               static_cast<const uint16_t*>(a.pre_in), static_cast<uint16_t*>(a.pre_out), a.out, 1};
}
// Upper bound of the tiles of `rows` rows: one partial tile per segment that has rows.
int64_t row_tiles(int M_total, int E, int rows) { return (int64_t)M_total / rows + (E < M_total ? E : M_total); }

template <int T, bool F16, int MODE, bool GATHER, bool GLU>
int launch_tiles(const Gemm16Args& a, hipStream_t s) {
  const int na = MODE == kForward ? a.N : a.K, n_ab = (na + T - 1) / T, n_bb = (a.N + T - 1) / T;
  GemmK k = kernel_args(a);
  int epi = a.epilogue;
  if (MODE == kWeights && T == 128) {
    k.splits = gemm16_splits(a.E, a.N, a.K, a.M_total, a.kernel);
    if (k.splits > 1) {
      k.out = a.ws;
      epi = kEpiF32;
    }
  }
  const int64_t tiles = (MODE == kWeights ? (int64_t)a.E * k.splits * n_bb : row_tiles(a.M_total, a.E, T)) * n_ab;
  if (tiles >= ((int64_t)1 << 30)) return (int)hipErrorInvalidConfiguration;
  const int64_t most = T == 256 ? kCUs : 2 * kCUs;  // workgroups that fit the chip at once
  const int64_t wgs = tiles < most ? (tiles + 7) / 8 * 8 : most;
  hipLaunchKernelGGL((tile_kernel<T, F16, MODE, GATHER, GLU>), dim3((unsigned)wgs), dim3(2 * T), 0, s, k, epi, n_ab, n_bb);
  const int e = (int)hipGetLastError();
  if (k.splits == 1 || e != 0) return e;
  const size_t n4 = (size_t)a.E * a.N * a.K / 4, blocks = (n4 + 255) / 256;
  hipLaunchKernelGGL(splits_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s, static_cast<const f32x4*>(a.ws),
                     k.splits, n4, a.epilogue, a.out);
  return (int)hipGetLastError();
}
template <int T, int MODE, bool GATHER, bool GLU>
int launch_typed(const Gemm16Args& a, hipStream_t s) {
  return a.dtype == 2 ? launch_tiles<T, true, MODE, GATHER, GLU>(a, s) : launch_tiles<T, false, MODE, GATHER, GLU>(a, s);
}
template <bool F16, int MODE, bool GATHER, bool GLU>
int launch_deep(const Gemm16Args& a, hipStream_t s) {
  const int n_ab = ((MODE == kForward ? a.N : a.K) + 127) / 128;
  const int64_t tiles = row_tiles(a.M_total, a.E, 128) * n_ab;
  if (tiles >= ((int64_t)1 << 30)) return (int)hipErrorInvalidConfiguration;
  const int64_t wgs = tiles < kCUs ? (tiles + 7) / 8 * 8 : kCUs;
  hipLaunchKernelGGL((deep_kernel<F16, MODE, GATHER, GLU>), dim3((unsigned)wgs), dim3(256), 0, s, kernel_args(a), a.epilogue, n_ab);
  return (int)hipGetLastError();
}
template <bool F16, int MODE, bool GATHER, bool GLU>
int launch_small(const Gemm16Args& a, hipStream_t s) {
  const int n_cb = MODE == kRows ? (a.K + 63) / 64 : (a.N + 31) / 32;
  const int64_t wgs = gemm16_small_workgroups(MODE, a.E, a.N, a.K, a.M_total);
  if (wgs >= kGemm16MostSmall) return (int)hipErrorInvalidConfiguration;  // (refused before)
  hipLaunchKernelGGL((small_kernel<F16, MODE, GATHER, GLU>), dim3((unsigned)wgs), dim3(256), 0, s, kernel_args(a), a.epilogue, n_cb);
  return (int)hipGetLastError();
}
template <int MODE, bool GATHER, bool GLU>
int launch(const Gemm16Args& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int path = gemm16_path(MODE, a.E, a.N, a.K, a.M_total, a.kernel);
  if (path == 256) return launch_typed<256, MODE, GATHER, GLU>(a, s);
  if (path == 128) return launch_typed<128, MODE, GATHER, GLU>(a, s);
  if constexpr (MODE == kWeights) return (int)hipErrorInvalidValue;
  else if (path == kGemm16Deep) return a.dtype == 2 ? launch_deep<true, MODE, GATHER, GLU>(a, s) : launch_deep<false, MODE, GATHER, GLU>(a, s);
  else return a.dtype == 2 ? launch_small<true, MODE, GATHER, GLU>(a, s) : launch_small<false, MODE, GATHER, GLU>(a, s);
}
}  // namespace

int launch_gemm16(const Gemm16Args& a, void* stream) {
  if (a.gather) return a.epilogue == kEpiSwiglu ? launch<kForward, true, true>(a, stream) : launch<kForward, true, false>(a, stream);
  return a.epilogue == kEpiSwiglu ? launch<kForward, false, true>(a, stream) : launch<kForward, false, false>(a, stream);
}
int launch_gemm16_grad_rows(const Gemm16Args& a, void* stream) {
  return a.epilogue == kEpiSwigluGrad ? launch<kRows, false, true>(a, stream) : launch<kRows, false, false>(a, stream);
}
int launch_gemm16_grad_weights(const Gemm16Args& a, void* stream) {
  return a.gather && a.M_total > 0 ? launch<kWeights, true, false>(a, stream) : launch<kWeights, false, false>(a, stream);
}

}  // namespace moe
