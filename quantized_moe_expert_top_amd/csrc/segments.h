// Rows grouped by segment, as the kernels of the 16-bit products and of the
// adapters find them: clamped bounds, and the tile that a workgroup takes.
#pragma once
#include "common.h"

namespace moe {

// 16-bit operand type of a kernel: bf16 or fp16.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
// 16 x 16 x 32: lane l holds row l % 16 (of either operand), k = 8*(l / 16) .. + 7;
// the accumulator's register r is row 4*(l / 16) + r of the first, column l % 16.
template <bool F16>
__device__ __forceinline__ f32x4 mfma16t(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}
template <bool F16>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (F16) return f32_to_f16(v);
  else return f32_to_bf16(v);
}
template <bool F16>
__device__ __forceinline__ float widen16(uint16_t v) {
  if constexpr (F16) return f16_to_f32(v);
  else return bf16_to_f32(v);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  if constexpr (F16) return (uint32_t)f32_to_f16(lo) | ((uint32_t)f32_to_f16(hi) << 16);
  else return pack_bf16x2(lo, hi);
}

// make_rsrc with its parts forced into scalar registers: values that the compiler
// worked out on the vector side (clamps, what came by shuffles) would make every
// access through the descriptor a loop over the lanes.
__device__ __forceinline__ rsrc_t scalar_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  return make_rsrc(reinterpret_cast<const void*>((uint64_t)hi << 32 | lo), (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes));
}

// pair / div = (pair * mul) >> (31 + shift), 0 <= pair < 2^31
struct PairDiv {
  uint32_t mul;
  int shift;
  __device__ __forceinline__ int operator()(int pair) const {
    return (int)(__umulhi(2u * (uint32_t)pair, mul) >> shift);
  }
};
inline PairDiv pair_div(int div) {
  int sh = 0;
  while (((int64_t)1 << sh) < div) ++sh;
  return {(uint32_t)((((uint64_t)1 << (31 + sh)) + div - 1) / div), sh};
}

// Segment e's rows, clamped to [0, rows).
__device__ __forceinline__ void segment_rows(const int32_t* seg, int e, int rows, int& s0, int& s1) {
  s0 = min(max(seg[e], 0), rows);
  s1 = min(max(seg[e + 1], s0), rows);
}

// Inclusive sum over the wavefront's lanes (DPP: shifts within rows of 16, then
// row broadcasts).
__device__ __forceinline__ int lane_scan(int v) {
#define MOE_STEP(CTRL, RMASK) v += __builtin_amdgcn_update_dpp(0, v, CTRL, RMASK, 0xF, false);
  MOE_STEP(0x111, 0xF) MOE_STEP(0x112, 0xF) MOE_STEP(0x114, 0xF) MOE_STEP(0x118, 0xF)
  MOE_STEP(0x142, 0xA) MOE_STEP(0x143, 0xC)
#undef MOE_STEP
  return v;
}

// The segment of row tile `idx` of all segments' tiles of TM rows, segment by segment;
// count: all of them.  false: there are fewer.
struct RowTile {
  int e, r0, s1;  // segment, its first row and its end
  int tiles;      // the segment's tiles
};
template <int TM>
__device__ __forceinline__ int segment_tiles(const int32_t* seg, int E, int rows, int e, int& s0, int& s1) {
  s0 = s1 = 0;
  if (e < E) segment_rows(seg, e, rows, s0, s1);
  return (s1 - s0 + TM - 1) / TM;
}
template <int TM>
__device__ __forceinline__ int count_tiles(const int32_t* seg, int E, int rows) {
  const int lane = threadIdx.x & 63;
  int total = 0, s0, s1;
  for (int e0 = 0; e0 < E; e0 += 64)
    total += __builtin_amdgcn_readlane(lane_scan(segment_tiles<TM>(seg, E, rows, e0 + lane, s0, s1)), 63);
  return total;
}
// weight: workgroups per row tile; idx counts workgroups and is reduced to the one
// within the segment.
template <int TM>
__device__ __forceinline__ bool find_tile(const int32_t* seg, int E, int rows, int weight, int& idx, RowTile& t) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int s0, s1;
    const int n = segment_tiles<TM>(seg, E, rows, e0 + lane, s0, s1);
    const int end = lane_scan(n), sum = __builtin_amdgcn_readlane(end, 63) * weight;
    if (idx >= sum) {
      idx -= sum;
      continue;
    }
    const int src = __builtin_ctzll(__ballot(idx < end * weight));
    t.tiles = __builtin_amdgcn_readlane(n, src);
    t.e = e0 + src;
    t.r0 = __builtin_amdgcn_readlane(s0, src);
    t.s1 = __builtin_amdgcn_readlane(s1, src);
    idx -= (__builtin_amdgcn_readlane(end, src) - t.tiles) * weight;
    return true;
  }
  return false;
}

}  // namespace moe
