// Device functions of the grouping (a stable counting sort) that more than one
// kernel runs: keys, block-wide scan, the scatter, and all phases in one
// workgroup.
#pragma once
#include "common.h"

namespace moe {

struct Keyer {
  const int32_t* ids;
  const uint8_t* bits;
  int E, S, NK;
  __device__ __forceinline__ int key(int p, uint32_t& bad) const {
    const int id = ids[p];
    bool ok = (unsigned)id < (unsigned)E;
    int k = id;
    if (S == 3) {
      const int b = bits[p];
      ok = ok && b >= 2 && b <= 4;
      k = id * 3 + (4 - b);
    }
    if (!ok) {
      bad = 1;
      return NK;
    }
    return k;
  }
};

__device__ __forceinline__ int nbits_for(int n) {  // bits to tell keys 0..n apart
  int b = 0;
  while ((1 << b) <= n) ++b;
  return b;
}

// Exclusive scan in place over data[0..n) (LDS), all NT threads of the block.
// Returns the total.
template <int NT>
__device__ int block_exclusive_scan(int* data, int n, int* scratch /* >= NT/64 + 1 ints */) {
  constexpr int kThreads = NT;
  const int tid = threadIdx.x;
  const int per = (n + kThreads - 1) / kThreads;
  const int lo = min(n, tid * per), hi = min(n, lo + per);
  int local = 0;
  for (int i = lo; i < hi; ++i) local += data[i];
  // inclusive scan across the wave
  const int lane = tid & 63;
  int v = local;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  if (lane == 63) scratch[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) {
    int run = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
      const int t = scratch[w];
      scratch[w] = run;
      run += t;
    }
    scratch[kThreads / 64] = run;
  }
  __syncthreads();
  int run = scratch[tid >> 6] + v - local;
  for (int i = lo; i < hi; ++i) {
    const int t = data[i];
    data[i] = run;
    run += t;
  }
  const int total = scratch[kThreads / 64];
  __syncthreads();
  return total;
}

// Stable scatter of pairs [p0, p1) whose key bases are in base[] (LDS; base[key]
// = output position of the next pair with that key).  tagbuf: NT/64 * (NK+1)
// ints.  NT threads take NT pairs per step.
template <int NT>
__device__ void scatter_chunk(const Keyer& kr, int p0, int p1, int* base, int* tagbuf, int32_t* sorted_pair,
                              int32_t* pair_pos) {
  constexpr int kThreads = NT;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int nk1 = kr.NK + 1;
  const int nbits = nbits_for(kr.NK);
  const uint64_t lt = (lane == 0) ? 0ull : (~0ull >> (64 - lane));
  int step = 0;
  for (int s0 = p0; s0 < p1; s0 += kThreads, ++step) {
    const int p = s0 + tid;
    const bool act = p < p1;
    uint32_t bad = 0;
    const int key = act ? kr.key(p, bad) : 0;
    uint64_t m = __ballot(act);
    for (int b = 0; b < nbits; ++b) {
      const bool bit = (key >> b) & 1;
      const uint64_t bb = __ballot(bit);
      m &= bit ? bb : ~bb;
    }
    const int rank = __popcll(m & lt);
    const int cnt = __popcll(m);
    const int tag = (step & 0xffff) << 16;
    if (act && rank == 0) tagbuf[wv * nk1 + key] = tag | cnt;
    __syncthreads();
    if (act) {
      int off = base[key];
      for (int w = 0; w < wv; ++w) {
        const int t = tagbuf[w * nk1 + key];
        if ((t & 0xffff0000) == tag) off += t & 0xffff;
      }
      const int pos = off + rank;
      sorted_pair[pos] = p;
      pair_pos[p] = pos;
    }
    __syncthreads();
    if (act && rank == 0) atomicAdd(&base[key], cnt);
    __syncthreads();
  }
}

// All three phases in one workgroup of NT threads.  hist: NK+1 ints,
// tagbuf: NT/64 * (NK+1) ints, scratch: NT/64 + 1 ints (all LDS).
template <int NT>
__device__ void permute_block(const Keyer& kr, int P, int32_t* counts, int32_t* seg_offsets, int32_t* sorted_pair,
                              int32_t* pair_pos, uint32_t* flag, int* hist, int* tagbuf, int* scratch,
                              uint32_t* sbad) {
  const int tid = threadIdx.x;
  const int nk1 = kr.NK + 1;
  for (int i = tid; i < nk1; i += NT) hist[i] = 0;
  for (int i = tid; i < (NT / 64) * nk1; i += NT) tagbuf[i] = -1;  // tag 0xffff never matches step 0..
  if (tid == 0) *sbad = 0;
  __syncthreads();
  uint32_t bad = 0;
  for (int p = tid; p < P; p += NT) atomicAdd(&hist[kr.key(p, bad)], 1);
  if (bad) atomicOr(sbad, 1u);
  __syncthreads();
  for (int e = tid; e < kr.E; e += NT) {
    int c = 0;
    for (int s = 0; s < kr.S; ++s) c += hist[e * kr.S + s];
    counts[e] = c;
  }
  __syncthreads();
  block_exclusive_scan<NT>(hist, nk1, scratch);
  for (int i = tid; i < nk1; i += NT) seg_offsets[i] = hist[i];
  if (tid == 0) flag[0] = *sbad;
  __syncthreads();
  scatter_chunk<NT>(kr, 0, P, hist, tagbuf, sorted_pair, pair_pos);
}

}  // namespace moe
