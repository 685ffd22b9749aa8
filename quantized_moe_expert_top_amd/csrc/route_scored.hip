// Expert choice from scores of all experts: softmax or sigmoid, a choice bias,
// expert groups, top-k, renormalised and scaled weights.
//
// One wavefront per token; lane l owns experts l, l + 64, ... (NS per lane).
// The choice is defined on float64 scores, but float64 exponentials of all
// experts and 64-bit arg-max rounds through LDS shuffles took 18 us for 8192
// tokens of 64 experts and 47 us for 16384 of 256 (0.5 and 3.6 us of memory
// traffic).  So the choice is prepared in fp32 and settled in float64:
//   1. fp32 keys, each within a margin of the choice score;
//   2. a key that at least k experts reach and few more do, by bisection (one
//      compare and ballot per 64 experts and step); every expert within the
//      margins of it can be among the first k and becomes a candidate;
//   3. candidate i in lane i, in index order: its float64 score, its rank among
//      the candidates, the weights of the first k; four tokens' at a time by one
//      wavefront of four.
// Groups are chosen from the keys too, or from float64 scores where two group
// scores at the border are within the margins.  Where the candidates exceed the
// 64 lanes (many equal scores) the token takes float64 rounds over all experts.
// Every way gives the same result.  8192 tokens of 64 experts take 5.6 us, 16384
// of 256 in 8 groups 18, bound by instruction issue (steps 1 and 2); one token 2.7,
// a chain of two loads and the float64 step.
#include <float.h>

#include <utility>

#include "mx.h"
#include "permute_dev.h"

namespace moe {

namespace {
constexpr int kWavesPerBlock = 4;

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ __forceinline__ double neg_inf() { return -__builtin_inf(); }

// float64 scores and choice scores of the lane's experts, by the definition.
// top: the largest logit (softmax).  Reads the logits again, so that no register
// of the usual path is kept for it.
template <int NS>
__device__ __forceinline__ void exact_scores(const ScoredArgs& a, int t, float top, double (&score)[NS], double (&c)[NS]) {
  const int lane = threadIdx.x & 63;
  const float* row = a.logits + (size_t)t * a.E;
  float x[NS], b[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int e = lane + 64 * s;
    const float v = e < a.E ? row[e] : -__builtin_inff();
    x[s] = v != v ? -__builtin_inff() : fminf(v, FLT_MAX);
    b[s] = (a.bias && e < a.E) ? a.bias[e] : 0.0f;
  }
  if (a.score == 0) {
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
}

// The open groups (bit g) by float64 sums; buf: the wavefront's LDS.
template <int NS>
__device__ __forceinline__ uint64_t exact_groups(const ScoredArgs& a, const double (&c)[NS], double* buf) {
  const int lane = threadIdx.x & 63;
  const int size = a.E / a.n_group;
#pragma unroll
  for (int s = 0; s < NS; ++s) buf[lane + 64 * s] = c[s];
  wave_fence();
  const int sh = 31 - __builtin_clz(64 / a.n_group), P = 1 << sh, g = lane >> sh;
  double best = neg_inf(), second = neg_inf();
  if (g < a.n_group)
    for (int i = lane & (P - 1); i < size; i += P) {
      const double v = buf[g * size + i];
      second = v > best ? best : (v > second ? v : second);
      best = v > best ? v : best;
    }
  for (int off = 1; off < P; off <<= 1) {
    const double ob = __shfl_xor(best, off, 64), os = __shfl_xor(second, off, 64);
    const double low = best < ob ? best : ob, hi2 = second > os ? second : os;
    best = best > ob ? best : ob;
    second = low > hi2 ? low : hi2;
  }
  if (a.group_top == 2 && second > neg_inf()) best += second;
  int before = 0;
  for (int j = 0; j < a.n_group; ++j) {
    const double v = __shfl(best, j << sh, 64);
    before += (v > best || (v == best && j < g)) ? 1 : 0;
  }
  const uint64_t by_lane = __ballot(g < a.n_group && before < a.topk_group && (lane & (P - 1)) == 0);
  wave_fence();
  uint64_t open = 0;
  for (int j = 0; j < a.n_group; ++j) open |= ((by_lane >> (j << sh)) & 1) << j;
  return open;
}

// float64 over all experts: the definition, step by step.
template <int NS>
__device__ __forceinline__ void route_exact(const ScoredArgs& a, int t, float top, double* buf, int* hist) {
  const int lane = threadIdx.x & 63;
  double score[NS], c[NS];
  exact_scores<NS>(a, t, top, score, c);
  if (a.n_group > 1) {
    const uint64_t open = exact_groups<NS>(a, c, buf);
    const int size = a.E / a.n_group;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (lane + 64 * s < a.E && !((open >> ((lane + 64 * s) / size)) & 1)) c[s] = neg_inf();
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
      if (hist) atomicAdd(&hist[none ? a.E : bi], 1);
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

// Signed integer that orders like the float (NaN-free).
__device__ __forceinline__ int order_key(float f) {
  const int i = __builtin_bit_cast(int, f);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float key_value(int k) {
  return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7FFFFFFF));
}
// Maximum over the wavefront (rows of 16 by shifts, then row broadcasts; the
// last lane has it).
__device__ __forceinline__ int wave_imax(int v) {
#define MOE_STEP(CTRL, RMASK)                                                                  \
  {                                                                                            \
    const int o = __builtin_amdgcn_update_dpp((int)0x80000000, v, CTRL, RMASK, 0xF, false);    \
    v = v > o ? v : o;                                                                         \
  }
  MOE_STEP(0x111, 0xF) MOE_STEP(0x112, 0xF) MOE_STEP(0x114, 0xF) MOE_STEP(0x118, 0xF)
  MOE_STEP(0x142, 0xA) MOE_STEP(0x143, 0xC)
#undef MOE_STEP
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ double readlane_f64(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Keys and how far they are from what orders the experts:
//   float64 softmax scores plus bias, rounded (SOFT_ALL): 2^-24 relative;
//   without a bias, where no scores are added up: the logit itself, which the
//   scores ascend with (float64 scores of logits closer than the margin may
//   tie; where the scores reach 0 or 1 in float64 they tie over wider
//   distances, so the keys end 700 below the largest logit, or at -700 and 20);
//   else the fp32 sigmoid plus bias: 1.9 * 2^-23 (the exponent's rounding, 2^-24
//   times s (1 - s) |x| <= 0.23; one ulp of the exponential times s (1 - s); half
//   an ulp of the sum and one of the reciprocal) and 2^-24 relative.
// kMargin * (1 + |key|), or kMargin * |key| with SOFT_ALL, is above all of these.
constexpr float kMargin = 0x1p-22f;
constexpr int kSpare = 6;  // candidates beyond k that cost less than another step of the bisection

// SOFT_ALL: the softmax denominator is needed (a bias, weights that are not
// renormalised, sums of two scores per group): float64 exponentials of all
// experts give it and the keys.
//
// The first two steps for token t by this wavefront: the number of candidates,
// listed at the start of buf (64 * NS doubles of LDS of the wavefront's own); or
// -1 where they exceed the lanes and the token was settled over all experts.
// hist: E + 1 counters in LDS that its pairs' experts (E: none) are added to, or
// nullptr.
template <int NS, bool SOFT_ALL>
__device__ __forceinline__ int route_candidates(const ScoredArgs& a, int t, double* buf, int* hist, float& top,
                                                double& soft_sum) {
  const int lane = threadIdx.x & 63;
  const float* row = a.logits + (size_t)t * a.E;

  float x[NS], b[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) x[s] = row[min(lane + 64 * s, a.E - 1)];  // no branch between the loads
  if (a.bias) {
#pragma unroll
    for (int s = 0; s < NS; ++s) b[s] = a.bias[min(lane + 64 * s, a.E - 1)];
  } else {
#pragma unroll
    for (int s = 0; s < NS; ++s) b[s] = 0.0f;
  }
  top = -__builtin_inff();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    x[s] = (x[s] != x[s] || lane + 64 * s >= a.E) ? -__builtin_inff() : fminf(x[s], FLT_MAX);
    top = fmaxf(top, x[s]);
  }
  soft_sum = 0.0;
  float key[NS];
  if (a.score == 0) top = key_value(wave_imax(order_key(top)));
  if constexpr (SOFT_ALL) {
    double ex[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      ex[s] = x[s] == -__builtin_inff() ? 0.0 : exp((double)x[s] - (double)top);
      soft_sum += ex[s];
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) soft_sum += __shfl_xor(soft_sum, off, 64);
    const double inv = soft_sum > 0.0 ? 1.0 / soft_sum : 0.0;
#pragma unroll
    for (int s = 0; s < NS; ++s) key[s] = (float)(ex[s] * inv + (double)b[s]);
  } else if (a.score == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) key[s] = fmaxf(x[s], top - 700.0f);
  } else if (!a.bias && (a.n_group == 1 || a.group_top == 1)) {
#pragma unroll
    for (int s = 0; s < NS; ++s) key[s] = fmaxf(fminf(x[s], 20.0f), -700.0f);
  } else {
#pragma unroll
    for (int s = 0; s < NS; ++s) key[s] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[s])) + b[s];
  }
  constexpr float kBase = SOFT_ALL ? 0.0f : 1.0f;
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (x[s] == -__builtin_inff() || key[s] != key[s]) key[s] = -__builtin_inff();

  if (a.n_group > 1) {
    // Best one or two keys of each group: P lanes per group stride over the
    // group's keys in LDS and merge.
    const int size = a.E / a.n_group;
    float* const fk = reinterpret_cast<float*>(buf);
#pragma unroll
    for (int s = 0; s < NS; ++s) fk[lane + 64 * s] = key[s];
    wave_fence();
    const int sh = 31 - __builtin_clz(64 / a.n_group), P = 1 << sh;
    const int g = lane >> sh;
    float best = -__builtin_inff(), second = -__builtin_inff();
    if (g < a.n_group)
      for (int i = lane & (P - 1); i < size; i += P) {
        const float v = fk[g * size + i];
        second = fmaxf(second, fminf(best, v));
        best = fmaxf(best, v);
      }
    for (int off = 1; off < P; off <<= 1) {
      const float ob = __shfl_xor(best, off, 64), os = __shfl_xor(second, off, 64);
      second = fmaxf(fmaxf(second, os), fminf(best, ob));
      best = fmaxf(best, ob);
    }
    float mag = fabsf(best);  // of what the group's score was made from
    if (a.group_top == 2 && second > -__builtin_inff()) {
      mag += fabsf(second);
      best += second;
    }
    // certainly and possibly better groups; one bound of the errors for all
    const bool some = g < a.n_group && best > -__builtin_inff();
    const float err = 2.0f * kMargin * (2.0f * kBase + __builtin_bit_cast(float, wave_imax(some ? __builtin_bit_cast(int, mag) : 0)));
    int sure = 0, maybe = -1;  // (a group is possibly as good as itself)
    for (int j = 0; j < a.n_group; ++j) {
      const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, best), j << sh));
      sure += v > best + err ? 1 : 0;
      maybe += v >= best - err ? 1 : 0;
    }
    const bool mine = g < a.n_group;
    // bit g: group g is open
    uint64_t open = 0;
    // (an infinite bound, from biases of +inf or sums past FLT_MAX, orders nothing)
    if (!(err < __builtin_inff()) || __ballot(mine && sure < a.topk_group && maybe >= a.topk_group)) {
      double score[NS], c[NS];
      wave_fence();
      exact_scores<NS>(a, t, top, score, c);
      open = exact_groups<NS>(a, c, buf);
    } else {
      const uint64_t by_lane = __ballot(mine && maybe < a.topk_group);
      for (int j = 0; j < a.n_group; ++j) open |= ((by_lane >> (j << sh)) & 1) << j;
    }
    // e / size in fp32: (e + 0.5) / size is at least 1 / 2048 away from a whole number
    const float inv = 1.0f / (float)size;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int e = lane + 64 * s;
      const int ge = (int)(((float)e + 0.5f) * inv);
      if (e < a.E && !((open >> ge) & 1)) key[s] = -__builtin_inff();
    }
    wave_fence();
  }

  // How many keys reach `from`
  auto reach = [&](float from) {
    int c = 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) c += __popcll(__ballot(key[s] >= from));
    return c;
  };
  float kmax = key[0], kmin = key[0];
#pragma unroll
  for (int s = 1; s < NS; ++s) kmax = fmaxf(kmax, key[s]);
  kmax = key_value(wave_imax(order_key(kmax)));
  kmin = __builtin_inff();
#pragma unroll
  for (int s = 0; s < NS; ++s) kmin = key[s] == -__builtin_inff() ? kmin : fminf(kmin, key[s]);
  kmin = key_value(~wave_imax(~order_key(kmin)));
  // at least min(k, eligible) keys reach `lo`; fewer than k reach `hi`
  float lo = kmin, hi = kmax;
  int n = kmax == -__builtin_inff() ? 0 : reach(kmin);
  for (int i = 0; n > a.k + kSpare && i < 40; ++i) {
    const float mid = 0.5f * lo + 0.5f * hi;
    if (!(mid > lo && mid < hi)) break;
    const int c = reach(mid);
    if (c >= a.k) {
      lo = mid;
      n = c;
    } else {
      hi = mid;
    }
  }
  if (n >= a.k) {
    lo = fmaxf(lo - 4.0f * kMargin * (kBase + fabsf(lo)), -FLT_MAX);
    n = reach(lo);
  }
  if (n > 64) {  // many (nearly) equal keys
    wave_fence();
    route_exact<NS>(a, t, top, buf, hist);
    return -1;
  }
  int* const list = reinterpret_cast<int*>(buf);
  int base = 0;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const bool in = n > 0 && key[s] >= lo;
    const uint64_t m = __ballot(in);
    if (in) list[base + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] = lane + 64 * s;
    base += __popcll(m);
  }
  wave_fence();
  return n;
}

// float64 score and choice score of candidate cand of token t.
template <bool SOFT_ALL>
__device__ __forceinline__ void candidate_score(const ScoredArgs& a, int t, int cand, float top, double soft_sum,
                                                double& score, double& c) {
  score = 0.0;
  c = neg_inf();
  if (cand < 0) return;
  const double xv = (double)fminf(a.logits[(size_t)t * a.E + cand], FLT_MAX);
  const double bv = a.bias ? (double)a.bias[cand] : 0.0;
  if (a.score == 0) {
    score = exp(xv - (double)top);
    if constexpr (SOFT_ALL) score = score / soft_sum;
  } else {
    score = 1.0 / (1.0 + exp(-xv));
  }
  c = score + bv;
}
// The results of a token, by W lanes (i: this one) that hold its n candidates.
template <int W>
__device__ __forceinline__ void store_token(const ScoredArgs& a, int t, int i, int n, int cand, int rank, double score,
                                            double sum, int* hist) {
  const size_t o = (size_t)t * a.k;
  if (cand >= 0 && rank < a.k) {
    a.ids[o + rank] = cand;
    a.w[o + rank] = sum > 0.0 ? (float)(score / sum * (double)a.scale) : 0.0f;
    if (hist) atomicAdd(&hist[cand], 1);
  }
  if (hist && n < a.k && i == 0) atomicAdd(&hist[a.E], a.k - n);
  for (int j = n + i; j < a.k; j += W) {  // fewer eligible experts than slots
    a.ids[o + j] = -1;
    a.w[o + j] = 0.0f;
  }
}

// The third step for one token: candidates' ranks, the sum over the chosen in
// index order.
template <bool SOFT_ALL>
__device__ __forceinline__ void settle_one(const ScoredArgs& a, int t, int cand, int n, float top, double soft_sum, int* hist) {
  const int lane = threadIdx.x & 63;
  double score, c;
  candidate_score<SOFT_ALL>(a, t, cand, top, soft_sum, score, c);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double cj = readlane_f64(c, j);
    rank += (cj > c || (cj == c && j < lane)) ? 1 : 0;
  }
  double sum = 1.0;
  if (a.renorm) {
    sum = 0.0;
    for (uint64_t left = __ballot(cand >= 0 && rank < a.k); left; left &= left - 1)
      sum += readlane_f64(score, __builtin_ctzll(left));
  }
  store_token<64>(a, t, lane, n, cand, rank, score, sum, hist);
}

// The same for four tokens at once, a row of 16 lanes each (n < 0: nothing left
// to do for the row's token).
template <int J>
__device__ __forceinline__ double row_value(double v) {  // of lane J of the row
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x150 + J, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), 0x150 + J, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int J>
__device__ __forceinline__ int row_before(double c, int i) {  // whether lane J's candidate precedes this one
  const double v = row_value<J>(c);  // by all lanes, outside any condition
  return (int)(v > c) | ((int)(v == c) & (int)(J < i));
}
template <int... J>
__device__ __forceinline__ int row_rank(std::integer_sequence<int, J...>, double c, int i) {
  int rank = 0;
  ((rank += row_before<J>(c, i)), ...);
  return rank;
}
template <int... J>
__device__ __forceinline__ double row_sum(std::integer_sequence<int, J...>, double v) {
  double sum = 0.0;
  ((sum += row_value<J>(v)), ...);
  return sum;
}
constexpr int kRow = 16;
template <bool SOFT_ALL>
__device__ __forceinline__ void settle_rows(const ScoredArgs& a, int t, int cand, int n, float top, double soft_sum, int* hist) {
  const int i = threadIdx.x & (kRow - 1);
  double score, c;
  candidate_score<SOFT_ALL>(a, t, cand, top, soft_sum, score, c);
  const std::make_integer_sequence<int, kRow> lanes{};
  const int rank = row_rank(lanes, c, i);
  const double sum = a.renorm ? row_sum(lanes, cand >= 0 && rank < a.k ? score : 0.0) : 1.0;
  if (n >= 0) store_token<kRow>(a, t, i, n, cand, rank, score, sum, hist);
}

// Token t0 + w by wavefront w of a workgroup of W; the third step of four tokens
// at a time by one of the first W / 4 wavefronts (a lane per candidate of one
// token would leave three quarters of the lanes idle, over the float64
// exponentials and divisions), but for tokens whose candidates exceed a row.
// (One wavefront with a loop over four tokens needs 50 registers more, for what
// the compiler moves out of the loop, and was slower from 128 experts up.)
struct RowToken {
  double soft_sum;
  float top;
  int n;
};
template <int W, int NS, bool SOFT_ALL>
__device__ __forceinline__ void route_block(const ScoredArgs& a, int t0, double (*buf)[64 * NS], RowToken* rows, int* hist) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  float top = 0.0f;
  double soft_sum = 1.0;
  int n = -1;
  if (t0 + wv < a.T) {
    n = route_candidates<NS, SOFT_ALL>(a, t0 + wv, buf[wv], hist, top, soft_sum);
    if (n > kRow) {
      const int* const list = reinterpret_cast<const int*>(buf[wv]);
      settle_one<SOFT_ALL>(a, t0 + wv, lane < n ? list[lane] : -1, n, top, soft_sum, hist);
      n = -1;
    }
  }
  if (lane == 0) rows[wv] = RowToken{soft_sum, top, n};
  __syncthreads();
  if (wv < W / 4) {
    const int r = 4 * wv + lane / kRow, i = lane % kRow;
    const RowToken m = rows[r];
    const int cand = i < m.n ? reinterpret_cast<const int*>(buf[r])[i] : -1;
    settle_rows<SOFT_ALL>(a, t0 + r, cand, m.n, m.top, m.soft_sum, hist);
  }
}
template <int NS, bool SOFT_ALL>
__global__ __launch_bounds__(64 * kWavesPerBlock) void route_scored_kernel(ScoredArgs a) {
  __shared__ double lds[kWavesPerBlock][64 * NS];
  __shared__ RowToken rows[kWavesPerBlock];
  route_block<kWavesPerBlock, NS, SOFT_ALL>(a, blockIdx.x * kWavesPerBlock, lds, rows, nullptr);
}

// ------------------------------------------------- the start of a layer's call
// Routing and the quantisation of the layer's rows do not depend on each other:
// one launch has workgroups for both.  Up to kFrontTokens tokens are routed by
// one workgroup, a wavefront each, which then groups the pairs as well.
template <int NT>
__device__ __forceinline__ void quantize_any(const FrontRows& q, size_t block) {
  const size_t n8 = q.n8;
#define MOE_Q(DT)                                                                        \
  if (q.fmt == kE4M3) quantize_block<DT, kE4M3, NT>(q.x, n8, q.codes, q.scales, block);  \
  else quantize_block<DT, kE2M1, NT>(q.x, n8, q.codes, q.scales, block)
  if (q.dtype == 0) { MOE_Q(0); }
  else if (q.dtype == 1) { MOE_Q(1); }
  else { MOE_Q(2); }
#undef MOE_Q
}

template <int NS, bool SOFT_ALL>
__global__ __launch_bounds__(64 * kWavesPerBlock) void mx_front_kernel(ScoredArgs a, FrontRows q, int n_route) {
  __shared__ double lds[kWavesPerBlock][64 * NS];
  __shared__ RowToken rows[kWavesPerBlock];
  if ((int)blockIdx.x >= n_route) {
    quantize_any<64 * kWavesPerBlock>(q, blockIdx.x - n_route);
    return;
  }
  route_block<kWavesPerBlock, NS, SOFT_ALL>(a, blockIdx.x * kWavesPerBlock, lds, rows, nullptr);
}

constexpr int kFrontTokens = 16, kFrontThreads = 64 * kFrontTokens;
template <int NS, bool SOFT_ALL>
__global__ __launch_bounds__(kFrontThreads) void mx_front_small_kernel(ScoredArgs a, FrontRows q, FrontGroups g) {
  __shared__ double lds[kFrontTokens][64 * NS];
  __shared__ RowToken rows[kFrontTokens];
  __shared__ int hist[64 * NS + 1], tags[kFrontTokens * (64 * NS + 1)], scratch[kFrontTokens + 1];
  __shared__ uint32_t bad;
  if (blockIdx.x > 0) {
    quantize_any<kFrontThreads>(q, blockIdx.x - 1);
    return;
  }
  route_block<kFrontTokens, NS, SOFT_ALL>(a, 0, lds, rows, nullptr);
  __syncthreads();  // the ids, read back by the whole workgroup
  const Keyer kr{a.ids, nullptr, a.E, 1, a.E};
  permute_block<kFrontThreads>(kr, a.T * a.k, g.counts, g.seg_offsets, g.sorted_pair, g.pair_pos, g.flag, hist, tags,
                               scratch, &bad);
}

// More tokens: chunks of a workgroup's tokens, whose workgroups also count their
// pairs per expert (order-free LDS counters), and a second launch in which every
// workgroup sums the chunks' counts for itself (they fit L2) and places the pairs
// of some chunks.  Two launches, 24 us for 8192 tokens x 8 of 64 experts with the
// quantisation of 2048 bf16 each; routing and quantising in one and counting,
// scanning and scattering in three more took 38 us.
template <int NS, bool SOFT_ALL>
__global__ __launch_bounds__(64 * chunk_tokens(NS)) void mx_front_chunk_kernel(ScoredArgs a, FrontRows q, int n_chunks,
                                                                               int* __restrict__ chunk_hist) {
  constexpr int W = chunk_tokens(NS), kThreads = 64 * W;
  __shared__ double lds[W][64 * NS];
  __shared__ RowToken rows[W];
  __shared__ int hist[64 * NS + 1];
  if ((int)blockIdx.x >= n_chunks) {
    quantize_any<kThreads>(q, blockIdx.x - n_chunks);
    return;
  }
  for (int i = threadIdx.x; i <= a.E; i += kThreads) hist[i] = 0;
  __syncthreads();
  route_block<W, NS, SOFT_ALL>(a, blockIdx.x * W, lds, rows, hist);
  __syncthreads();
  for (int i = threadIdx.x; i <= a.E; i += kThreads) chunk_hist[(size_t)blockIdx.x * (a.E + 1) + i] = hist[i];
}

constexpr int kPlaceThreads = 1024;
__global__ __launch_bounds__(kPlaceThreads) void mx_place_kernel(Keyer kr, int P, int chunk_pairs, int per_block,
                                                                 int n_chunks, const int* __restrict__ chunk_hist, FrontGroups g) {
  __shared__ int base[1025], before[1025], tags[(kPlaceThreads / 64) * 1025], scratch[kPlaceThreads / 64 + 1];
  const int tid = threadIdx.x, nk1 = kr.NK + 1, b = blockIdx.x * per_block;  // b: its first chunk
  for (int i = tid; i < nk1; i += kPlaceThreads) base[i] = before[i] = 0;
  for (int i = tid; i < (kPlaceThreads / 64) * nk1; i += kPlaceThreads) tags[i] = -1;
  __syncthreads();
  // a thread per key and slice of the chunks (a few loads one after another each)
  const int slices = max(kPlaceThreads / nk1, 1), slice = tid / nk1;
  for (int key = tid - slice * nk1; key < nk1 && slice < slices; key += kPlaceThreads) {
    int all = 0, prior = 0;
#pragma unroll 8
    for (int c = slice; c < n_chunks; c += slices) {
      const int n = chunk_hist[(size_t)c * nk1 + key];
      all += n;
      prior += c < b ? n : 0;
    }
    atomicAdd(&base[key], all);
    atomicAdd(&before[key], prior);
  }
  __syncthreads();
  if (b == 0) {
    for (int e = tid; e < kr.E; e += kPlaceThreads) g.counts[e] = base[e];
    if (tid == 0) g.flag[0] = base[kr.E] != 0;
    __syncthreads();
  }
  block_exclusive_scan<kPlaceThreads>(base, nk1, scratch);
  if (b == 0)
    for (int i = tid; i < nk1; i += kPlaceThreads) g.seg_offsets[i] = base[i];
  __syncthreads();
  for (int i = tid; i < nk1; i += kPlaceThreads) base[i] += before[i];
  __syncthreads();
  const int p0 = b * chunk_pairs;
  scatter_chunk<kPlaceThreads>(kr, p0, min((int64_t)P, p0 + (int64_t)per_block * chunk_pairs), base, tags, g.sorted_pair, g.pair_pos);
}

inline bool soft_all(const ScoredArgs& a) {
  return a.score == 0 && (a.bias || !a.renorm || (a.n_group > 1 && a.group_top == 2));
}
template <int NS>
void launch_ns(const ScoredArgs& a, hipStream_t s) {
  const dim3 grid((a.T + kWavesPerBlock - 1) / kWavesPerBlock), block(64 * kWavesPerBlock);
  if (soft_all(a)) hipLaunchKernelGGL((route_scored_kernel<NS, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_scored_kernel<NS, false>), grid, block, 0, s, a);
}
inline unsigned quant_blocks(const FrontRows& q, int threads) {
  const size_t per = (size_t)threads * kQuantUnroll;
  return (unsigned)((q.n8 + per - 1) / per);
}
template <int NS>
void launch_front_ns(const ScoredArgs& a, const FrontRows& q, hipStream_t s) {
  const int n_route = (a.T + kWavesPerBlock - 1) / kWavesPerBlock;
  const dim3 grid(n_route + quant_blocks(q, 64 * kWavesPerBlock)), block(64 * kWavesPerBlock);
  if (soft_all(a)) hipLaunchKernelGGL((mx_front_kernel<NS, true>), grid, block, 0, s, a, q, n_route);
  else hipLaunchKernelGGL((mx_front_kernel<NS, false>), grid, block, 0, s, a, q, n_route);
}
template <int NS>
void launch_front_chunk_ns(const ScoredArgs& a, const FrontRows& q, int* hist, hipStream_t s) {
  constexpr int W = chunk_tokens(NS), kThreads = 64 * W;
  const int n_chunks = (a.T + W - 1) / W;
  const dim3 grid(n_chunks + quant_blocks(q, kThreads)), block(kThreads);
  if (soft_all(a)) hipLaunchKernelGGL((mx_front_chunk_kernel<NS, true>), grid, block, 0, s, a, q, n_chunks, hist);
  else hipLaunchKernelGGL((mx_front_chunk_kernel<NS, false>), grid, block, 0, s, a, q, n_chunks, hist);
}
template <int NS>
void launch_front_small_ns(const ScoredArgs& a, const FrontRows& q, const FrontGroups& g, hipStream_t s) {
  const dim3 grid(1 + quant_blocks(q, kFrontThreads)), block(kFrontThreads);
  if (soft_all(a)) hipLaunchKernelGGL((mx_front_small_kernel<NS, true>), grid, block, 0, s, a, q, g);
  else hipLaunchKernelGGL((mx_front_small_kernel<NS, false>), grid, block, 0, s, a, q, g);
}
}  // namespace

int launch_mx_front(const ScoredArgs& a, const FrontRows& q, const FrontGroups& g, bool* grouped, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int tokens = front_chunk_tokens(a.T, a.k, a.E);
  *grouped = (a.T <= kFrontTokens && a.E <= 256) || tokens > 0;
  if (a.T <= kFrontTokens && a.E <= 256) {
    if (a.E <= 64) launch_front_small_ns<1>(a, q, g, s);
    else if (a.E <= 128) launch_front_small_ns<2>(a, q, g, s);
    else launch_front_small_ns<4>(a, q, g, s);
  } else if (tokens > 0) {
    if (a.E <= 64) launch_front_chunk_ns<1>(a, q, g.chunk_hist, s);
    else if (a.E <= 128) launch_front_chunk_ns<2>(a, q, g.chunk_hist, s);
    else if (a.E <= 256) launch_front_chunk_ns<4>(a, q, g.chunk_hist, s);
    else if (a.E <= 512) launch_front_chunk_ns<8>(a, q, g.chunk_hist, s);
    else launch_front_chunk_ns<16>(a, q, g.chunk_hist, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    const Keyer kr{a.ids, nullptr, a.E, 1, a.E};
    const int n_chunks = (a.T + tokens - 1) / tokens, per_block = (n_chunks + 255) / 256;
    hipLaunchKernelGGL(mx_place_kernel, dim3((n_chunks + per_block - 1) / per_block), dim3(kPlaceThreads), 0, s, kr,
                       a.T * a.k, tokens * a.k, per_block, n_chunks, g.chunk_hist, g);
  } else if (a.E <= 64) {
    launch_front_ns<1>(a, q, s);
  } else if (a.E <= 128) {
    launch_front_ns<2>(a, q, s);
  } else if (a.E <= 256) {
    launch_front_ns<4>(a, q, s);
  } else if (a.E <= 512) {
    launch_front_ns<8>(a, q, s);
  } else {
    launch_front_ns<16>(a, q, s);
  }
  return (int)hipGetLastError();
}

int launch_route_scored(const ScoredArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.E <= 64) launch_ns<1>(a, s);
  else if (a.E <= 128) launch_ns<2>(a, s);
  else if (a.E <= 256) launch_ns<4>(a, s);
  else if (a.E <= 512) launch_ns<8>(a, s);
  else launch_ns<16>(a, s);
  return (int)hipGetLastError();
}

}  // namespace moe
