// Interface between the host layer (abi.cpp: argument validation, status
// codes, error details) and the device side (the .hip sources: kernels and
// the launches that issue them).  Plain C++ types only: the host layer
// builds without the HIP headers, so it can also be linked against stand-in
// launchers in a CPU-only test build.
//
// Every launch returns the HIP status of what it issued (0 = success) and
// never synchronises with the device.  Streams travel as void* (hipStream_t).
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace moe {

// --------------------------------------------------------- device runtime
// 0 on success, else a HIP error code.
int rt_current_device(int* dev);
// Architecture name of device `dev` (e.g. "gfx950:sramecc+:xnack-") into name[n].
int rt_device_arch(int dev, char* name, size_t n);
// Returns and clears the calling thread's last HIP error (0 if none).
int rt_take_error();
const char* rt_error_string(int err);
// rows pieces of width bytes, pitch bytes apart in both buffers, host (pinned) to device, on stream
int rt_copy_rows_h2d(void* dst, const void* src, size_t rows, size_t pitch, size_t width, void* stream);

// ---------------------------------------------------------------- routing
int launch_route_topk(const float* logits, int T, int E, int k, int32_t* ids, float* w, void* stream);

// --------------------------------------------------------------- grouping
constexpr int kPermuteChunk = 2048;     // pairs per workgroup in the multi-workgroup grouping
constexpr int kPermuteSmallMax = 4096;  // up to this many pairs: one workgroup
constexpr int kRoutePermuteMaxE = 64;   // fused routing + grouping: at most this many experts
struct PermuteArgs {
  const int32_t* ids;
  const uint8_t* bits;
  int P, k, E, S;
  int32_t* counts;
  int32_t* seg_offsets;
  int32_t* sorted_pair;
  int32_t* pair_pos;
  const uint16_t* x;
  int H;
  uint16_t* x_perm;
  void* ws;
};
size_t permute_workspace_bytes(int P, int E, int S);
int launch_permute(const PermuteArgs& a, void* stream);
// Routing + grouping in one launch (E <= 64 experts, T*k <= 4096 pairs).
bool route_permute_fusable(int T, int k, int E);
int launch_route_permute(const float* logits, int T, int E, int k, const uint8_t* bits, int32_t* ids, float* w,
                         int32_t* counts, int32_t* seg_offsets, int32_t* sorted_pair, int32_t* pair_pos, void* ws,
                         void* stream);

// ---------------------------------------------------------------- combine
// y_dtype: MOE_DTYPE_BF16, MOE_DTYPE_F32 or MOE_DTYPE_F16 (validated by the caller)
int launch_combine(const void* y, int y_dtype, const int32_t* pos, const int32_t* n_valid, const float* w, int T,
                   int k, int H, uint16_t* out, void* stream);

// ---------------------------------------------------------- grouped GEMM
// Weight descriptor as the kernels see it (tiled layout only).
struct QWeights {
  int fmt;  // 1 INT4, 2 MWQ, 3 DELTA2, 4 per-expert widths
  int E, N, K, G, z, n_sal;
  const int32_t* xbits;  // per-expert widths / zero points (host arrays, format 4)
  const int32_t* xzero;
  const uint8_t* codes;
  const uint8_t* p3;
  const uint8_t* p4;
  const uint16_t* scales;
  const int32_t* sal_idx;
  const uint16_t* sal_val;
  const uint16_t* base;
};
struct QGemmArgs {
  QWeights w;
  const uint16_t* A;
  int A_rows;
  const int32_t* gather;
  int k;
  const int32_t* seg_offsets;
  int nseg;
  int M_total;
  int epilogue;  // 0 bf16, 1 SwiGLU bf16, 2 fp32
  int kernel;    // MOE_KERNEL_* (0 = chosen from the shapes)
  void* out;
  void* ws;
};
// Whether `kernel` (MOE_KERNEL_*) can run format `fmt`.
bool qgemm_kernel_supported(int fmt, int kernel);
// Workspace bytes for either epilogue (the larger need) with that kernel choice.
size_t qgemm_workspace_bytes(const QWeights& w, int A_rows, int M_total, int kernel);
int launch_qgemm(const QGemmArgs& a, void* stream);
// The no-allocation grouped GEMM's device scratch: its size, and its address
// on the current device (looked up once per device).
constexpr size_t kStaticScratchBytes = (size_t)8 << 20;
int qgemm_static_scratch(void** ptr);
// Planning (plan.cpp).  path: 0 = 16-row tiles (DELTA2: 32-row tiles), 1 = 16-row
// tiles of one width (MWQ), 64 / 65 = 64-row tiles with 8 / 4 wavefront
// columns, 128 = 128-row register-fed tiles, 2 = 128-row LDS-DMA (INT4, MWQ),
// 3 = 128-row LDS-DMA delta kernel.
int pick_path(const QWeights& w, int M_total, int nseg, int epi, int kernel);
int decode_splits(int n_items, int K);
int decode_row_tiles(int fmt, int path, int M_total, int E);

// ----------------------------------------------------------------- repack
constexpr int kMaxMixedExperts = 256;
int launch_repack(const QWeights& src, const QWeights& dst, void* stream);
size_t tiled_salient_bytes(int E, int N, int n_sal);

// ---------------------------------------------------------- scored routing
struct ScoredArgs {
  const float* logits;
  const float* bias;  // or nullptr
  int T, E, k;
  int score;  // MOE_SCORE_*
  int n_group, topk_group, group_top, renorm;
  float scale;
  int32_t* ids;
  float* w;
};
int launch_route_scored(const ScoredArgs& a, void* stream);
// The start of a layer's call in one launch: routing, the quantisation of n8
// 8-value groups (0: none), and for few tokens the grouping of the pairs too
// (*grouped says whether).
struct FrontRows {
  const void* x;
  int dtype, fmt;  // MOE_DTYPE_*, MOE_MX_*
  size_t n8;
  uint8_t* codes;
  uint8_t* scales;
};
struct FrontGroups {
  int32_t* counts;
  int32_t* seg_offsets;
  int32_t* sorted_pair;
  int32_t* pair_pos;
  uint32_t* flag;
  int* chunk_hist;  // mx_layer_workspace_bytes behind the flag's 256 bytes
};
// Tokens per workgroup of the layer's start where it also counts the pairs (ns:
// experts per lane; the registers of 9 and more allow half), front_chunk_tokens:
// the same for E experts, or 0 where it does not count; the workspace.
constexpr int chunk_tokens(int ns) { return ns <= 8 ? 16 : 8; }
int front_chunk_tokens(int T, int k, int E);
size_t mx_layer_workspace_bytes(int T, int k, int E);
int launch_mx_front(const ScoredArgs& a, const FrontRows& q, const FrontGroups& g, bool* grouped, void* stream);

// ----------------------------------------------------------------- MX rows
// dtypes MOE_DTYPE_*, fmt MOE_MX_*
int launch_quantize_mx(const void* x, int x_dtype, int64_t rows, int K, int fmt, uint8_t* codes, uint8_t* scales,
                       void* stream);
int launch_dequantize_mx(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, int fmt, int out_dtype,
                         void* out, void* stream);
struct NormArgs {
  const void* x;
  const void* residual;  // or nullptr
  const void* weight;
  int dtype;
  int64_t rows;
  int H;
  float eps;
  void* sum;  // or nullptr
  void* y;    // or nullptr
  int fmt;    // MOE_MX_*, or 0: no MX output
  uint8_t* codes;
  uint8_t* scales;
};
constexpr int kNormMaxH = 16384;
int launch_rmsnorm_mx(const NormArgs& a, void* stream);

// -------------------------------------------------------- MX grouped product
struct MxGemmArgs {
  const uint8_t* wcodes;  // tiled
  const uint8_t* wscales;
  int E, N, K;
  const uint8_t* a;
  const uint8_t* as;
  int a_fmt;  // MOE_MX_*
  int A_rows;
  const int32_t* gather;
  int k;
  const int32_t* seg;
  int M_total;
  int epilogue;
  int kernel;  // MOE_KERNEL_*
  void* out;
  uint8_t* out_scales;
};
int launch_mx_repack(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* tcodes,
                     uint8_t* tscales, void* stream);
// Planning (plan.cpp): 0, 64 or 128.
constexpr int kMxSplit = 65;  // 64-row tiles (e2m1 rows) with K split over two groups of wavefronts
int mxgemm_path(int M_total, int E, int N, int K, bool e2m1, int kernel);
int launch_mxgemm(const MxGemmArgs& a, void* stream);

}  // namespace moe
