// C ABI entry points of the experts in 16 bits (grouped product and its
// gradients, the combine's gradient) and of the low-rank adapters: host-side
// validation, then stream-ordered launches.  Plain C++, the manner of abi.cpp.
#include <stdint.h>

#include "moe_qexpert.h"
#include "abi_util.h"
#include "launch.h"

using moe::aligned;
using moe::check_device;
using moe::fail;
using moe::hip_status;
using moe::ok;

namespace {
constexpr int64_t kMaxBytes = (int64_t)1 << 32;  // buffers that the kernels address with 32-bit offsets
bool dtype16(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }
bool known_dtype(int d) { return dtype16(d) || d == MOE_DTYPE_F32; }
bool plain(int epi) { return epi == MOE_EPI_NONE || epi == MOE_EPI_NONE_F16 || epi == MOE_EPI_NONE_F32; }

moe_status check_kernel(int32_t kernel, bool small) {
  if (kernel < MOE_KERNEL_AUTO || kernel > MOE_KERNEL_TILE256)
    return fail(MOE_ERR_BAD_FORMAT, "unknown kernel choice %d", kernel);
  if (kernel != MOE_KERNEL_AUTO && !(small && kernel == MOE_KERNEL_SMALL) && kernel != MOE_KERNEL_TILE128 &&
      kernel != MOE_KERNEL_TILE256)
    return fail(MOE_ERR_UNSUPPORTED, "kernel choice %d does not run this product of 16-bit weights", kernel);
  return MOE_OK;
}

moe_status check_sizes(int32_t dtype, int32_t E, int32_t N, int32_t K, int32_t M_total, int32_t kernel, bool small) {
  if (!dtype16(dtype)) return fail(MOE_ERR_BAD_FORMAT, "dtype %d (bf16 or fp16)", dtype);
  if (E < 1 || E > 1024 || N < 1 || K < 1) return fail(MOE_ERR_BAD_SHAPE, "E=%d N=%d K=%d out of range", E, N, K);
  if (N % 8 != 0 || K % 8 != 0) return fail(MOE_ERR_UNSUPPORTED, "N=%d and K=%d must be multiples of 8", N, K);
  if (N > 1 << 20 || K > 1 << 20) return fail(MOE_ERR_UNSUPPORTED, "N=%d or K=%d above 2^20", N, K);
  if (M_total < 0) return fail(MOE_ERR_BAD_SHAPE, "M_total=%d < 0", M_total);
  // (room for a partial tile's and a last step's rows in 32 bits)
  if (M_total >= 1 << 30) return fail(MOE_ERR_UNSUPPORTED, "M_total=%d of 2^30 or more", M_total);
  if ((int64_t)N * K * 2 >= kMaxBytes)
    return fail(MOE_ERR_UNSUPPORTED, "an expert's weights of %lld bytes (4 GiB or more)", (long long)N * K * 2);
  return check_kernel(kernel, small);
}

// The kernel for few rows is chosen for many only by the caller.
moe_status check_small(int what, int32_t E, int32_t N, int32_t K, int32_t M_total, int32_t kernel) {
  if (kernel != MOE_KERNEL_SMALL || moe::gemm16_small_workgroups(what, E, N, K, M_total) < moe::kGemm16MostSmall) return MOE_OK;
  return fail(MOE_ERR_UNSUPPORTED, "M_total=%d: 2^24 or more tiles of 32 rows with MOE_KERNEL_SMALL", M_total);
}

moe_status check_rows(int32_t K, int32_t A_rows, const int32_t* gather_pair, int32_t k, int32_t M_total) {
  if (A_rows < 0) return fail(MOE_ERR_BAD_SHAPE, "A_rows=%d < 0", A_rows);
  if (gather_pair) {
    if (k < 1) return fail(MOE_ERR_BAD_SHAPE, "k=%d with gather_pair", k);
    if ((int64_t)A_rows * k < M_total) return fail(MOE_ERR_BAD_SHAPE, "A_rows*k < M_total");
    if ((int64_t)A_rows * K * 2 >= moe::kGatherBytes)
      return fail(MOE_ERR_UNSUPPORTED, "gathered rows of %lld bytes (fewer than 4 GiB - 4 MiB)", (long long)A_rows * K * 2);
  } else if (A_rows < M_total) {
    return fail(MOE_ERR_BAD_SHAPE, "A_rows=%d < M_total=%d", A_rows, M_total);
  }
  return MOE_OK;
}
}  // namespace

extern "C" {

moe_status moe_grouped_gemm(const void* w, int32_t dtype, int32_t E, int32_t N, int32_t K, const void* A, int32_t A_rows,
                            const int32_t* gather_pair, int32_t k, const int32_t* seg_offsets, int32_t M_total,
                            int32_t epilogue, int32_t kernel, void* pre, void* out, void* stream) {
  moe_status st = check_sizes(dtype, E, N, K, M_total, kernel, true);
  if (st != MOE_OK) return st;
  if (!plain(epilogue) && epilogue != MOE_EPI_SWIGLU)
    return fail(MOE_ERR_BAD_FORMAT, "epilogue %d of a 16-bit product", epilogue);
  if (epilogue == MOE_EPI_SWIGLU && N % 16 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "N=%d must be a multiple of 16 with a SwiGLU epilogue", N);
  st = check_rows(K, A_rows, gather_pair, k, M_total);
  if (st != MOE_OK) return st;
  st = check_small(0, E, N, K, M_total, kernel);
  if (st != MOE_OK) return st;
  if (M_total == 0) return ok();
  if (!w || !A || !seg_offsets || !out) return fail(MOE_ERR_NULL_ARG, "w, A, seg_offsets and out are required");
  if (pre && epilogue != MOE_EPI_SWIGLU) return fail(MOE_ERR_BAD_FORMAT, "pre goes with the SwiGLU epilogue");
  if (out == A || out == w || pre == A || pre == w || pre == out)
    return fail(MOE_ERR_BAD_SHAPE, "an output shares a buffer");
  if (!aligned(w, 16) || !aligned(A, 16) || !aligned(out, 16) || !aligned(pre, 16))
    return fail(MOE_ERR_MISALIGNED, "w, A, pre and out must be 16-byte aligned");
  if (!aligned(seg_offsets, 4) || !aligned(gather_pair, 4))
    return fail(MOE_ERR_MISALIGNED, "seg_offsets and gather_pair must be 4-byte aligned");
  st = check_device();
  if (st != MOE_OK) return st;
  const moe::Gemm16Args a{w, A, nullptr, dtype, E, N, K, A_rows, gather_pair, k, seg_offsets, M_total, epilogue, kernel,
                          nullptr, pre, out, nullptr};
  return hip_status(moe::launch_gemm16(a, stream), "grouped_gemm launch");
}

moe_status moe_grouped_gemm_grad_rows(const void* w, int32_t dtype, int32_t E, int32_t N, int32_t K, const void* dy,
                                      const int32_t* seg_offsets, int32_t M_total, int32_t epilogue, int32_t kernel,
                                      const void* pre, void* out, void* stream) {
  moe_status st = check_sizes(dtype, E, N, K, M_total, kernel, true);
  if (st != MOE_OK) return st;
  if (!plain(epilogue) && epilogue != MOE_EPI_SWIGLU_GRAD)
    return fail(MOE_ERR_BAD_FORMAT, "epilogue %d of a gradient by the rows", epilogue);
  st = check_small(1, E, N, K, M_total, kernel);
  if (st != MOE_OK) return st;
  if (M_total == 0) return ok();
  if (!w || !dy || !seg_offsets || !out) return fail(MOE_ERR_NULL_ARG, "w, dy, seg_offsets and out are required");
  if ((epilogue == MOE_EPI_SWIGLU_GRAD) != (pre != nullptr))
    return fail(MOE_ERR_NULL_ARG, "pre goes with the SwiGLU gradient epilogue (%d)", epilogue);
  if (out == dy || out == w || out == pre) return fail(MOE_ERR_BAD_SHAPE, "the gradient cannot run in place");
  if (!aligned(w, 16) || !aligned(dy, 16) || !aligned(out, 16) || !aligned(pre, 16))
    return fail(MOE_ERR_MISALIGNED, "w, dy, pre and out must be 16-byte aligned");
  if (!aligned(seg_offsets, 4)) return fail(MOE_ERR_MISALIGNED, "seg_offsets must be 4-byte aligned");
  st = check_device();
  if (st != MOE_OK) return st;
  const moe::Gemm16Args a{w, nullptr, dy, dtype, E, N, K, 0, nullptr, 1, seg_offsets, M_total, epilogue, kernel,
                          pre, nullptr, out, nullptr};
  return hip_status(moe::launch_gemm16_grad_rows(a, stream), "grouped_gemm_grad_rows launch");
}

size_t moe_grouped_gemm_grad_weights_workspace_size(int32_t E, int32_t N, int32_t K, int32_t M_total, int32_t kernel) {
  if (check_sizes(MOE_DTYPE_BF16, E, N, K, M_total, kernel, false) != MOE_OK) return 0;
  ok();
  return moe::gemm16_grad_weights_workspace_bytes(E, N, K, M_total, kernel);
}

moe_status moe_grouped_gemm_grad_weights(const void* dy, const void* A, int32_t dtype, int32_t E, int32_t N, int32_t K,
                                         int32_t A_rows, const int32_t* gather_pair, int32_t k,
                                         const int32_t* seg_offsets, int32_t M_total, int32_t epilogue, int32_t kernel,
                                         void* out, void* workspace, size_t workspace_bytes, void* stream) {
  moe_status st = check_sizes(dtype, E, N, K, M_total, kernel, false);
  if (st != MOE_OK) return st;
  if (!plain(epilogue)) return fail(MOE_ERR_BAD_FORMAT, "epilogue %d of a gradient by the weights", epilogue);
  st = check_rows(K, A_rows, gather_pair, k, M_total);
  if (st != MOE_OK) return st;
  // (an empty batch still has a gradient: zeros)
  if (!out) return fail(MOE_ERR_NULL_ARG, "out is required");
  if (M_total > 0 && (!dy || !A || !seg_offsets)) return fail(MOE_ERR_NULL_ARG, "dy, A and seg_offsets are required");
  if (out == dy || out == A) return fail(MOE_ERR_BAD_SHAPE, "the gradient cannot run in place");
  if (!aligned(dy, 16) || !aligned(A, 16) || !aligned(out, 16) || !aligned(workspace, 16))
    return fail(MOE_ERR_MISALIGNED, "dy, A, out and workspace must be 16-byte aligned");
  if (!aligned(seg_offsets, 4) || !aligned(gather_pair, 4))
    return fail(MOE_ERR_MISALIGNED, "seg_offsets and gather_pair must be 4-byte aligned");
  const size_t need = moe::gemm16_grad_weights_workspace_bytes(E, N, K, M_total, kernel);
  if (need && !workspace) return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "no workspace, %zu bytes needed", need);
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", workspace_bytes, need);
  st = check_device();
  if (st != MOE_OK) return st;
  const moe::Gemm16Args a{nullptr, A, dy, dtype, E, N, K, A_rows, gather_pair, k, seg_offsets, M_total, epilogue, kernel,
                          nullptr, nullptr, out, workspace};
  return hip_status(moe::launch_gemm16_grad_weights(a, stream), "grouped_gemm_grad_weights launch");
}

moe_status moe_unpermute_combine_grad(const uint16_t* dout, const void* y_perm, int32_t y_dtype, const int32_t* pair_pos,
                                      const int32_t* n_valid, const float* topk_w, const int32_t* ids, int32_t T,
                                      int32_t k, int32_t H, int32_t E, int32_t dy_dtype, void* dy, float* dw,
                                      float* dlogits, void* stream) {
  if (!known_dtype(y_dtype)) return fail(MOE_ERR_BAD_FORMAT, "y_dtype %d", y_dtype);
  if (!dtype16(dy_dtype)) return fail(MOE_ERR_BAD_FORMAT, "dy_dtype %d (bf16 or fp16)", dy_dtype);
  if (T < 0 || T >= 1 << 24) return fail(MOE_ERR_BAD_SHAPE, "T=%d (0 or more, fewer than 2^24)", T);
  if (k < 1 || k > 1024 || (int64_t)T * k >= (int64_t)1 << 31) return fail(MOE_ERR_BAD_SHAPE, "k=%d (T=%d)", k, T);
  if (H < 8 || H % 8 != 0) return fail(MOE_ERR_BAD_SHAPE, "H=%d must be a positive multiple of 8", H);
  if ((ids != nullptr) != (dlogits != nullptr)) return fail(MOE_ERR_NULL_ARG, "ids and dlogits go together");
  if (dlogits && !topk_w) return fail(MOE_ERR_NULL_ARG, "dlogits needs topk_w");
  if (dlogits && (E < 1 || E > 1024)) return fail(MOE_ERR_BAD_SHAPE, "E=%d outside 1..1024", E);
  if (T == 0) return ok();
  if (!dout || !y_perm || !pair_pos || !dy || !dw)
    return fail(MOE_ERR_NULL_ARG, "dout, y_perm, pair_pos, dy and dw are required");
  if (dy == dout || dy == y_perm || (const void*)dw == (const void*)topk_w || dw == dlogits)
    return fail(MOE_ERR_BAD_SHAPE, "an output shares a buffer");
  if (!aligned(dout, 16) || !aligned(y_perm, 16) || !aligned(dy, 16))
    return fail(MOE_ERR_MISALIGNED, "dout, y_perm and dy must be 16-byte aligned");
  if (!aligned(pair_pos, 4) || !aligned(n_valid, 4) || !aligned(topk_w, 4) || !aligned(ids, 4) || !aligned(dw, 4) ||
      !aligned(dlogits, 4))
    return fail(MOE_ERR_MISALIGNED, "pair_pos, n_valid, topk_w, ids, dw and dlogits must be 4-byte aligned");
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  const moe::CombineGradArgs a{dout, y_perm, y_dtype, pair_pos, n_valid, topk_w, ids, T, k, H, E, dy_dtype, dy, dw, dlogits};
  return hip_status(moe::launch_combine_grad(a, stream), "unpermute_combine_grad launch");
}

moe_status moe_adapter_add(const void* y, int32_t y_dtype, const void* x, const void* A, const void* B, int32_t dtype,
                           const float* scale, int32_t n, int32_t r, int32_t K, int32_t N, const int32_t* seg_offsets,
                           const int32_t* rows, int32_t T, void* out, void* stream) {
  if (!known_dtype(y_dtype)) return fail(MOE_ERR_BAD_FORMAT, "y_dtype %d", y_dtype);
  if (!dtype16(dtype)) return fail(MOE_ERR_BAD_FORMAT, "dtype %d (bf16 or fp16)", dtype);
  if (n < 1 || n > 1024) return fail(MOE_ERR_BAD_SHAPE, "n=%d adapters outside 1..1024", n);
  if (T < 0 || T >= 1 << 24) return fail(MOE_ERR_BAD_SHAPE, "T=%d (0 or more, fewer than 2^24)", T);
  if (r < 1 || K < 1 || N < 1) return fail(MOE_ERR_BAD_SHAPE, "r=%d K=%d N=%d out of range", r, K, N);
  if (r % 8 != 0 || r > moe::kAdapterMaxRank)
    return fail(MOE_ERR_UNSUPPORTED, "rank %d must be a multiple of 8 up to %d", r, moe::kAdapterMaxRank);
  if (K % 8 != 0 || N % 8 != 0) return fail(MOE_ERR_UNSUPPORTED, "K=%d and N=%d must be multiples of 8", K, N);
  // (the factors' products stay below 2^63: n, r and T are bounded above)
  if ((int64_t)T * K * 2 >= kMaxBytes || (int64_t)n * r * K * 2 >= kMaxBytes || (int64_t)n * r * N * 2 >= kMaxBytes)
    return fail(MOE_ERR_UNSUPPORTED, "x, A or B of 4 GiB or more");
  if (T == 0) return ok();
  if (!y || !x || !A || !B || !seg_offsets || !rows || !out)
    return fail(MOE_ERR_NULL_ARG, "y, x, A, B, seg_offsets, rows and out are required");
  if (out == x || out == A || out == B) return fail(MOE_ERR_BAD_SHAPE, "out shares a buffer with x, A or B");
  if (!aligned(y, 16) || !aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(out, 16))
    return fail(MOE_ERR_MISALIGNED, "y, x, A, B and out must be 16-byte aligned");
  if (!aligned(scale, 4) || !aligned(seg_offsets, 4) || !aligned(rows, 4))
    return fail(MOE_ERR_MISALIGNED, "scale, seg_offsets and rows must be 4-byte aligned");
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  const moe::AdapterArgs a{y, y_dtype, x, A, B, dtype, scale, n, r, K, N, seg_offsets, rows, T, out};
  return hip_status(moe::launch_adapter_add(a, stream), "adapter_add launch");
}

}  // extern "C"
