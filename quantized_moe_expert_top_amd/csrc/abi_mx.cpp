// C ABI entry points of the scored routing, the MX rows (quantisation, norm)
// and the MX grouped product: host-side validation, then one stream-ordered
// launch.  Plain C++, the manner of abi.cpp.
#include <math.h>
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
bool known_dtype(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32 || d == MOE_DTYPE_F16; }
bool known_fmt(int f) { return f == MOE_MX_E4M3 || f == MOE_MX_E2M1; }

moe_status check_rows(int64_t rows, int32_t K) {
  if (rows < 0) return fail(MOE_ERR_BAD_SHAPE, "rows=%lld < 0", (long long)rows);
  if (K < 32 || K % 32 != 0) return fail(MOE_ERR_BAD_SHAPE, "row width %d must be a positive multiple of 32", K);
  // (a launch of one thread per 8 or 16 values has fewer than 2^32 threads)
  if (rows >= ((int64_t)1 << 34) / K) return fail(MOE_ERR_BAD_SHAPE, "rows * width too large");
  return MOE_OK;
}

moe_status check_mxdesc(const moe_mxdesc* w, int layout, bool need_buffers) {
  if (!w) return fail(MOE_ERR_NULL_ARG, "weight descriptor is NULL");
  if (w->abi_version != MOE_ABI_VERSION)
    return fail(MOE_ERR_BAD_FORMAT, "descriptor abi_version %d, library %d", w->abi_version, MOE_ABI_VERSION);
  if (w->layout != layout || (layout != MOE_LAYOUT_CANONICAL && layout != MOE_LAYOUT_TILED))
    return fail(MOE_ERR_BAD_FORMAT, "layout %d where %d is required%s", w->layout, layout,
                layout == MOE_LAYOUT_TILED ? " (run moe_mx_repack first)" : "");
  if (w->E < 1 || w->E > 1024 || w->N < 1 || w->K < 1)
    return fail(MOE_ERR_BAD_SHAPE, "E=%d N=%d K=%d out of range", w->E, w->N, w->K);
  if (w->N % 32 != 0 || w->K % 128 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "N=%d must be a multiple of 32 and K=%d of 128", w->N, w->K);
  if ((int64_t)w->N * (w->K + 128) >= ((int64_t)1 << 32)) return fail(MOE_ERR_BAD_SHAPE, "weights too large");
  if (!need_buffers) return MOE_OK;
  if (!w->codes || !w->scales) return fail(MOE_ERR_NULL_ARG, "codes or scales is NULL");
  if (!aligned(w->codes, 16)) return fail(MOE_ERR_MISALIGNED, "codes must be 16-byte aligned");
  if (!aligned(w->scales, 4)) return fail(MOE_ERR_MISALIGNED, "scales must be 4-byte aligned");
  return MOE_OK;
}
moe_status check_route(const float* logits, const float* bias, int32_t T, int32_t E, int32_t k, int32_t score,
                       int32_t n_group, int32_t topk_group, int32_t group_top, float scale, const int32_t* topk_ids,
                       const float* topk_w) {
  if (T < 0) return fail(MOE_ERR_BAD_SHAPE, "T=%d < 0", T);
  if (E < 1 || E > 1024) return fail(MOE_ERR_BAD_SHAPE, "E=%d outside 1..1024", E);
  if (k < 1 || k > E) return fail(MOE_ERR_BAD_SHAPE, "k=%d outside 1..E (E=%d)", k, E);
  if ((int64_t)T * k >= ((int64_t)1 << 31) || T >= 1 << 25) return fail(MOE_ERR_BAD_SHAPE, "T=%d, T*k too large", T);
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return fail(MOE_ERR_BAD_FORMAT, "unknown score %d", score);
  if (n_group < 1 || n_group > 64 || E % n_group != 0)
    return fail(MOE_ERR_BAD_SHAPE, "n_group=%d must be in 1..64 and divide E=%d", n_group, E);
  if (topk_group < 1 || topk_group > n_group)
    return fail(MOE_ERR_BAD_SHAPE, "topk_group=%d outside 1..n_group (%d)", topk_group, n_group);
  if (group_top != 1 && group_top != 2) return fail(MOE_ERR_BAD_SHAPE, "group_top=%d (1 or 2)", group_top);
  if (!isfinite(scale)) return fail(MOE_ERR_BAD_SHAPE, "scale must be finite");
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w) return fail(MOE_ERR_NULL_ARG, "logits, topk_ids and topk_w are required");
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return fail(MOE_ERR_MISALIGNED, "route buffers must be 4-byte aligned");
  return MOE_OK;
}

moe_status check_kernel(int32_t kernel, int32_t K, bool e2m1) {
  if (kernel < MOE_KERNEL_AUTO || kernel > MOE_KERNEL_TILE64_SPLIT_K)
    return fail(MOE_ERR_BAD_FORMAT, "unknown kernel choice %d", kernel);
  if (kernel != MOE_KERNEL_AUTO && kernel != MOE_KERNEL_SMALL && kernel != MOE_KERNEL_TILE64 &&
      kernel != MOE_KERNEL_TILE128 && kernel != MOE_KERNEL_TILE64_SPLIT_K)
    return fail(MOE_ERR_UNSUPPORTED, "kernel choice %d does not run MX weights", kernel);
  if (kernel == MOE_KERNEL_TILE64_SPLIT_K && K <= 256)
    return fail(MOE_ERR_UNSUPPORTED, "K=%d is not split (more than 256)", K);
  if (kernel == MOE_KERNEL_TILE64_SPLIT_K && !e2m1) return fail(MOE_ERR_UNSUPPORTED, "K is split for e2m1 rows only");
  return MOE_OK;
}

moe_status check_code_bytes(int64_t rows, int32_t K, int32_t fmt) {
  const int64_t n = rows * (fmt == MOE_MX_E4M3 ? K : K / 2);
  if (n >= ((int64_t)1 << 32))
    return fail(MOE_ERR_UNSUPPORTED, "activation codes of %lld bytes (4 GiB or more)", (long long)n);
  return MOE_OK;
}
}  // namespace

extern "C" {

moe_status moe_route_scored(const float* logits, const float* bias, int32_t T, int32_t E, int32_t k, int32_t score,
                            int32_t n_group, int32_t topk_group, int32_t group_top, int32_t renormalize, float scale,
                            int32_t* topk_ids, float* topk_w, void* stream) {
  moe_status st = check_route(logits, bias, T, E, k, score, n_group, topk_group, group_top, scale, topk_ids, topk_w);
  if (st != MOE_OK) return st;
  if (T == 0) return ok();
  st = check_device();
  if (st != MOE_OK) return st;
  const moe::ScoredArgs a{logits, bias, T, E, k, score, n_group, topk_group, group_top, renormalize != 0, scale,
                          topk_ids, topk_w};
  return hip_status(moe::launch_route_scored(a, stream), "route_scored launch");
}

moe_status moe_quantize_mx(const void* x, int32_t x_dtype, int64_t rows, int32_t K, int32_t fmt, uint8_t* codes,
                           uint8_t* scales, void* stream) {
  if (!known_dtype(x_dtype)) return fail(MOE_ERR_BAD_FORMAT, "x_dtype %d", x_dtype);
  if (!known_fmt(fmt)) return fail(MOE_ERR_BAD_FORMAT, "unknown MX format %d", fmt);
  moe_status st = check_rows(rows, K);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  if (!x || !codes || !scales) return fail(MOE_ERR_NULL_ARG, "x, codes and scales are required");
  if (!aligned(x, 16) || !aligned(codes, 16)) return fail(MOE_ERR_MISALIGNED, "x and codes must be 16-byte aligned");
  if (x == codes) return fail(MOE_ERR_BAD_SHAPE, "quantisation cannot run in place");
  st = check_device();
  if (st != MOE_OK) return st;
  return hip_status(moe::launch_quantize_mx(x, x_dtype, rows, K, fmt, codes, scales, stream), "quantize_mx launch");
}

moe_status moe_dequantize_mx(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K, int32_t fmt,
                             int32_t out_dtype, void* out, void* stream) {
  if (!known_dtype(out_dtype)) return fail(MOE_ERR_BAD_FORMAT, "out_dtype %d", out_dtype);
  if (!known_fmt(fmt)) return fail(MOE_ERR_BAD_FORMAT, "unknown MX format %d", fmt);
  moe_status st = check_rows(rows, K);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  if (!out || !codes || !scales) return fail(MOE_ERR_NULL_ARG, "codes, scales and out are required");
  if (!aligned(out, 16) || !aligned(codes, 16)) return fail(MOE_ERR_MISALIGNED, "out and codes must be 16-byte aligned");
  if (out == codes) return fail(MOE_ERR_BAD_SHAPE, "dequantisation cannot run in place");
  st = check_device();
  if (st != MOE_OK) return st;
  return hip_status(moe::launch_dequantize_mx(codes, scales, rows, K, fmt, out_dtype, out, stream),
                    "dequantize_mx launch");
}

moe_status moe_rmsnorm_mx(const void* x, const void* residual, const void* weight, int32_t dtype, int64_t rows,
                          int32_t H, float eps, void* sum, void* y, int32_t fmt, uint8_t* codes, uint8_t* scales,
                          void* stream) {
  if (!known_dtype(dtype)) return fail(MOE_ERR_BAD_FORMAT, "dtype %d", dtype);
  if (fmt != 0 && !known_fmt(fmt)) return fail(MOE_ERR_BAD_FORMAT, "unknown MX format %d", fmt);
  moe_status st = check_rows(rows, H);
  if (st != MOE_OK) return st;
  if (H > moe::kNormMaxH) return fail(MOE_ERR_UNSUPPORTED, "H=%d (at most %d)", H, moe::kNormMaxH);
  if (rows >= 1 << 24) return fail(MOE_ERR_BAD_SHAPE, "rows=%lld (fewer than 2^24)", (long long)rows);
  if (!(eps >= 0.0f) || !isfinite(eps)) return fail(MOE_ERR_BAD_SHAPE, "eps must be finite and not negative");
  if (rows == 0) return ok();
  if (!x || !weight) return fail(MOE_ERR_NULL_ARG, "x and weight are required");
  if (sum && !residual) return fail(MOE_ERR_NULL_ARG, "sum needs residual");
  if ((fmt != 0) != (codes != nullptr) || (fmt != 0) != (scales != nullptr))
    return fail(MOE_ERR_NULL_ARG, "codes and scales go with an MX format (fmt %d)", fmt);
  if (!sum && !y && fmt == 0) return fail(MOE_ERR_NULL_ARG, "no output requested");
  if (y && y == sum) return fail(MOE_ERR_BAD_SHAPE, "sum and y share a buffer");
  if (codes && (codes == x || codes == residual || codes == sum || codes == y))
    return fail(MOE_ERR_BAD_SHAPE, "codes share a buffer with rows of values");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) || !aligned(y, 16) ||
      !aligned(codes, 16))
    return fail(MOE_ERR_MISALIGNED, "norm buffers must be 16-byte aligned");
  st = check_device();
  if (st != MOE_OK) return st;
  const moe::NormArgs a{x, residual, weight, dtype, rows, H, eps, sum, y, fmt, codes, scales};
  return hip_status(moe::launch_rmsnorm_mx(a, stream), "rmsnorm_mx launch");
}

size_t moe_mx_field_bytes(const moe_mxdesc* w, int32_t field) {
  if (check_mxdesc(w, w ? w->layout : 0, false) != MOE_OK) return 0;
  const size_t EN = (size_t)w->E * w->N;
  const size_t K = w->layout == MOE_LAYOUT_TILED ? ((size_t)w->K + 255) / 256 * 256 : (size_t)w->K;
  if (field == MOE_FIELD_CODES) return EN * K / 2;
  if (field == MOE_FIELD_SCALES) return EN * K / 32;
  return 0;
}

moe_status moe_mx_repack(const moe_mxdesc* src, const moe_mxdesc* dst, void* stream) {
  moe_status st = check_mxdesc(src, MOE_LAYOUT_CANONICAL, true);
  if (st != MOE_OK) return st;
  st = check_mxdesc(dst, MOE_LAYOUT_TILED, true);
  if (st != MOE_OK) return st;
  if (src->E != dst->E || src->N != dst->N || src->K != dst->K)
    return fail(MOE_ERR_BAD_SHAPE, "source and destination descriptors disagree");
  if ((int64_t)src->E * src->N * ((src->K + 255) / 256 * 256) >= (int64_t)1 << 36)
    return fail(MOE_ERR_BAD_SHAPE, "2^36 weights or more: repack the experts in parts");
  if (src->codes == dst->codes || src->scales == dst->scales) return fail(MOE_ERR_BAD_SHAPE, "repack cannot run in place");
  st = check_device();
  if (st != MOE_OK) return st;
  return hip_status(moe::launch_mx_repack(src->codes, src->scales, src->E, src->N, src->K,
                                          const_cast<uint8_t*>(dst->codes), const_cast<uint8_t*>(dst->scales), stream),
                    "mx_repack launch");
}

moe_status moe_grouped_mxgemm(const moe_mxdesc* w, const uint8_t* a_codes, const uint8_t* a_scales, int32_t a_fmt,
                              int32_t A_rows, const int32_t* gather_pair, int32_t k, const int32_t* seg_offsets,
                              int32_t M_total, int32_t epilogue, int32_t kernel, void* out, uint8_t* out_scales,
                              void* stream) {
  moe_status st = check_mxdesc(w, MOE_LAYOUT_TILED, true);
  if (st != MOE_OK) return st;
  if (!known_fmt(a_fmt)) return fail(MOE_ERR_BAD_FORMAT, "unknown MX format %d", a_fmt);
  if (M_total < 0 || A_rows < 0) return fail(MOE_ERR_BAD_SHAPE, "M_total=%d A_rows=%d", M_total, A_rows);
  if (epilogue < MOE_EPI_NONE || epilogue > MOE_EPI_SWIGLU_E2M1)
    return fail(MOE_ERR_BAD_FORMAT, "unknown epilogue %d", epilogue);
  const bool mx_out = epilogue == MOE_EPI_SWIGLU_E4M3 || epilogue == MOE_EPI_SWIGLU_E2M1;
  if ((epilogue == MOE_EPI_SWIGLU || mx_out) && w->N % 64 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "N=%d must be a multiple of 64 with a SwiGLU epilogue", w->N);
  st = check_kernel(kernel, w->K, a_fmt == MOE_MX_E2M1);
  if (st != MOE_OK) return st;
  if (gather_pair) {
    if (k < 1) return fail(MOE_ERR_BAD_SHAPE, "k=%d with gather_pair", k);
    if ((int64_t)A_rows * k < M_total) return fail(MOE_ERR_BAD_SHAPE, "A_rows*k < M_total");
  } else if (A_rows < M_total) {
    return fail(MOE_ERR_BAD_SHAPE, "A_rows=%d < M_total=%d", A_rows, M_total);
  }
  if (M_total == 0) return ok();
  if (!a_codes || !a_scales || !seg_offsets || !out)
    return fail(MOE_ERR_NULL_ARG, "a_codes, a_scales, seg_offsets and out are required");
  if (out == a_codes || out == a_scales) return fail(MOE_ERR_BAD_SHAPE, "the product cannot run in place");
  if (mx_out != (out_scales != nullptr)) return fail(MOE_ERR_NULL_ARG, "out_scales goes with an MX epilogue (%d)", epilogue);
  if (!aligned(a_codes, 16) || !aligned(out, 16)) return fail(MOE_ERR_MISALIGNED, "a_codes and out must be 16-byte aligned");
  if (!aligned(a_scales, 4) || !aligned(seg_offsets, 4) || !aligned(gather_pair, 4))
    return fail(MOE_ERR_MISALIGNED, "a_scales, seg_offsets and gather_pair must be 4-byte aligned");
  st = check_code_bytes(A_rows, w->K, a_fmt);
  if (st != MOE_OK) return st;
  st = check_device();
  if (st != MOE_OK) return st;
  const moe::MxGemmArgs a{w->codes, w->scales, w->E, w->N, w->K, a_codes, a_scales, a_fmt, A_rows, gather_pair, k,
                          seg_offsets, M_total, epilogue, kernel, out, out_scales};
  return hip_status(moe::launch_mxgemm(a, stream), "grouped_mxgemm launch");
}

size_t moe_mx_layer_workspace_size(int32_t T, int32_t k, int32_t E) {
  // (pairs are rounded up to whole chunks in 32 bits)
  if (T < 0 || k < 1 || E < 1 || E > 1024 || T >= 1 << 25 || (int64_t)T * k > INT32_MAX - moe::kPermuteChunk) return 0;
  return moe::mx_layer_workspace_bytes(T, k, E);
}

moe_status moe_mx_layer(const moe_mxlayer* l, void* stream) {
  if (!l) return fail(MOE_ERR_NULL_ARG, "layer is NULL");
  if (l->abi_version != MOE_ABI_VERSION)
    return fail(MOE_ERR_BAD_FORMAT, "layer abi_version %d, library %d", l->abi_version, MOE_ABI_VERSION);
  moe_status st = check_mxdesc(l->gate_up, MOE_LAYOUT_TILED, true);
  if (st != MOE_OK) return st;
  st = check_mxdesc(l->down, MOE_LAYOUT_TILED, true);
  if (st != MOE_OK) return st;
  const moe_mxdesc &gu = *l->gate_up, &dn = *l->down;
  const int32_t E = gu.E, H = gu.K, I = dn.K, T = l->T, k = l->k;
  if (dn.E != E || dn.N != H || gu.N != 2 * I)
    return fail(MOE_ERR_BAD_SHAPE, "gate_up [%d][%d][%d] and down [%d][%d][%d] do not fit together", E, gu.N, H, dn.E, dn.N, I);
  st = check_route(l->logits, l->bias, T, E, k, l->score, l->n_group, l->topk_group, l->group_top, l->scale,
                   l->topk_ids, l->topk_w);
  if (st != MOE_OK) return st;
  // (the combine's launch, 256 threads a token, has fewer than 2^32 threads)
  if (T >= 1 << 24) return fail(MOE_ERR_BAD_SHAPE, "T=%d (fewer than 2^24)", T);
  if (l->x && !known_dtype(l->x_dtype)) return fail(MOE_ERR_BAD_FORMAT, "x_dtype %d", l->x_dtype);
  if (!known_fmt(l->x_fmt) || !known_fmt(l->h_fmt))
    return fail(MOE_ERR_BAD_FORMAT, "unknown MX format (x %d, h %d)", l->x_fmt, l->h_fmt);
  if (!known_dtype(l->y_dtype)) return fail(MOE_ERR_BAD_FORMAT, "y_dtype %d", l->y_dtype);
  st = check_kernel(l->kernel, H < I ? H : I, l->x_fmt == MOE_MX_E2M1 && l->h_fmt == MOE_MX_E2M1);
  if (st != MOE_OK) return st;
  st = check_code_bytes(T, H, l->x_fmt);
  if (st != MOE_OK) return st;
  st = check_code_bytes((int64_t)T * k, I, l->h_fmt);
  if (st != MOE_OK) return st;
  if (T == 0) return ok();
  if (!l->expert_counts || !l->seg_offsets || !l->sorted_pair || !l->pair_pos || !l->workspace)
    return fail(MOE_ERR_NULL_ARG, "the grouping's buffers are required");
  if (!l->x_codes || !l->x_scales || !l->h_codes || !l->h_scales || !l->y || !l->out)
    return fail(MOE_ERR_NULL_ARG, "x, h, y and out buffers are required");
  if (l->x == l->x_codes || l->x_codes == l->h_codes || l->h_codes == l->y || l->x_codes == l->y || l->y == l->out)
    return fail(MOE_ERR_BAD_SHAPE, "x, x_codes, h_codes, y and out share a buffer");
  const size_t need = moe::mx_layer_workspace_bytes(T, k, E);
  if (l->workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", l->workspace_bytes, need);
  if (!aligned(l->x, 16) || !aligned(l->x_codes, 16) || !aligned(l->h_codes, 16) || !aligned(l->y, 16) ||
      !aligned(l->out, 16) || !aligned(l->workspace, 16))
    return fail(MOE_ERR_MISALIGNED, "x, codes, y, out and workspace must be 16-byte aligned");
  if (!aligned(l->x_scales, 4) || !aligned(l->h_scales, 4) || !aligned(l->expert_counts, 4) ||
      !aligned(l->seg_offsets, 4) || !aligned(l->sorted_pair, 4) || !aligned(l->pair_pos, 4))
    return fail(MOE_ERR_MISALIGNED, "scales and grouping buffers must be 4-byte aligned");
  st = check_device();
  if (st != MOE_OK) return st;

  const moe::ScoredArgs route{l->logits, l->bias, T, E, k, l->score, l->n_group, l->topk_group, l->group_top,
                              l->renormalize != 0, l->scale, l->topk_ids, l->topk_w};
  const moe::FrontRows rows{l->x, l->x_dtype, l->x_fmt, l->x ? (size_t)T * H / 8 : 0, l->x_codes, l->x_scales};
  const moe::FrontGroups groups{l->expert_counts, l->seg_offsets, l->sorted_pair, l->pair_pos,
                                static_cast<uint32_t*>(l->workspace),
                                reinterpret_cast<int*>(static_cast<uint8_t*>(l->workspace) + 256)};
  bool grouped = false;
  int e = moe::launch_mx_front(route, rows, groups, &grouped, stream);
  if (e == 0 && !grouped) {
    const moe::PermuteArgs p{l->topk_ids, nullptr, T * k, k, E, 1, l->expert_counts, l->seg_offsets, l->sorted_pair,
                             l->pair_pos, nullptr, 0, nullptr, l->workspace};
    e = moe::launch_permute(p, stream);
  }
  if (e == 0) {
    const moe::MxGemmArgs g{gu.codes, gu.scales, E, gu.N, H, l->x_codes, l->x_scales, l->x_fmt, T, l->sorted_pair, k,
                            l->seg_offsets, T * k, l->h_fmt == MOE_MX_E4M3 ? MOE_EPI_SWIGLU_E4M3 : MOE_EPI_SWIGLU_E2M1,
                            l->kernel, l->h_codes, l->h_scales};
    e = moe::launch_mxgemm(g, stream);
  }
  if (e == 0) {
    const int epi = l->y_dtype == MOE_DTYPE_F32 ? MOE_EPI_NONE_F32 : l->y_dtype == MOE_DTYPE_F16 ? MOE_EPI_NONE_F16 : MOE_EPI_NONE;
    const moe::MxGemmArgs g{dn.codes, dn.scales, E, H, I, l->h_codes, l->h_scales, l->h_fmt, T * k, nullptr, 1,
                            l->seg_offsets, T * k, epi, l->kernel, l->y, nullptr};
    e = moe::launch_mxgemm(g, stream);
  }
  if (e == 0)
    e = moe::launch_combine(l->y, l->y_dtype, l->pair_pos, l->seg_offsets + E, l->topk_w, T, k, H, l->out, stream);
  return hip_status(e, "mx_layer launch");
}

}  // extern "C"
