"""Binding of the experts in 16 bits (grouped product, its gradients, the
combine's gradient, a layer of them forward and backward) and of the low-rank
adapters beside a shared projection.

Argument checks and marshalling only, as in the rest of the binding.  Every
function runs on the device that holds its tensors, on that device's current
stream unless `stream` is given; outputs it allocates belong to that stream.
The gradients are plain calls, no autograd graph: a program calls them where
its backward pass needs them, and may capture them like the forward ones.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import (MOE_EPI_NONE, MOE_EPI_NONE_F16, MOE_EPI_NONE_F32, MOE_EPI_SWIGLU, MOE_EPI_SWIGLU_GRAD,
               MOE_KERNEL_AUTO, MOE_KERNEL_SMALL, Permutation, _DTYPE_EPI, lib, moe_route_permute, moe_unpermute_combine)
from .mx import _call, _device, _DTYPES, _elsewhere, _guard, _p, _want

_PLAIN = {MOE_EPI_NONE: torch.bfloat16, MOE_EPI_NONE_F16: torch.float16, MOE_EPI_NONE_F32: torch.float32}
_TYPES16 = (torch.bfloat16, torch.float16)


def _weights(w: torch.Tensor, what: str = "w") -> tuple:
    if w.dtype not in _TYPES16 or w.dim() != 3:
        raise ValueError(f"{what} must be bfloat16 or float16 [E][N][K] (got {w.dtype}, {tuple(w.shape)})")
    return w.shape


def _rows(t: torch.Tensor, what: str, dtype: torch.dtype, width: int, rows: int) -> torch.Tensor:
    if t.dtype != dtype or t.dim() != 2 or t.shape[1] != width or t.shape[0] < rows:
        raise ValueError(f"{what} must be {dtype} [{rows} or more][{width}] (got {t.dtype}, {tuple(t.shape)})")
    return t


def _segments(seg_offsets: torch.Tensor, E: int) -> None:
    if seg_offsets.dtype != torch.int32 or seg_offsets.dim() != 1 or seg_offsets.numel() < E + 1:
        raise ValueError(f"seg_offsets must be int32 with at least {E + 1} entries (got {seg_offsets.dtype}, "
                         f"{tuple(seg_offsets.shape)})")


def _pairs(gather_pair: Optional[torch.Tensor], M_total: int) -> None:
    if gather_pair is not None and (gather_pair.dtype != torch.int32 or gather_pair.numel() < M_total):
        raise ValueError(f"gather_pair must be int32 with at least M_total = {M_total} entries")


# ------------------------------------------------------------------ products
def moe_grouped_gemm(w: torch.Tensor, A: torch.Tensor, seg_offsets: torch.Tensor, M_total: int,
                     epilogue: int = MOE_EPI_NONE, gather_pair: torch.Tensor = None, k: int = 1,
                     out: torch.Tensor = None, pre: torch.Tensor = None, stream=None,
                     kernel: int = MOE_KERNEL_AUTO) -> torch.Tensor:
    """Grouped product of rows A [A_rows][K] with 16-bit experts w [E][N][K].  Plain epilogues give [M_total][N] in their
    type; MOE_EPI_SWIGLU [M_total][N/2] in w's, and writes what enters it to `pre` [M_total][N] if given.  Rows of no
    segment are not written."""
    E, N, K = _weights(w)
    _segments(seg_offsets, E)
    _pairs(gather_pair, M_total)
    _rows(A, "A", w.dtype, K, 0 if gather_pair is not None else M_total)
    if epilogue == MOE_EPI_SWIGLU:
        dt, n_out = w.dtype, N // 2
        if pre is not None:
            _want(pre, "pre", w.dtype, (M_total, N))
    elif epilogue in _PLAIN:
        dt, n_out = _PLAIN[epilogue], N
        if pre is not None:
            raise ValueError("pre goes with MOE_EPI_SWIGLU")
    else:
        raise ValueError(f"epilogue {epilogue} of a 16-bit product")
    dev = _device(w, A, seg_offsets, gather_pair, out, pre)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_grouped_gemm(w, A, seg_offsets, M_total, epilogue, gather_pair, k, out, pre, None, kernel)
    out = w.new_empty((M_total, n_out), dtype=dt) if out is None else _want(out, "out", dt, (M_total, n_out))
    _call("moe_grouped_gemm", dev, w.data_ptr(), _DTYPES[w.dtype], E, N, K, A.data_ptr(), A.shape[0], _p(gather_pair), k,
          seg_offsets.data_ptr(), M_total, epilogue, kernel, _p(pre), out.data_ptr())
    return out


def moe_grouped_gemm_grad_rows(w: torch.Tensor, dy: torch.Tensor, seg_offsets: torch.Tensor, M_total: int,
                               epilogue: int = MOE_EPI_NONE, pre: torch.Tensor = None, out: torch.Tensor = None,
                               stream=None, kernel: int = MOE_KERNEL_AUTO) -> torch.Tensor:
    """Gradient of moe_grouped_gemm by its rows, grouped: dy [M_total][N] -> [M_total][K] in the epilogue's type; with
    MOE_EPI_SWIGLU_GRAD further through the SwiGLU that `pre` [M_total][2K] entered -> [M_total][2K] in w's type."""
    E, N, K = _weights(w)
    _segments(seg_offsets, E)
    _rows(dy, "dy", w.dtype, N, M_total)
    if epilogue == MOE_EPI_SWIGLU_GRAD:
        dt, n_out = w.dtype, 2 * K
        if pre is None:
            raise ValueError("MOE_EPI_SWIGLU_GRAD needs pre")
        _want(pre, "pre", w.dtype, (M_total, n_out))
    elif epilogue in _PLAIN:
        dt, n_out = _PLAIN[epilogue], K
        if pre is not None:
            raise ValueError("pre goes with MOE_EPI_SWIGLU_GRAD")
    else:
        raise ValueError(f"epilogue {epilogue} of a gradient by the rows")
    dev = _device(w, dy, seg_offsets, pre, out)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_grouped_gemm_grad_rows(w, dy, seg_offsets, M_total, epilogue, pre, out, None, kernel)
    out = w.new_empty((M_total, n_out), dtype=dt) if out is None else _want(out, "out", dt, (M_total, n_out))
    _call("moe_grouped_gemm_grad_rows", dev, w.data_ptr(), _DTYPES[w.dtype], E, N, K, dy.data_ptr(),
          seg_offsets.data_ptr(), M_total, epilogue, kernel, _p(pre), out.data_ptr())
    return out


def moe_grouped_gemm_grad_weights_workspace_size(E: int, N: int, K: int, M_total: int,
                                                 kernel: int = MOE_KERNEL_AUTO) -> int:
    return lib().moe_grouped_gemm_grad_weights_workspace_size(E, N, K, M_total, kernel)


def moe_grouped_gemm_grad_weights(dy: torch.Tensor, A: torch.Tensor, seg_offsets: torch.Tensor, E: int, M_total: int,
                                  epilogue: int = MOE_EPI_NONE_F32, gather_pair: torch.Tensor = None, k: int = 1,
                                  out: torch.Tensor = None, workspace: torch.Tensor = None, stream=None,
                                  kernel: int = MOE_KERNEL_AUTO) -> torch.Tensor:
    """Gradient of moe_grouped_gemm by its weights: dy [M_total][N] and the product's rows A -> [E][N][K] in the
    epilogue's type (zeros for an expert without rows)."""
    if dy.dtype not in _TYPES16 or dy.dim() != 2 or A.dim() != 2:
        raise ValueError(f"dy and A must be bfloat16 or float16 rows (got {dy.dtype}, {tuple(dy.shape)}, {tuple(A.shape)})")
    N, K = dy.shape[1], A.shape[1]
    _segments(seg_offsets, E)
    _pairs(gather_pair, M_total)
    _rows(dy, "dy", dy.dtype, N, M_total)
    _rows(A, "A", dy.dtype, K, 0 if gather_pair is not None else M_total)
    dt = _PLAIN.get(epilogue)
    if dt is None:
        raise ValueError(f"epilogue {epilogue} of a gradient by the weights")
    dev = _device(dy, A, seg_offsets, gather_pair, out, workspace)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_grouped_gemm_grad_weights(dy, A, seg_offsets, E, M_total, epilogue, gather_pair, k, out, workspace,
                                                 None, kernel)
    out = dy.new_empty((E, N, K), dtype=dt) if out is None else _want(out, "out", dt, (E, N, K))
    if workspace is None:
        need = lib().moe_grouped_gemm_grad_weights_workspace_size(E, N, K, M_total, kernel)
        if need:
            workspace = dy.new_empty(need, dtype=torch.uint8)
    _call("moe_grouped_gemm_grad_weights", dev, dy.data_ptr(), A.data_ptr(), _DTYPES[dy.dtype], E, N, K, A.shape[0],
          _p(gather_pair), k, seg_offsets.data_ptr(), M_total, epilogue, kernel, out.data_ptr(), _p(workspace),
          workspace.nbytes if workspace is not None else 0)
    return out


# ------------------------------------------------------- the combine's gradient
@dataclass
class CombineGrad:
    dy: torch.Tensor                  # by the experts' outputs, grouped [T*k][H]
    dw: torch.Tensor                  # by the gate weights, float32 [T][k]
    dlogits: Optional[torch.Tensor]   # by the router's logits, float32 [T][E] (None without ids)


def moe_unpermute_combine_grad(dout: torch.Tensor, y_perm: torch.Tensor, pair_pos: torch.Tensor,
                               topk_w: Optional[torch.Tensor], T: int, k: int, dtype: torch.dtype = torch.bfloat16,
                               dy: torch.Tensor = None, dw: torch.Tensor = None, dlogits: torch.Tensor = None,
                               ids: torch.Tensor = None, E: int = 0, n_valid: torch.Tensor = None,
                               stream=None) -> CombineGrad:
    """Gradient of moe_unpermute_combine from its output's, dout bf16 [T][H].  dtype: of dy (the grouped products'
    type).  With ids (and topk_w) the gradient by the E router logits too, for gates that are the softmax over the
    selected ones (moe_route_topk).  n_valid: as for the combine; rows of dy past it are left as they are."""
    if dout.dtype != torch.bfloat16 or dout.dim() != 2 or dout.shape[0] != T:
        raise ValueError(f"dout must be bfloat16 [{T}][H] (got {dout.dtype}, {tuple(dout.shape)})")
    H, P = dout.shape[1], T * k
    if y_perm.dtype not in _DTYPES or y_perm.shape != (P, H):
        raise ValueError(f"y_perm must be bfloat16, float16 or float32 [{P}][{H}] (got {y_perm.dtype}, "
                         f"{tuple(y_perm.shape)})")
    if pair_pos.dtype != torch.int32 or pair_pos.numel() != P:
        raise ValueError(f"pair_pos must be int32 with {P} entries")
    if dtype not in _TYPES16:
        raise ValueError(f"dy in {dtype}: bfloat16 or float16")
    if topk_w is not None:
        _want(topk_w, "topk_w", torch.float32, (T, k))
    if ids is not None:
        _want(ids, "ids", torch.int32, (T, k))
        if topk_w is None:
            raise ValueError("the gradient by the logits needs topk_w")
    elif dlogits is not None:
        raise ValueError("dlogits needs ids")
    if n_valid is not None and (n_valid.dtype != torch.int32 or n_valid.numel() < 1):
        raise ValueError("n_valid must be an int32 device tensor")
    dev = _device(dout, y_perm, pair_pos, topk_w, ids, n_valid, dy, dw, dlogits)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_unpermute_combine_grad(dout, y_perm, pair_pos, topk_w, T, k, dtype, dy, dw, dlogits, ids, E, n_valid)
    dy = dout.new_empty((P, H), dtype=dtype) if dy is None else _want(dy, "dy", dtype, (P, H))
    dw = dout.new_empty((T, k), dtype=torch.float32) if dw is None else _want(dw, "dw", torch.float32, (T, k))
    if ids is not None:
        dlogits = (dout.new_empty((T, E), dtype=torch.float32) if dlogits is None
                   else _want(dlogits, "dlogits", torch.float32, (T, E)))
    _call("moe_unpermute_combine_grad", dev, dout.data_ptr(), y_perm.data_ptr(), _DTYPES[y_perm.dtype],
          pair_pos.data_ptr(), _p(n_valid), _p(topk_w), _p(ids), T, k, H, E, _DTYPES[dtype], dy.data_ptr(),
          dw.data_ptr(), _p(dlogits))
    return CombineGrad(dy, dw, dlogits)


# --------------------------------------------------------------------- layer
@dataclass
class ExpertLayerBuffers:
    """Preallocated intermediates of one layer of 16-bit experts; a backward pass reads them."""
    sizes: tuple  # (T, E, k, H, I)
    ids: torch.Tensor
    w: torch.Tensor
    perm: Permutation
    pre: Optional[torch.Tensor]  # what enters the SwiGLU (None: not kept, no backward pass)
    h: torch.Tensor
    y_perm: torch.Tensor
    out: torch.Tensor


@dataclass
class ExpertLayerGrads:
    dx: torch.Tensor       # bf16 [T][H]
    dlogits: torch.Tensor  # float32 [T][E]
    dgate_up: torch.Tensor
    ddown: torch.Tensor


def alloc_expert_layer(T: int, E: int, k: int, H: int, I: int, device, dtype: torch.dtype = torch.bfloat16,
                       keep: bool = False, y_dtype: torch.dtype = torch.float16) -> ExpertLayerBuffers:
    """dtype: the weights'; keep: also what the backward pass needs; y_dtype: the experts' outputs before the combine,
    as in alloc_layer."""
    if y_dtype not in _DTYPE_EPI:
        raise ValueError(f"expert outputs in {y_dtype}: float16, float32 or bfloat16")
    if dtype not in _TYPES16:
        raise ValueError(f"weights in {dtype}: bfloat16 or float16")
    i32 = dict(dtype=torch.int32, device=device)
    perm = Permutation(counts=torch.empty(E, **i32), seg_offsets=torch.empty(E + 1, **i32),
                       sorted_pair=torch.empty(T * k, **i32), pair_pos=torch.empty(T * k, **i32),
                       workspace=torch.zeros(max(lib().moe_permute_workspace_size(T, k, E, 1), 16), dtype=torch.uint8,
                                             device=device))
    new = lambda width, dt: torch.empty((T * k, width), dtype=dt, device=device)  # noqa: E731
    return ExpertLayerBuffers(sizes=(T, E, k, H, I), ids=torch.empty((T, k), **i32),
                              w=torch.empty((T, k), dtype=torch.float32, device=device), perm=perm,
                              pre=new(2 * I, dtype) if keep else None, h=new(I, dtype), y_perm=new(H, y_dtype),
                              out=torch.empty((T, H), dtype=torch.bfloat16, device=device))


def _layer_sizes(x: torch.Tensor, E: int, k: int, gate_up: torch.Tensor, down: torch.Tensor) -> tuple:
    _weights(gate_up, "gate_up")
    _weights(down, "down")
    H, I = gate_up.shape[2], down.shape[2]
    if (x.dim() != 2 or x.shape[1] != H or gate_up.shape != (E, 2 * I, H) or down.shape != (E, H, I)
            or x.dtype != gate_up.dtype or down.dtype != gate_up.dtype):
        raise ValueError(f"x {tuple(x.shape)} {x.dtype}, {E} experts, gate_up {tuple(gate_up.shape)} {gate_up.dtype} and "
                         f"down {tuple(down.shape)} {down.dtype} do not fit together")
    return x.shape[0], E, k, H, I


def moe_expert_layer_forward(x: torch.Tensor, logits: torch.Tensor, k: int, gate_up: torch.Tensor, down: torch.Tensor,
                             buf: ExpertLayerBuffers = None, keep: bool = False, stream=None,
                             kernel: int = MOE_KERNEL_AUTO) -> ExpertLayerBuffers:
    """Route -> group -> gate_up (+SwiGLU) -> down -> combine with experts in 16 bits (gate_up [E][2I][H]: gate rows, then
    up rows; down [E][H][I]), one stream.  The output is bf16 for either type of weights.  keep (or buffers made with it): what moe_expert_layer_backward needs stays."""
    if logits.dim() != 2:
        raise ValueError("logits must be float32 [T][E]")
    sizes = _layer_sizes(x, logits.shape[1], k, gate_up, down)
    T, E, _, H, I = sizes
    if logits.dtype != torch.float32 or logits.shape[0] != T:
        raise ValueError(f"logits must be float32 [{T}][E] (got {logits.dtype}, {tuple(logits.shape)})")
    dev = _device(x, logits, gate_up, down)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_expert_layer_forward(x, logits, k, gate_up, down, buf, keep, None, kernel)
    if buf is None:
        buf = alloc_expert_layer(T, E, k, H, I, dev, x.dtype, keep)
    elif buf.sizes != sizes or buf.h.dtype != x.dtype or (keep and buf.pre is None):
        raise ValueError(f"buffers of (T, E, k, H, I) = {buf.sizes}, {buf.h.dtype} for a layer of {sizes}, {x.dtype}"
                         + (" whose backward pass follows" if keep else ""))
    p = buf.perm
    moe_route_permute(logits, k, ids=buf.ids, w=buf.w, out=p)
    moe_grouped_gemm(gate_up, x, p.seg_offsets, T * k, MOE_EPI_SWIGLU, gather_pair=p.sorted_pair, k=k, out=buf.h,
                     pre=buf.pre, kernel=kernel)
    moe_grouped_gemm(down, buf.h, p.seg_offsets, T * k, _DTYPE_EPI[buf.y_perm.dtype], out=buf.y_perm, kernel=kernel)
    moe_unpermute_combine(buf.y_perm, p.pair_pos, buf.w, T, k, out=buf.out, n_valid=p.seg_offsets[-1:])
    return buf


def moe_expert_layer_backward(dout: torch.Tensor, x: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor,
                              buf: ExpertLayerBuffers, grad_dtype: torch.dtype = torch.float32, stream=None,
                              kernel: int = MOE_KERNEL_AUTO) -> ExpertLayerGrads:
    """Gradients of moe_expert_layer_forward from its output's (dout bf16 [T][H]), with the buffers that it kept: by x
    (the k experts' fp32 shares added in fp32, then bf16), the logits, and both weights (grad_dtype).  The routing's choice is
    taken as given, as everywhere; down's gradient sees the experts' outputs as the forward pass rounded them."""
    T, E, k, H, I = buf.sizes
    if _layer_sizes(x, E, k, gate_up, down) != buf.sizes:
        raise ValueError(f"buffers of (T, E, k, H, I) = {buf.sizes} for x {tuple(x.shape)}, gate_up {tuple(gate_up.shape)}")
    if buf.pre is None:
        raise ValueError("the forward pass kept nothing for this one (keep=True)")
    epi = _DTYPE_EPI.get(grad_dtype)
    if epi is None:
        raise ValueError(f"weights' gradients in {grad_dtype}: float32, bfloat16 or float16")
    dev = _device(dout, x, gate_up, down, buf.pre)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_expert_layer_backward(dout, x, gate_up, down, buf, grad_dtype, None, kernel)
    p, P = buf.perm, T * k
    weights_kernel = MOE_KERNEL_AUTO if kernel == MOE_KERNEL_SMALL else kernel  # (a choice of the gradient by the rows alone)
    c = moe_unpermute_combine_grad(dout, buf.y_perm, p.pair_pos, buf.w, T, k, dtype=x.dtype, ids=buf.ids, E=E,
                                   n_valid=p.seg_offsets[-1:])
    ddown = moe_grouped_gemm_grad_weights(c.dy, buf.h, p.seg_offsets, E, P, epi, kernel=weights_kernel)
    dpre = moe_grouped_gemm_grad_rows(down, c.dy, p.seg_offsets, P, MOE_EPI_SWIGLU_GRAD, pre=buf.pre, kernel=kernel)
    dgate_up = moe_grouped_gemm_grad_weights(dpre, x, p.seg_offsets, E, P, epi, gather_pair=p.sorted_pair, k=k,
                                             kernel=weights_kernel)
    # the shares stay in fp32 up to their sum: 16 bits would round each, and fp16 ends at 65504
    dx = moe_grouped_gemm_grad_rows(gate_up, dpre, p.seg_offsets, P, MOE_EPI_NONE_F32, kernel=kernel)
    dx = moe_unpermute_combine(dx, p.pair_pos, None, T, k, n_valid=p.seg_offsets[-1:])
    return ExpertLayerGrads(dx, c.dlogits, dgate_up, ddown)


# ------------------------------------------------------------------ adapters
def moe_adapter_add(y: torch.Tensor, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, seg_offsets: torch.Tensor,
                    rows: torch.Tensor, scale: torch.Tensor = None, out: torch.Tensor = None,
                    stream=None) -> torch.Tensor:
    """y [T][N] + scale[a] * B_a (A_a x_t) for every token t of adapter a; A [n][r][K], B [n][N][r] and x [T][K] in one
    16-bit type, y in any, scale float32 [n] (None: 1).  seg_offsets, rows: the tokens grouped by adapter,
    p = moe_permute(ids [T][1], n): p.seg_offsets, p.sorted_pair (an id outside [0, n): no adapter, y as it is).
    out: y's own buffer for an addition in place."""
    n, r, K = _weights(A, "A")
    if y.dtype not in _DTYPES or y.dim() != 2:
        raise ValueError(f"y must be bfloat16, float16 or float32 [T][N] (got {y.dtype}, {tuple(y.shape)})")
    T, N = y.shape
    _want(B, "B", A.dtype, (n, N, r))
    _want(x, "x", A.dtype, (T, K))
    _segments(seg_offsets, n)
    if rows.dtype != torch.int32 or rows.numel() < T:
        raise ValueError(f"rows must be int32 with at least {T} entries")
    if scale is not None:
        _want(scale, "scale", torch.float32, (n,))
    dev = _device(y, x, A, B, seg_offsets, rows, scale, out)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_adapter_add(y, x, A, B, seg_offsets, rows, scale, out)
    out = torch.empty_like(y) if out is None else _want(out, "out", y.dtype, (T, N))
    _call("moe_adapter_add", dev, y.data_ptr(), _DTYPES[y.dtype], x.data_ptr(), A.data_ptr(), B.data_ptr(),
          _DTYPES[A.dtype], _p(scale), n, r, K, N, seg_offsets.data_ptr(), rows.data_ptr(), T, out.data_ptr())
    return out
