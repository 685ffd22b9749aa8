"""Binding of the library's scored routing and of its microscaled (MX) path:
rows quantised to 8- or 4-bit MX blocks, the residual RMS norm that writes such
rows, the experts' MX weights, their grouped product and the layer of all.

Argument checks and marshalling only, as in the rest of the binding.  Every
function runs on the device that holds its tensors, on that device's current
stream unless `stream` is given; outputs it allocates belong to that stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from typing import Optional, Union

import torch

from . import (MOE_ABI_VERSION, MOE_DTYPE_BF16, MOE_DTYPE_F16, MOE_DTYPE_F32, MOE_EPI_NONE, MOE_EPI_NONE_F16,
               MOE_EPI_NONE_F32, MOE_EPI_SWIGLU, MOE_EPI_SWIGLU_E2M1, MOE_EPI_SWIGLU_E4M3, MOE_FIELD_CODES,
               MOE_FIELD_SCALES, MOE_KERNEL_AUTO, MOE_LAYOUT_CANONICAL, MOE_LAYOUT_TILED, MOE_MX_E2M1, MOE_MX_E4M3,
               MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, MxDesc, MxLayer, Permutation, _check, _DTYPE_EPI, lib)

_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32, torch.float16: MOE_DTYPE_F16}
_MX_EPI = {MOE_MX_E4M3: MOE_EPI_SWIGLU_E4M3, MOE_MX_E2M1: MOE_EPI_SWIGLU_E2M1}
_EPI_FMT = {v: k for k, v in _MX_EPI.items()}
_EPI_OUT = {MOE_EPI_NONE: torch.bfloat16, MOE_EPI_SWIGLU: torch.bfloat16, MOE_EPI_NONE_F32: torch.float32,
            MOE_EPI_NONE_F16: torch.float16}


# ------------------------------------------------------------------ plumbing
# Small calls are bound by the host: these helpers read raw handles instead of
# building Stream and device objects, and outputs made here skip the checks of
# caller-made ones.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_fns: dict = {}


def _device(*tensors: Optional[torch.Tensor]) -> torch.device:
    """The one GPU that holds all of `tensors` (None entries aside), which must be contiguous."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensor must live on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return dev


def _elsewhere(dev: torch.device, stream) -> bool:
    """Whether a call has to change the current device or stream first."""
    return stream is not None or dev.index != _current_device()


def _guard(dev: torch.device, stream):
    """Makes `dev` current, and `stream` (if given) the stream that work and allocations belong to."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream of {stream.device} for tensors on {dev}")
    return torch.cuda.stream(stream)


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _call(name: str, dev: torch.device, *args) -> None:
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    status = fn(*args, _raw_stream(dev.index))
    if status:
        _check(status, name)


def _want(t: torch.Tensor, what: str, dtype: torch.dtype, shape: tuple) -> torch.Tensor:
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)} (got {t.dtype}, {tuple(t.shape)})")
    return t


# ------------------------------------------------------------ scored routing
@dataclass
class ScoredRouting:
    """How moe_route_scored chooses experts; the defaults are softmax scores, renormalised over the chosen."""
    score: int = MOE_SCORE_SOFTMAX
    bias: Optional[torch.Tensor] = None
    n_group: int = 1
    topk_group: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0


def moe_route_scored(logits: torch.Tensor, k: int, score: int = MOE_SCORE_SOFTMAX, bias: torch.Tensor = None,
                     n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                     scale: float = 1.0, ids: torch.Tensor = None, w: torch.Tensor = None, stream=None):
    """Top-k experts by score (MOE_SCORE_*) plus choice bias, within the best expert groups; returns
    (ids int32 [T][k], w float32 [T][k]).  Slots without an eligible expert hold id -1 and weight 0."""
    if logits.dtype != torch.float32 or logits.dim() != 2:
        raise ValueError("logits must be float32 [T][E]")
    T, E = logits.shape
    if bias is not None:
        _want(bias, "bias", torch.float32, (E,))
    dev = _device(logits, bias, ids, w)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_route_scored(logits, k, score, bias, n_group, topk_group, group_top, renormalize, scale, ids, w)
    ids = logits.new_empty((T, k), dtype=torch.int32) if ids is None else _want(ids, "ids", torch.int32, (T, k))
    w = logits.new_empty((T, k)) if w is None else _want(w, "w", torch.float32, (T, k))
    _call("moe_route_scored", dev, _p(logits), _p(bias), T, E, k, score, n_group, topk_group, group_top,
          1 if renormalize else 0, scale, _p(ids), _p(w))
    return ids, w


# ------------------------------------------------------------------- MX rows
@dataclass
class MxRows:
    """Rows in MX blocks of 32: codes uint8 [...][K] (MOE_MX_E4M3) or [...][K/2] (MOE_MX_E2M1), scales uint8
    [...][K/32]."""
    codes: torch.Tensor
    scales: torch.Tensor
    fmt: int

    def __post_init__(self):
        if self.fmt not in _MX_EPI:
            raise ValueError(f"unknown MX format {self.fmt}")
        if self.codes.dtype != torch.uint8 or self.scales.dtype != torch.uint8:
            raise ValueError("MX codes and scales are uint8")
        if self.codes.dim() < 1 or self.codes.shape != _mx_shape(self.shape, self.fmt):
            raise ValueError(f"codes {tuple(self.codes.shape)} and scales {tuple(self.scales.shape)} do not match")

    @property
    def K(self) -> int:
        return 32 * self.scales.shape[-1]

    @property
    def shape(self) -> tuple:
        return tuple(self.scales.shape[:-1]) + (self.K,)


def _mx_shape(shape: tuple, fmt: int) -> tuple:
    return shape if fmt == MOE_MX_E4M3 else shape[:-1] + (shape[-1] // 2,)


def _new_rows(like: torch.Tensor, shape: tuple, fmt: int) -> MxRows:
    rows = object.__new__(MxRows)
    rows.codes = like.new_empty(_mx_shape(shape, fmt), dtype=torch.uint8)
    rows.scales = like.new_empty(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8)
    rows.fmt = fmt
    return rows


def alloc_mx_rows(shape: tuple, fmt: int, device) -> MxRows:
    """Uninitialised MX rows of `shape` (the last dimension a multiple of 32)."""
    if not shape or shape[-1] < 32 or shape[-1] % 32:
        raise ValueError(f"the last dimension of {tuple(shape)} must be a positive multiple of 32")
    if fmt not in _MX_EPI:
        raise ValueError(f"unknown MX format {fmt}")
    return MxRows(torch.empty(_mx_shape(tuple(shape), fmt), dtype=torch.uint8, device=device),
                  torch.empty(tuple(shape[:-1]) + (shape[-1] // 32,), dtype=torch.uint8, device=device), fmt)


def _rows_out(out: Optional[MxRows], like: torch.Tensor, shape: tuple, fmt: int) -> MxRows:
    if out is None:
        if shape[-1] < 32 or shape[-1] % 32 or fmt not in _MX_EPI:
            return alloc_mx_rows(shape, fmt, like.device)  # says what is wrong
        return _new_rows(like, shape, fmt)
    if out.fmt != fmt or out.shape != shape:
        raise ValueError(f"out holds MX rows {out.shape} of format {out.fmt}, not {shape} of {fmt}")
    return out


def _count(shape: tuple) -> int:
    n = 1
    for v in shape[:-1]:
        n *= v
    return n


def moe_quantize_mx(x: torch.Tensor, fmt: int = MOE_MX_E4M3, out: MxRows = None, stream=None) -> MxRows:
    """bf16, fp16 or fp32 [...][K] -> MX rows."""
    if x.dtype not in _DTYPES or x.dim() < 1:
        raise ValueError(f"x must be bfloat16, float16 or float32 rows (got {x.dtype}, {tuple(x.shape)})")
    dev = _device(x) if out is None else _device(x, out.codes, out.scales)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_quantize_mx(x, fmt, out)
    shape = tuple(x.shape)
    out = _rows_out(out, x, shape, fmt)
    _call("moe_quantize_mx", dev, _p(x), _DTYPES[x.dtype], _count(shape), shape[-1], fmt, _p(out.codes), _p(out.scales))
    return out


def moe_dequantize_mx(rows: MxRows, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor = None,
                      stream=None) -> torch.Tensor:
    """The values that MX rows stand for."""
    shape = rows.shape
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"values in {dtype}: bfloat16, float16 or float32")
    dev = _device(rows.codes, rows.scales, out)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_dequantize_mx(rows, dtype, out)
    out = rows.codes.new_empty(shape, dtype=dtype) if out is None else _want(out, "out", dtype, shape)
    _call("moe_dequantize_mx", dev, _p(rows.codes), _p(rows.scales), _count(shape), shape[-1], rows.fmt, _DTYPES[dtype],
          _p(out))
    return out


@dataclass
class NormOutput:
    sum: Optional[torch.Tensor]  # x + residual (None without residual)
    y: Optional[torch.Tensor]    # the norm in x's type (None unless wanted)
    rows: Optional[MxRows]       # the norm as MX rows (None without a format)


def moe_rmsnorm_mx(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor = None,
                   fmt: Optional[int] = MOE_MX_E4M3, want_y: bool = False, sum: torch.Tensor = None,
                   y: torch.Tensor = None, out: MxRows = None, stream=None) -> NormOutput:
    """Root-mean-square norm of x + residual times weight, in one pass: the sum (with a residual; `sum` may be
    x's or residual's own buffer), the norm in x's type (want_y, or a `y` to write) and the norm as MX rows
    of `fmt` (None: no MX rows)."""
    if x.dtype not in _DTYPES or x.dim() < 1:
        raise ValueError(f"x must be bfloat16, float16 or float32 rows (got {x.dtype}, {tuple(x.shape)})")
    shape = tuple(x.shape)
    _want(weight, "weight", x.dtype, shape[-1:])
    if residual is not None:
        _want(residual, "residual", x.dtype, shape)
    elif sum is not None:
        raise ValueError("sum without residual")
    if out is not None and fmt is None:
        raise ValueError("out without an MX format")
    dev = _device(x, weight, residual, sum, y)
    if out is not None:
        _device(x, out.codes, out.scales)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_rmsnorm_mx(x, weight, eps, residual, fmt, want_y, sum, y, out)
    if residual is not None:
        sum = torch.empty_like(x) if sum is None else _want(sum, "sum", x.dtype, shape)
    if y is not None:
        _want(y, "y", x.dtype, shape)
    elif want_y:
        y = torch.empty_like(x)
    rows = None if fmt is None else _rows_out(out, x, shape, fmt)
    _call("moe_rmsnorm_mx", dev, _p(x), _p(residual), _p(weight), _DTYPES[x.dtype], _count(shape), shape[-1], eps,
          _p(sum), _p(y), fmt or 0, rows and rows.codes.data_ptr(), rows and rows.scales.data_ptr())
    return NormOutput(sum, y, rows)


# ---------------------------------------------------------------- MX experts
@dataclass
class MxExperts:
    """MX expert weights in one layout; keeps its tensors alive with the descriptor."""
    desc: MxDesc
    tensors: dict = field(default_factory=dict)

    @property
    def N(self) -> int:
        return self.desc.N

    @property
    def K(self) -> int:
        return self.desc.K


def _mx_desc(layout: int, E: int, N: int, K: int, codes=None, scales=None) -> MxExperts:
    d = MxDesc()
    d.abi_version, d.layout, d.E, d.N, d.K = MOE_ABI_VERSION, layout, E, N, K
    d.codes, d.scales = _p(codes), _p(scales)
    return MxExperts(d, {k: v for k, v in (("codes", codes), ("scales", scales)) if v is not None})


def mx_experts(codes: Union[torch.Tensor, MxRows], scales: torch.Tensor = None) -> MxExperts:
    """Canonical MX expert weights: codes u8 [E][N][K/2] and scales u8 [E][N][K/32], or the MX rows
    [E][N][K] that moe_quantize_mx gives (MOE_MX_E2M1)."""
    rows = codes if isinstance(codes, MxRows) else MxRows(codes, scales, MOE_MX_E2M1)
    if rows.fmt != MOE_MX_E2M1 or len(rows.shape) != 3:
        raise ValueError(f"expert weights are 4-bit MX rows [E][N][K] (got {rows.shape}, format {rows.fmt})")
    _device(rows.codes, rows.scales)
    return _mx_desc(MOE_LAYOUT_CANONICAL, *rows.shape, rows.codes, rows.scales)


def moe_mx_field_bytes(w: MxExperts, fld: int) -> int:
    return lib().moe_mx_field_bytes(ctypes.byref(w.desc), fld)


def moe_mx_repack(src: MxExperts, stream=None) -> MxExperts:
    """Canonical -> tiled copy of MX expert weights (offline; allocates the tiled buffers)."""
    s = src.desc
    dev = _device(*src.tensors.values())
    with _guard(dev, stream):
        probe = _mx_desc(MOE_LAYOUT_TILED, s.E, s.N, s.K)
        # (an invalid descriptor has 0 bytes; the call below says why)
        t = [torch.empty(max(moe_mx_field_bytes(probe, f), 16), dtype=torch.uint8, device=dev)
             for f in (MOE_FIELD_CODES, MOE_FIELD_SCALES)]
        dst = _mx_desc(MOE_LAYOUT_TILED, s.E, s.N, s.K, *t)
        _call("moe_mx_repack", dev, ctypes.byref(s), ctypes.byref(dst.desc))
    return dst


def moe_grouped_mxgemm(w: MxExperts, A: MxRows, seg_offsets: torch.Tensor, M_total: int,
                       epilogue: int = MOE_EPI_NONE, gather_pair: torch.Tensor = None, k: int = 1,
                       out: Union[torch.Tensor, MxRows] = None, stream=None, kernel: int = MOE_KERNEL_AUTO):
    """Grouped product of MX rows A [A_rows][K] with tiled MX experts; `out` (and the result) is a tensor, or MX
    rows for MOE_EPI_SWIGLU_E4M3 / MOE_EPI_SWIGLU_E2M1."""
    d = w.desc
    if len(A.shape) != 2 or A.K != d.K:
        raise ValueError(f"A must be MX rows [A_rows][{d.K}] (got {A.shape})")
    if seg_offsets.dtype != torch.int32 or seg_offsets.dim() != 1 or seg_offsets.numel() < d.E + 1:
        raise ValueError(f"seg_offsets must be int32 with at least {d.E + 1} entries (got {seg_offsets.dtype}, "
                         f"{tuple(seg_offsets.shape)})")
    if gather_pair is not None and (gather_pair.dtype != torch.int32 or gather_pair.numel() < M_total):
        raise ValueError(f"gather_pair must be int32 with at least M_total = {M_total} entries")
    fmt = _EPI_FMT.get(epilogue)
    if fmt is None and epilogue not in _EPI_OUT:
        raise ValueError(f"unknown epilogue {epilogue}")
    n_out = d.N if epilogue in _DTYPE_EPI.values() else d.N // 2
    if (isinstance(out, MxRows) if fmt is None else out is not None and not isinstance(out, MxRows)):
        raise ValueError("out must be MX rows exactly for the MX epilogues")
    bufs = (out.codes, out.scales) if isinstance(out, MxRows) else (out,)
    dev = _device(A.codes, A.scales, seg_offsets, gather_pair, *w.tensors.values(), *bufs)
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_grouped_mxgemm(w, A, seg_offsets, M_total, epilogue, gather_pair, k, out, None, kernel)
    if fmt is not None:
        out = _rows_out(out, A.codes, (M_total, n_out), fmt)
        o, osc = _p(out.codes), _p(out.scales)
    else:
        dt = _EPI_OUT[epilogue]
        out = A.codes.new_empty((M_total, n_out), dtype=dt) if out is None else _want(out, "out", dt, (M_total, n_out))
        o, osc = _p(out), None
    _call("moe_grouped_mxgemm", dev, ctypes.byref(d), _p(A.codes), _p(A.scales), A.fmt, A.shape[0], _p(gather_pair), k,
          _p(seg_offsets), M_total, epilogue, kernel, o, osc)
    return out


# --------------------------------------------------------------------- layer
@dataclass
class MxLayerBuffers:
    """Preallocated intermediates of one MX layer forward."""
    sizes: tuple  # (T, E, k, H, I)
    ids: torch.Tensor
    w: torch.Tensor
    perm: Permutation
    x: MxRows
    h: MxRows
    y_perm: torch.Tensor
    out: torch.Tensor


def alloc_mx_layer(T: int, E: int, k: int, H: int, I: int, device, act: int = MOE_MX_E4M3, h_fmt: int = MOE_MX_E4M3,
                   y_dtype: torch.dtype = torch.float16) -> MxLayerBuffers:
    """act: MX format of the layer's input rows; h_fmt: of the SwiGLU activations; y_dtype: the experts' outputs
    before the combine: float16 (default, as in alloc_layer: half the bytes of float32, 11 significant bits, and
    infinities past 65504), float32 (as the product sums them) or bfloat16 (8 bits, float32's range)."""
    if y_dtype not in _DTYPE_EPI:
        raise ValueError(f"expert outputs in {y_dtype}: float16, float32 or bfloat16")
    i32 = dict(dtype=torch.int32, device=device)
    perm = Permutation(counts=torch.empty(E, **i32), seg_offsets=torch.empty(E + 1, **i32),
                       sorted_pair=torch.empty(T * k, **i32), pair_pos=torch.empty(T * k, **i32),
                       workspace=torch.zeros(max(lib().moe_mx_layer_workspace_size(T, k, E), 16), dtype=torch.uint8,
                                             device=device))
    return MxLayerBuffers(sizes=(T, E, k, H, I), ids=torch.empty((T, k), **i32),
                          w=torch.empty((T, k), dtype=torch.float32, device=device), perm=perm,
                          x=alloc_mx_rows((T, H), act, device), h=alloc_mx_rows((T * k, I), h_fmt, device),
                          y_perm=torch.empty((T * k, H), dtype=y_dtype, device=device),
                          out=torch.empty((T, H), dtype=torch.bfloat16, device=device))


def moe_mx_layer_forward(x: Union[torch.Tensor, MxRows], logits: torch.Tensor, k: int, gate_up: MxExperts,
                         down: MxExperts, routing: ScoredRouting = None, buf: MxLayerBuffers = None, stream=None,
                         kernel: int = MOE_KERNEL_AUTO) -> MxLayerBuffers:
    """Scored routing -> grouping -> gate_up with SwiGLU, its activations quantised to MX rows -> down -> combine,
    one stream.  x: bf16, fp16 or fp32 [T][H], quantised to buf.x's format, or MX rows (moe_rmsnorm_mx).  Buffers made
    here (buf None) have alloc_mx_layer's defaults: expert outputs past 65504 need buffers with another y_dtype."""
    T, H = x.shape
    E = logits.shape[1]
    I = gate_up.N // 2
    if gate_up.desc.E != E or down.desc.E != E or gate_up.K != H or down.N != H or down.K != I or logits.shape[0] != T:
        raise ValueError(f"x [{T}][{H}], logits {tuple(logits.shape)}, gate_up [{gate_up.desc.E}][{gate_up.N}]"
                         f"[{gate_up.K}] and down [{down.desc.E}][{down.N}][{down.K}] do not fit together")
    rows = x if isinstance(x, MxRows) else None
    dev = (rows.codes if rows else x).device
    r = routing or ScoredRouting()
    if dev.type != "cuda":
        raise ValueError("tensor must live on the GPU")
    if _elsewhere(dev, stream):
        with _guard(dev, stream):
            return moe_mx_layer_forward(x, logits, k, gate_up, down, routing, buf, None, kernel)
    if buf is None:
        buf = alloc_mx_layer(T, E, k, H, I, dev, act=rows.fmt if rows else MOE_MX_E4M3)
    elif buf.sizes != (T, E, k, H, I):
        raise ValueError(f"buffers of (T, E, k, H, I) = {buf.sizes} for a layer of {(T, E, k, H, I)}")
    if rows is None:
        if x.dtype not in _DTYPES:
            raise ValueError(f"x must be bfloat16, float16, float32 or MX rows (got {x.dtype})")
        q = buf.x
    else:
        q = rows
    if logits.dtype != torch.float32:
        raise ValueError(f"logits must be float32 (got {logits.dtype})")
    if r.bias is not None:
        _want(r.bias, "bias", torch.float32, (E,))
    p = buf.perm
    P = T * k
    if (q.shape != (T, H) or buf.h.shape != (P, I) or buf.y_perm.shape != (P, H) or buf.y_perm.dtype not in _DTYPES
            or buf.ids.nbytes != 4 * P or buf.w.nbytes != 4 * P or buf.out.nbytes != 2 * T * H
            or p.counts.nbytes < 4 * E or p.seg_offsets.nbytes < 4 * E + 4 or p.sorted_pair.nbytes < 4 * P
            or p.pair_pos.nbytes < 4 * P):
        raise ValueError("a layer buffer was replaced by one of another size")
    if _device(logits, r.bias, q.codes, q.scales, buf.ids, buf.w, p.counts, p.seg_offsets, p.sorted_pair, p.pair_pos,
               p.workspace, buf.h.codes, buf.h.scales, buf.y_perm, buf.out, *gate_up.tensors.values(),
               *down.tensors.values()) != dev or (rows is None and not x.is_contiguous()):
        raise ValueError(f"x (contiguous, on {dev}) and the layer's tensors must be on one GPU")
    args = MxLayer(MOE_ABI_VERSION, T, k, MOE_DTYPE_BF16 if rows else _DTYPES[x.dtype], q.fmt, buf.h.fmt,
                   _DTYPES[buf.y_perm.dtype], kernel, r.score, r.n_group, r.topk_group, r.group_top,
                   1 if r.renormalize else 0, r.scale, ctypes.pointer(gate_up.desc), ctypes.pointer(down.desc),
                   None if rows else x.data_ptr(), logits.data_ptr(), _p(r.bias), buf.ids.data_ptr(), buf.w.data_ptr(),
                   p.counts.data_ptr(), p.seg_offsets.data_ptr(), p.sorted_pair.data_ptr(), p.pair_pos.data_ptr(),
                   p.workspace.data_ptr(), p.workspace.numel(), q.codes.data_ptr(), q.scales.data_ptr(),
                   buf.h.codes.data_ptr(), buf.h.scales.data_ptr(), buf.y_perm.data_ptr(), buf.out.data_ptr())
    _call("moe_mx_layer", dev, ctypes.byref(args))
    return buf
