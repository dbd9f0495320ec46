"""RMS norm with the residual's addition in front of an FP8 product
(include/fp8lin_block.h), and its backward pass.

    h = x + residual (in the residual's type; h = x without one)
    y = h * rstd * w,   rstd = (mean(h^2) + eps)^-1/2 per row

rmsnorm_quantize returns y as FP8 codes with current scaling, rmsnorm_cast at a
given bias (static or delayed scaling), rmsnorm_fwd in bf16.  FP8NormLinear is
the norm and the FP8-AMAX linear layer behind it as one autograd module: the
codes go straight into the product.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (E4M3, E5M2, OP_DGRAD, OP_FWD, OP_WGRAD, Fp8Error, _check, _dtype_code, _empty, _need, _need_kind,
               _need_place, _places, _ptr, _stream, lib, scaled_gemm_accumulate, scaled_gemm_auto)
from .linear import ScalingState

MAX_D, MAX_ODD_D = 32768, 16384   # longest rows: a multiple of 4, any


def _like(t, dtype, stream):
    """A new tensor of t's shape for a call on `stream` (as _empty)."""
    if stream is None:
        return torch.empty_like(t, dtype=dtype)
    return _empty(t.shape, dtype, t.device, stream)


def _opt(t):
    return 0 if t is None else t.data_ptr()


def _here(t, name, dev):
    """_need_place, its checks in line: a call per tensor is a fifth of a small
    norm's host time."""
    if not t.is_contiguous() or t.device != dev:
        _need_place(t, name, dev)


def _fwd_args(x, w, residual, eps, h, rstd, stream):
    """Checks; (rows, arguments up to rstd, h, rstd) of the forward calls.
    x and residual: [..., d]."""
    if not isinstance(x, torch.Tensor) or not isinstance(w, torch.Tensor):
        raise ValueError(f"x and w must be tensors, got {type(x).__name__} and {type(w).__name__}")
    shape, wshape = x.shape, w.shape
    if not shape or len(wshape) != 1 or shape[-1] != wshape[0]:
        raise ValueError(f"x [..., d] and w [d] do not match: {tuple(shape)}, {tuple(wshape)}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    d = shape[-1]
    if not 1 <= d <= (MAX_D if d % 4 == 0 else MAX_ODD_D):
        raise ValueError(f"rows of {d} elements: 1 to {MAX_D}, or {MAX_ODD_D} where not a multiple of 4")
    rows = x.numel() // d
    xt, wt, rt, rptr, hptr = _dtype_code(x), _dtype_code(w), 0, 0, 0
    dev = x.device
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.shape != shape:
            raise ValueError(f"residual must be a tensor of shape {tuple(shape)}, got "
                             f"{tuple(residual.shape) if isinstance(residual, torch.Tensor) else type(residual).__name__}")
        rt = _dtype_code(residual)
    elif h is not None:
        raise ValueError("h is written only where there is a residual")
    if not x.is_cuda:
        _need_place(x, "x", dev)
    _here(x, "x", dev)
    _here(w, "w", dev)
    out = x
    if residual is not None:
        _here(residual, "residual", dev)
        if h is not None:
            _need(h, "h", residual.dtype, dev, shape=shape)
        else:
            h = _like(residual, residual.dtype, stream)
        out, rptr, hptr = h, residual.data_ptr(), h.data_ptr()
    if rstd is not None:
        _need(rstd, "rstd", torch.float32, dev, numel=rows)
    else:
        rstd = _empty(rows, torch.float32, dev, stream)
    return rows, (x.data_ptr(), xt, rptr, rt, w.data_ptr(), wt, rows, d, eps, hptr, rstd.data_ptr()), out, rstd


def rmsnorm_fwd(x, w, residual=None, eps=1e-5, out=None, h=None, rstd=None, amax=None, stream=None):
    """(y, h, rstd): y in bf16 (fp8_rmsnorm_fwd).  h is x itself without a
    residual.  amax: optional float32[1] device tensor that receives max |y|."""
    rows, args, h_out, rstd = _fwd_args(x, w, residual, eps, h, rstd, stream)
    if out is not None:
        _need_kind(out, "out", torch.bfloat16, shape=x.shape)
    if amax is not None:
        _need_kind(amax, "amax", torch.float32, numel=1)
    _places(x.device, (out, "out"), (amax, "amax"))
    out = _like(x, torch.bfloat16, stream) if out is None else out
    _check("fp8_rmsnorm_fwd", lib.fp8_rmsnorm_fwd(*args, _ptr(out), _ptr(amax), _stream(stream)))
    return out, h_out, rstd


def rmsnorm_cast(x, w, bias, fmt, residual=None, eps=1e-5, out=None, h=None, rstd=None, amax=None, stream=None):
    """(codes, h, rstd): y as FP8 codes at `bias` (int32[1] device tensor)
    (fp8_rmsnorm_cast).  amax: optional float32[1] device tensor that receives
    max |y| -- delayed scaling takes the next step's bias from it."""
    rows, args, h_out, rstd = _fwd_args(x, w, residual, eps, h, rstd, stream)
    _need_kind(bias, "bias", torch.int32, numel=1)
    if out is not None:
        _need_kind(out, "out", torch.uint8, shape=x.shape)
    if amax is not None:
        _need_kind(amax, "amax", torch.float32, numel=1)
    _places(x.device, (bias, "bias"), (out, "out"), (amax, "amax"))
    out = _like(x, torch.uint8, stream) if out is None else out
    _check("fp8_rmsnorm_cast", lib.fp8_rmsnorm_cast(*args, _ptr(bias), int(fmt), _ptr(out), _ptr(amax),
                                                    _stream(stream)))
    return out, h_out, rstd


def rmsnorm_quantize(x, w, fmt, residual=None, eps=1e-5, margin=0, out=None, bias=None, amax=None, h=None, rstd=None,
                     row_amax=None, stream=None):
    """(codes, bias, amax, h, rstd): y as FP8 codes with current scaling
    (fp8_rmsnorm_quantize).  row_amax: optional float32[rows] device tensor
    that receives every row's max |y|."""
    rows, args, h_out, rstd = _fwd_args(x, w, residual, eps, h, rstd, stream)
    dev = x.device
    if out is not None:
        _need_kind(out, "out", torch.uint8, shape=x.shape)
        _need_place(out, "out", dev)
    else:
        out = _like(x, torch.uint8, stream)
    if bias is not None:
        _need(bias, "bias", torch.int32, dev, numel=1)
    else:
        bias = _empty(1, torch.int32, dev, stream)
    if amax is not None:
        _need(amax, "amax", torch.float32, dev, numel=1)
    else:
        amax = _empty(1, torch.float32, dev, stream)
    if row_amax is not None:
        _need(row_amax, "row_amax", torch.float32, dev, numel=rows)
    else:   # one row: its amax is the tensor's
        row_amax = amax if rows == 1 else _empty(rows, torch.float32, dev, stream)
    _check("fp8_rmsnorm_quantize",
           lib.fp8_rmsnorm_quantize(*args, int(fmt), int(margin), out.data_ptr(), row_amax.data_ptr(),
                                    amax.data_ptr(), bias.data_ptr(), _stream(stream)))
    return out, bias, amax, h_out, rstd


def rmsnorm_bwd_workspace_bytes(rows, d):
    """Workspace bytes of rmsnorm_bwd (fp8_rmsnorm_bwd_workspace_bytes)."""
    v = lib.fp8_rmsnorm_bwd_workspace_bytes(int(rows), int(d))
    if v < 0:
        raise Fp8Error("fp8_rmsnorm_bwd_workspace_bytes", v)
    return v


def rmsnorm_bwd(dy, h, w, rstd, dh=None, dx=None, dw=None, amax=None, workspace=None, stream=None):
    """(dx, dw) of the norm (fp8_rmsnorm_bwd): dx in h's type (the gradient of x
    and of the residual), dw float32.  dh: the gradient that reaches h past the
    norm, added into dx.  amax: optional float32[1] device tensor that receives
    max |dx|.  workspace: optional device tensor of at least
    rmsnorm_bwd_workspace_bytes(rows, d) bytes."""
    for t, name in ((dy, "dy"), (h, "h"), (w, "w")):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
    if h.dim() < 1 or w.dim() != 1 or h.shape[-1] != w.shape[0] or dy.shape != h.shape:
        raise ValueError(f"dy, h [..., d] and w [d] do not match: {tuple(dy.shape)}, {tuple(h.shape)}, {tuple(w.shape)}")
    d = w.shape[0]
    rows = h.numel() // max(d, 1)
    yt, ht, wt = _dtype_code(dy), _dtype_code(h), _dtype_code(w)
    nbytes = rmsnorm_bwd_workspace_bytes(rows, d)
    _need_kind(rstd, "rstd", torch.float32, numel=rows)
    dev = h.device
    if not h.is_cuda:
        _need_place(h, "h", dev)
    _here(h, "h", dev)
    _here(dy, "dy", dev)
    _here(w, "w", dev)
    _here(rstd, "rstd", dev)
    if dh is not None:
        _need(dh, "dh", h.dtype, dev, shape=h.shape)
    if workspace is not None:
        _need_place(workspace, "workspace", dev)
    if amax is not None:
        _need(amax, "amax", torch.float32, dev, numel=1)
    if dx is not None:
        _need(dx, "dx", h.dtype, dev, shape=h.shape)
    else:
        dx = _like(h, h.dtype, stream)
    if dw is not None:
        _need(dw, "dw", torch.float32, dev, shape=w.shape)
    else:
        dw = _like(w, torch.float32, stream)
    workspace = _empty(nbytes, torch.uint8, dev, stream) if workspace is None else workspace
    _check("fp8_rmsnorm_bwd",
           lib.fp8_rmsnorm_bwd(dy.data_ptr(), yt, h.data_ptr(), ht, w.data_ptr(), wt, rstd.data_ptr(), _opt(dh), rows,
                               d, dx.data_ptr(), dw.data_ptr(), _opt(amax), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream(stream)))
    return dx, dw


class RMSNormFunction(torch.autograd.Function):
    """(y bf16, h) = norm(x + residual) w; gradients for x, residual and w."""

    @staticmethod
    def forward(ctx, x, residual, w, eps):
        y, h, rstd = rmsnorm_fwd(x.contiguous(), w.contiguous(), residual=None if residual is None else
                                 residual.contiguous(), eps=eps)
        ctx.save_for_backward(h, w, rstd)
        ctx.has_residual = residual is not None
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, w, rstd = ctx.saved_tensors
        dx, dw = rmsnorm_bwd(dy.contiguous(), h.contiguous(), w.contiguous(), rstd,
                             dh=None if dh is None else dh.contiguous())
        return dx, (dx if ctx.has_residual else None), dw.to(w.dtype), None


class FP8NormLinearFunction(torch.autograd.Function):
    """(y, h): h = x + residual, y = fp8_linear(norm(h) w_norm, w).  What the
    backward pass reads is held by autograd: h (an output, or the input x) and
    w_norm may not change in between, and everything goes with the graph."""

    @staticmethod
    def forward(ctx, x, residual, w_norm, w, state, eps):
        x = x.contiguous()
        n8, bn, an, h, rstd = rmsnorm_quantize(x, w_norm.contiguous(), E4M3, eps=eps, margin=state.margins["x"],
                                               residual=None if residual is None else residual.contiguous())
        state.amax["x"] = an
        if state.log is not None:
            state.log.record("x", bn)
        n8 = n8.reshape(-1, n8.shape[-1])
        w8, bw = state.quantise("w", w.contiguous())
        y = scaled_gemm_auto(OP_FWD, n8, E4M3, bn, w8, E4M3, bw, math=state.math)
        ctx.save_for_backward(n8, bn, w8, bw, h, rstd, w_norm)
        # the weight itself is only asked for its .grad; its codes are w8
        ctx.state, ctx.weight, ctx.has_residual = state, w, residual is not None
        y = y.reshape(*x.shape[:-1], w.shape[0])
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        n8, bn, w8, bw, h, rstd, w_norm = ctx.saved_tensors
        state, w = ctx.state, ctx.weight
        dy8, bdy = state.quantise("dy", dy.contiguous().reshape(-1, dy.shape[-1]))
        dn = scaled_gemm_auto(OP_DGRAD, dy8, E5M2, bdy, w8, E4M3, bw, math=state.math)
        if state.fuse_wgrad_accumulation and w.grad is not None:
            scaled_gemm_accumulate(OP_WGRAD, dy8, E5M2, bdy, n8, E4M3, bn, w.grad, math=state.math)
            dw = None
        else:
            dw = scaled_gemm_auto(OP_WGRAD, dy8, E5M2, bdy, n8, E4M3, bn, math=state.math)
        dx, dwn = rmsnorm_bwd(dn.reshape(h.shape), h, w_norm.contiguous(), rstd,
                              dh=None if dh is None else dh.contiguous())
        return dx, (dx if ctx.has_residual else None), dwn.to(w_norm.dtype), dw, None, None


class FP8NormLinear(torch.nn.Module):
    """The RMS norm and the FP8-AMAX linear layer behind it.  layer(x) is y;
    layer(x, residual) is (y, x + residual).  Scaling of the normed activations
    is current; the other tensors' as in FP8Linear."""

    def __init__(self, in_features, out_features, eps=1e-5, margins=None, log=None, device=None, dtype=torch.float32,
                 std=0.02, **state):
        super().__init__()
        self.eps = eps
        self.state = ScalingState("current", margins, log=log, **state)
        self.norm_weight = torch.nn.Parameter(torch.ones(in_features, device=device, dtype=dtype))
        self.weight = torch.nn.Parameter(torch.randn(out_features, in_features, device=device, dtype=dtype) * std)

    def forward(self, x, residual=None):
        return FP8NormLinearFunction.apply(x, residual, self.norm_weight, self.weight, self.state, self.eps)
