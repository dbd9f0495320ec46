"""Norms of queries and keys for each head with the rotary positions, in one
pass over the fused product's rows, and their gradients
(include/fp8lin_train.h).

    q, k, v = qk_norm_rope_fwd(qkv, q_heads, kv_heads, wq, wk, rope=(cos, sin), positions=pos)
    dqkv, dwq, dwk = qk_norm_rope_bwd(dq, dk, dv, qkv, wq, wk, rope=(cos, sin), positions=pos)
    q, k, v = qk_norm_rope(qkv, q_heads, kv_heads, wq, wk, ...)     # autograd

qkv [tokens, q_heads + 2 kv_heads, head_dim] bf16 or float32: queries, keys,
values.  Outputs are bf16: queries and keys normed and rotated, values rounded.
"""
import torch
from torch.autograd.function import once_differentiable

from . import Fp8Error, _aligned, _check, _dtype_code, _empty, _need, _need_place, _stream, lib
from .attention import HEAD_DIMS, _head_rows, _packed


def _opt(t):
    return 0 if t is None else t.data_ptr()


def _here(t, name, dtype, shape, dev):
    """_need, its checks in line."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_cuda or \
            t.device != dev or not t.is_contiguous():
        _need(t, name, dtype, dev, shape=shape)


def _args(qkv, q_heads, kv_heads, wq, wk, eps, rope, positions, rope_pairs):
    """Checks; (tokens, head_dim, arguments from x to rope_pairs)."""
    if not isinstance(qkv, torch.Tensor) or qkv.dim() != 3:
        raise ValueError("qkv must be a [tokens, q_heads + 2 kv_heads, head_dim] tensor")
    T, n, D = qkv.shape
    Hq, H = int(q_heads), int(kv_heads)
    if Hq < 1 or H < 1 or n != Hq + 2 * H:
        raise ValueError(f"{n} heads in a row: {Hq} + 2 * {H} are wanted")
    if D not in HEAD_DIMS:
        raise ValueError(f"head dimensions are {HEAD_DIMS}, got {D}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    dt, dev, wt = _dtype_code(qkv), qkv.device, 0
    stride = _head_rows(qkv, "qkv", T, n, D, dev)
    if (wq is None) != (wk is None):
        raise ValueError("norm weights for both queries and keys, or for neither")
    if wq is not None:
        wt = _dtype_code(wq)
        _here(wq, "wq", wq.dtype, (D,), dev)
        _here(wk, "wk", wq.dtype, (D,), dev)
    if positions is not None:
        _here(positions, "positions", torch.int32, (T,), dev)
    cos = sin = None
    rows = 0
    if rope is not None:
        cos, sin = rope
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError(f"cos must be a [positions, {D // 2}] tensor")
        rows = cos.shape[0]
        _here(cos, "cos", torch.float32, (rows, D // 2), dev)
        _here(sin, "sin", torch.float32, (rows, D // 2), dev)
        if rows < (1 if positions is not None else T):
            raise ValueError(f"cos holds {rows} positions for {T} tokens")
    return T, D, (qkv.data_ptr(), dt, stride, T, Hq, H, D, _opt(wq), _opt(wk), wt, float(eps), _opt(positions), _opt(cos),
                  _opt(sin), rows, int(bool(rope_pairs)))


def qk_norm_rope_fwd(qkv, q_heads, kv_heads, wq=None, wk=None, eps=1e-5, rope=None, positions=None, rope_pairs=False,
                     out=None, stream=None):
    """(q, k, v) bf16, views of one [tokens, q_heads + 2 kv_heads, head_dim] tensor
    (`out` if given) (fp8_qk_norm_rope_fwd).  wq, wk: [head_dim] bf16 or float32,
    or None: no norm.  rope: (cos, sin) float32 [positions, head_dim / 2], or None;
    rope_pairs as in kv_append.  positions: int32 [tokens], or None: row t is at
    position t."""
    T, D, args = _args(qkv, q_heads, kv_heads, wq, wk, eps, rope, positions, rope_pairs)
    if out is not None:
        _need(out, "out", torch.bfloat16, qkv.device, shape=qkv.shape)
    else:
        out = _empty(qkv.shape, torch.bfloat16, qkv.device, stream)
    _check("fp8_qk_norm_rope_fwd", lib.fp8_qk_norm_rope_fwd(*args, out.data_ptr(), _stream(stream)))
    return out.split_with_sizes((q_heads, kv_heads, kv_heads), 1)   # one call: half the time of three slices


def qk_norm_rope_bwd_workspace_bytes(tokens, q_heads, kv_heads, head_dim):
    """Workspace bytes of qk_norm_rope_bwd with weights
    (fp8_qk_norm_rope_bwd_workspace_bytes)."""
    v = lib.fp8_qk_norm_rope_bwd_workspace_bytes(int(tokens), int(q_heads), int(kv_heads), int(head_dim))
    if v < 0:
        raise Fp8Error("fp8_qk_norm_rope_bwd_workspace_bytes", v)
    return v


def qk_norm_rope_bwd(dq, dk, dv, qkv, wq=None, wk=None, eps=1e-5, rope=None, positions=None, rope_pairs=False, out=None,
                     dwq=None, dwk=None, workspace=None, stream=None):
    """(dqkv, dwq, dwk) (fp8_qk_norm_rope_bwd): dqkv of qkv's type and shape, the
    weights' gradients float32 [head_dim] (None without weights).  dq [tokens,
    q_heads, head_dim], dk, dv [tokens, kv_heads, head_dim] bf16, rows any stride
    apart; the other arguments as the forward had them.  workspace: optional
    device tensor of at least qk_norm_rope_bwd_workspace_bytes(...) bytes."""
    for t, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a [tokens, heads, head_dim] tensor")
    Hq, H = dq.shape[1], dk.shape[1]
    T, D, args = _args(qkv, Hq, H, wq, wk, eps, rope, positions, rope_pairs)
    dev = qkv.device
    strides = [_head_rows(t, name, T, n, D, dev, torch.bfloat16)
               for t, name, n in ((dq, "dq", Hq), (dk, "dk", H), (dv, "dv", H))]
    if out is not None:
        _need(out, "out", qkv.dtype, dev, shape=qkv.shape)
    else:
        out = _empty(qkv.shape, qkv.dtype, dev, stream)
    nbytes = 0
    if wq is None:
        if dwq is not None or dwk is not None:
            raise ValueError("dwq and dwk without weights")
        workspace = None
    else:
        for t, name in ((dwq, "dwq"), (dwk, "dwk")):
            if t is not None:
                _need(t, name, torch.float32, dev, shape=(D,))
        if dwq is None and dwk is None:
            dwq, dwk = _empty((2, D), torch.float32, dev, stream).unbind()
        else:
            dwq = _empty((D,), torch.float32, dev, stream) if dwq is None else dwq
            dwk = _empty((D,), torch.float32, dev, stream) if dwk is None else dwk
        if workspace is not None:
            _need_place(workspace, "workspace", dev)
        else:
            workspace = _empty(qk_norm_rope_bwd_workspace_bytes(T, Hq, H, D), torch.uint8, dev, stream)
        nbytes = workspace.numel() * workspace.element_size()
    _check("fp8_qk_norm_rope_bwd",
           lib.fp8_qk_norm_rope_bwd(dq.data_ptr(), strides[0], dk.data_ptr(), strides[1], dv.data_ptr(), strides[2], *args,
                                    out.data_ptr(), _opt(dwq), _opt(dwk), _opt(workspace), nbytes, _stream(stream)))
    return out, dwq, dwk


class QKNormRopeFunction(torch.autograd.Function):
    """(q, k, v) of qk_norm_rope_fwd; gradients for qkv and the weights."""

    @staticmethod
    def forward(ctx, qkv, wq, wk, q_heads, kv_heads, eps, rope, positions, rope_pairs):
        cos, sin = (None, None) if rope is None else rope
        qkv, wq, wk = _packed(qkv), *(None if w is None else _aligned(w) for w in (wq, wk))
        ctx.save_for_backward(qkv, wq, wk, cos, sin, positions)
        ctx.heads, ctx.eps, ctx.rope_pairs = (q_heads, kv_heads), eps, rope_pairs
        # three tensors to autograd, though they share their rows: outputs that are
        # views of one may not be changed in place
        return tuple(t.data for t in qk_norm_rope_fwd(qkv, q_heads, kv_heads, wq, wk, eps, rope, positions, rope_pairs))

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk, dv):
        qkv, wq, wk, cos, sin, positions = ctx.saved_tensors
        dx, dwq, dwk = qk_norm_rope_bwd(_packed(dq), _packed(dk), _packed(dv), qkv, wq, wk, ctx.eps,
                                        None if cos is None else (cos, sin), positions, ctx.rope_pairs)
        if wq is not None:
            dwq, dwk = dwq.to(wq.dtype), dwk.to(wk.dtype)
        return dx, dwq, dwk, None, None, None, None, None, None


def qk_norm_rope(qkv, q_heads, kv_heads, wq=None, wk=None, eps=1e-5, rope=None, positions=None, rope_pairs=False):
    """qk_norm_rope_fwd with gradients.  qkv of any strides."""
    return QKNormRopeFunction.apply(qkv, wq, wk, q_heads, kv_heads, eps, rope, positions, rope_pairs)
