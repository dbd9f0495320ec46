"""Attention over packed sequences, for training, with its gradients
(include/fp8lin_train.h).

    seqs = Sequences.from_lists([500, 37], device="cuda")     # 537 rows
    out = attention(q, k, v, seqs)                            # autograd
    out, lse = attention_fwd(q, k, v, seqs)                   # the calls below it
    dq, dk, dv = attention_bwd(dout, q, k, v, out, lse, seqs)

q [tokens, q_heads, head_dim], k and v [tokens, kv_heads, head_dim], bf16; rows
any stride apart (slices of a fused product's rows).  Serving reads keys and
values from the FP8 cache instead (attention.py).
"""
import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import Fp8Error, _check, _empty, _need, _need_kind, _need_place, _stream, lib
from .attention import HEAD_DIMS, _head_rows, _packed

MAX_STRIDE = 1 << 24   # elements between two rows


class _SeqsStruct(ctypes.Structure):
    """fp8_seqs_t"""
    _fields_ = [("cu_tokens", ctypes.c_void_p), ("batch", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("pad", ctypes.c_int32)]


class Sequences:
    """Sequences packed one behind the other: cu_tokens [batch + 1] int32 on the
    device, sequence i in rows cu_tokens[i] .. cu_tokens[i + 1] - 1.  max_len
    bounds their lengths, `tokens` is the packed tensors' row count (the host's
    numbers: the device array is not read here).  whole: every row belongs to a
    sequence; otherwise the autograd function clears the rows that may not.
    cu_tokens may be rewritten for other sequences, but not between a pass through
    the autograd function and its backward pass, which reads it again."""

    def __init__(self, cu_tokens, max_len, tokens, whole=False):
        _need_kind(cu_tokens, "cu_tokens", torch.int32)
        if cu_tokens.dim() != 1 or cu_tokens.shape[0] < 1:
            raise ValueError(f"cu_tokens must be [batch + 1], got {tuple(cu_tokens.shape)}")
        _need_place(cu_tokens, "cu_tokens", cu_tokens.device)
        for v, name, most in ((max_len, "max_len", 1 << 30), (tokens, "tokens", (1 << 31) - 1)):
            if not 0 <= int(v) <= most:
                raise ValueError(f"{name} is out of range: {v}")
        self.cu_tokens, self.whole = cu_tokens, bool(whole)
        self.batch, self.tokens, self.max_len = cu_tokens.shape[0] - 1, int(tokens), int(max_len)
        self.device = cu_tokens.device
        self._struct = _SeqsStruct(cu_tokens.data_ptr(), self.batch, self.tokens, self.max_len, 0)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def from_lists(cls, lens, device="cuda"):
        """From the host's list of lengths."""
        lens = [int(n) for n in lens]
        if any(n < 0 for n in lens):
            raise ValueError("a length is negative")
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        if cu[-1] >= 1 << 31:
            raise ValueError(f"{cu[-1]} tokens: fewer than 2^31 are wanted")
        return cls(torch.tensor(cu, dtype=torch.int32).to(device), max([0, *lens]), cu[-1], whole=True)

    def positions(self):
        """Each row's place in its sequence, int32 [tokens], from what cu_tokens
        holds now (rows behind the last sequence count on)."""
        t = torch.arange(self.tokens, dtype=torch.int32, device=self.device)
        if self.batch == 0:
            return t
        i = torch.searchsorted(self.cu_tokens[1:], t, right=True).clamp_(max=self.batch - 1)
        return t - self.cu_tokens[i]


def _rows(t, name, T, heads, d, dev):
    """Row stride in elements of [T, heads, d] bf16 rows with packed heads.  (The
    checks in line: a call for each of a step's tensors is a third of its host time.)"""
    if t.shape == (T, heads, d) and t.dtype is torch.bfloat16 and t.device == dev and t.is_cuda and T > 1:
        row, head, one = t.stride()
        if one == 1 and (head == d or heads == 1) and row <= MAX_STRIDE:
            return row
    row = _head_rows(t, name, T, heads, d, dev, torch.bfloat16)
    if row > MAX_STRIDE:
        raise ValueError(f"{name}: rows {row} elements apart, {MAX_STRIDE} at most")
    return row


def _args(q, k, v, seqs, scale, causal, window):
    """Checks; (q heads, kv heads, head_dim, strides, scale, causal, window)."""
    if not isinstance(seqs, Sequences):
        raise ValueError("seqs must be a Sequences")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a [tokens, heads, head_dim] tensor")
    _, Hq, D = q.shape
    H = k.shape[1]
    if D not in HEAD_DIMS:
        raise ValueError(f"head dimensions are {HEAD_DIMS}, got {D}")
    if H < 1 or Hq < 1 or Hq % H:
        raise ValueError(f"{Hq} query heads over {H} key heads: a positive multiple is wanted")
    if window < 0 or (window and not causal):
        raise ValueError("a window is positive and needs causal")
    T, dev = seqs.tokens, seqs.device
    strides = (_rows(q, "q", T, Hq, D, dev), _rows(k, "k", T, H, D, dev), _rows(v, "v", T, H, D, dev))
    # a window past every position is none: what the library's 32 bits hold
    return Hq, H, D, strides, float(D ** -0.5 if scale is None else scale), int(bool(causal)), min(int(window), 0x7FFFFFFF)


def attention_fwd(q, k, v, seqs, scale=None, causal=True, window=0, out=None, lse=None, stream=None):
    """(out [tokens, q_heads, head_dim] bf16, lse [tokens, q_heads] float32)
    (fp8_attention_fwd).  scale: head_dim ** -0.5 by default.  window > 0: only
    the last `window` positions, the query's own among them (needs causal)."""
    Hq, H, D, (qs, ks, vs), scale, causal, window = _args(q, k, v, seqs, scale, causal, window)
    shape, dev = (seqs.tokens, Hq, D), seqs.device
    if out is not None:
        _need(out, "out", torch.bfloat16, dev, shape=shape)
    else:
        out = _empty(shape, torch.bfloat16, dev, stream)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev, shape=shape[:2])
    else:
        lse = _empty(shape[:2], torch.float32, dev, stream)
    _check("fp8_attention_fwd",
           lib.fp8_attention_fwd(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, seqs._ref, Hq, H, D, scale, causal,
                                 window, out.data_ptr(), lse.data_ptr(), _stream(stream)))
    return out, lse


def attention_bwd_workspace_bytes(seqs, q_heads, kv_heads, head_dim):
    """Workspace bytes of attention_bwd (fp8_attention_bwd_workspace_bytes).
    Grows with the sequences' bounds, not with the device's lengths."""
    n = lib.fp8_attention_bwd_workspace_bytes(seqs._ref, int(q_heads), int(kv_heads), int(head_dim))
    if n < 0:
        raise Fp8Error("fp8_attention_bwd_workspace_bytes", n)
    return n


def attention_bwd(dout, q, k, v, out, lse, seqs, scale=None, causal=True, window=0, dq=None, dk=None, dv=None,
                  workspace=None, stream=None):
    """(dq, dk, dv) bf16 of attention_fwd's out (fp8_attention_bwd), by default
    views of one [tokens, q_heads + 2 kv_heads, head_dim] tensor.  dq, dk, dv:
    optional outputs, rows any stride apart (slices of one tensor's rows).
    workspace: optional device tensor of at least
    attention_bwd_workspace_bytes(...) bytes, otherwise from torch's allocator."""
    Hq, H, D, (qs, ks, vs), scale, causal, window = _args(q, k, v, seqs, scale, causal, window)
    T, dev = seqs.tokens, seqs.device
    if not isinstance(dout, torch.Tensor):
        raise ValueError(f"dout must be a tensor, got {type(dout).__name__}")
    gs = _rows(dout, "dout", T, Hq, D, dev)
    _need(out, "out", torch.bfloat16, dev, shape=(T, Hq, D))
    _need(lse, "lse", torch.float32, dev, shape=(T, Hq))
    row = (Hq + 2 * H) * D
    if dq is None and dk is None and dv is None and row <= MAX_STRIDE:   # one tensor's heads
        dq, dk, dv = _empty((T, Hq + 2 * H, D), torch.bfloat16, dev, stream).split_with_sizes((Hq, H, H), 1)
        strides = (row, row, row)
    else:
        grads = [_empty((T, n, D), torch.bfloat16, dev, stream) if t is None else t
                 for t, n in ((dq, Hq), (dk, H), (dv, H))]
        if not all(isinstance(t, torch.Tensor) for t in grads):
            raise ValueError("dq, dk and dv must be tensors")
        strides = [_rows(t, name, T, n, D, dev) for t, name, n in zip(grads, ("dq", "dk", "dv"), (Hq, H, H))]
        dq, dk, dv = grads
    need = attention_bwd_workspace_bytes(seqs, Hq, H, D)
    if workspace is not None:
        _need_place(workspace, "workspace", dev)
    else:
        workspace = _empty(need, torch.uint8, dev, stream)
    _check("fp8_attention_bwd",
           lib.fp8_attention_bwd(dout.data_ptr(), gs, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, out.data_ptr(),
                                 lse.data_ptr(), seqs._ref, Hq, H, D, scale, causal, window, dq.data_ptr(), strides[0],
                                 dk.data_ptr(), strides[1], dv.data_ptr(), strides[2], workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))
    return dq, dk, dv


class AttentionFunction(torch.autograd.Function):
    """out = attention(q, k, v); gradients for q, k and v."""

    @staticmethod
    def forward(ctx, q, k, v, seqs, scale, causal, window):
        q, k, v = (_packed(t, MAX_STRIDE) for t in (q, k, v))
        out = lse = None
        if not seqs.whole and isinstance(q, torch.Tensor):   # rows of no sequence: zeros
            out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
            lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=q.device)
        out, lse = attention_fwd(q, k, v, seqs, scale, causal, window, out, lse)
        # held with the rest: rewritten before the backward pass, it is refused
        # there (what was made in inference mode has no versions to tell by)
        cu = None if seqs.cu_tokens.is_inference() else seqs.cu_tokens
        ctx.save_for_backward(q, k, v, out, lse, cu)
        ctx.call = (seqs, scale, causal, window)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, _ = ctx.saved_tensors
        new = torch.empty if ctx.call[0].whole else torch.zeros
        grads = [new(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v)]
        return (*attention_bwd(_packed(dout, MAX_STRIDE), q, k, v, out, lse, *ctx.call, *grads), None, None, None, None)


def attention(q, k, v, seqs, scale=None, causal=True, window=0):
    """attention_fwd's out, with gradients.  Tensors of any strides."""
    return AttentionFunction.apply(q, k, v, seqs, scale, causal, window)
