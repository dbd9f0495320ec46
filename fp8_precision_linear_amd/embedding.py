"""Embedding with scaling, and its gradient by sorted tokens
(include/fp8lin_train.h).

    x = embedding_fwd(ids, table, scale=d ** 0.5)          # bf16 [..., d]
    dtable = embedding_bwd(dx, ids, vocab, scale=d ** 0.5) # float32 [vocab, d]
    x = Embedding(vocab, d, device="cuda")(ids)            # trains

ids: int32 or int64 of any shape; an id outside 0 .. vocab - 1 (padding: -1) is
no token: a row of zeros, and no gradient.
"""
import torch
from torch.autograd.function import once_differentiable

from . import Fp8Error, _aligned, _check, _dtype_code, _empty, _need, _need_place, _stream, lib


def _ids(ids):
    """(bits, tokens) of an id tensor."""
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be an int32 or int64 tensor")
    return (32 if ids.dtype == torch.int32 else 64), ids.numel()


def embedding_fwd(ids, table, scale=1.0, dtype=torch.bfloat16, out=None, stream=None):
    """scale * table[ids] as [*ids.shape, d] of `dtype`, bfloat16 or float32
    (fp8_embedding_fwd).  table: [vocab, d] bf16 or float32."""
    bits, n = _ids(ids)
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[1] < 1:
        raise ValueError("table must be a [vocab, d] tensor")
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"outputs are bfloat16 or float32, got {dtype}")
    tt, dev = _dtype_code(table), table.device
    _need_place(table, "table", dev)
    _need_place(ids, "ids", dev)
    shape = (*ids.shape, table.shape[1])
    if out is not None:
        _need(out, "out", dtype, dev, shape=shape)
    else:
        out = _empty(shape, dtype, dev, stream)
    _check("fp8_embedding_fwd",
           lib.fp8_embedding_fwd(ids.data_ptr(), bits, n, table.data_ptr(), tt, table.shape[0], table.shape[1], float(scale),
                                 out.data_ptr(), _dtype_code(out), _stream(stream)))
    return out


def embedding_bwd_workspace_bytes(tokens, vocab, d):
    """Workspace bytes of embedding_bwd (fp8_embedding_bwd_workspace_bytes)."""
    v = lib.fp8_embedding_bwd_workspace_bytes(int(tokens), int(vocab), int(d))
    if v < 0:
        raise Fp8Error("fp8_embedding_bwd_workspace_bytes", v)
    return v


def embedding_bwd(dout, ids, vocab, scale=1.0, out=None, accumulate=False, workspace=None, stream=None):
    """The table's gradient, float32 [vocab, d] (fp8_embedding_bwd).  dout:
    [*ids.shape, d] bf16 or float32.  accumulate: added to what `out` holds
    (gradient accumulation); rows without tokens are then left alone.
    workspace: optional device tensor of at least
    embedding_bwd_workspace_bytes(tokens, vocab, d) bytes."""
    bits, n = _ids(ids)
    if not isinstance(dout, torch.Tensor) or dout.dim() < 1 or dout.shape[:-1] != ids.shape or dout.shape[-1] < 1:
        raise ValueError(f"dout must be {tuple(ids.shape)} and d, got "
                         f"{tuple(dout.shape) if isinstance(dout, torch.Tensor) else type(dout).__name__}")
    dt, dev, d = _dtype_code(dout), dout.device, dout.shape[-1]
    if accumulate and out is None:
        raise ValueError("accumulate adds into the caller's gradient: out is required")
    need = embedding_bwd_workspace_bytes(n, vocab, d)
    _need_place(dout, "dout", dev)
    _need_place(ids, "ids", dev)
    if out is not None:
        _need(out, "out", torch.float32, dev, shape=(int(vocab), d))
    else:
        out = _empty((int(vocab), d), torch.float32, dev, stream)
    if workspace is not None:
        _need_place(workspace, "workspace", dev)
    else:
        workspace = _empty(need, torch.uint8, dev, stream)
    _check("fp8_embedding_bwd",
           lib.fp8_embedding_bwd(dout.data_ptr(), dt, ids.data_ptr(), bits, n, int(vocab), d, float(scale),
                                 int(bool(accumulate)), out.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


class EmbeddingFunction(torch.autograd.Function):
    """scale * table[ids]; a gradient for the table."""

    @staticmethod
    def forward(ctx, ids, table, scale, dtype):
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale, ctx.dtype = table.shape[0], scale, table.dtype
        return embedding_fwd(ids, _aligned(table), scale, dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        return None, embedding_bwd(_aligned(dout), ids, ctx.vocab, ctx.scale).to(ctx.dtype), None, None


class Embedding(torch.nn.Module):
    """The table of a model's tokens; forward(ids) is scale * table[ids] in
    `out_dtype`.  The weight is an fp32 master by default."""

    def __init__(self, vocab, d, scale=1.0, out_dtype=torch.bfloat16, device=None, dtype=torch.float32, std=0.02):
        super().__init__()
        self.scale, self.out_dtype = scale, out_dtype
        self.weight = torch.nn.Parameter(torch.randn(vocab, d, device=device, dtype=dtype) * std)

    def forward(self, ids):
        return EmbeddingFunction.apply(ids, self.weight, self.scale, self.out_dtype)
