"""A paged cache of keys and values in FP8, and attention over it
(include/fp8lin_block.h).

KVCache holds the codes and, for each block of tokens and head, one
power-of-two bias for the keys and one for the values.  KVBatch says which
sequences a call is about: how many tokens each has in the cache, how many of
them are new, and which blocks they lie in.

    cache = KVCache(num_blocks, heads, head_dim, device="cuda")
    batch = KVBatch.from_lists(new=[1, 1], lens=[500, 37], tables=[[4, 0, ...], [7]], device="cuda")
    q = kv_append(cache, batch, k, v, q=q, rope=(cos, sin))   # writes k, v; rotated queries in bf16
    out = kv_attention(cache, batch, q)                       # [tokens, q_heads, head_dim] bf16
"""
import ctypes

import torch

from . import (E4M3, E5M2, Fp8Error, _aligned, _check, _dtype_code, _empty, _need_kind, _need_place, _places, _stream, lib)

BLOCK_SIZES = (16, 32, 64, 128)
HEAD_DIMS = (64, 128, 256)
MAX_BIAS = 126   # FP8_KV_MAX_BIAS


class _CacheStruct(ctypes.Structure):
    """fp8_kv_cache_t"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_bias", ctypes.c_void_p),
                ("v_bias", ctypes.c_void_p), ("num_blocks", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("pad", ctypes.c_int32)]


class _BatchStruct(ctypes.Structure):
    """fp8_kv_batch_t"""
    _fields_ = [("cu_tokens", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("table_width", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("max_len", ctypes.c_int32), ("pad", ctypes.c_int32)]


class KVCache:
    """k [num_blocks, heads, block_size, head_dim] and v [num_blocks, heads,
    head_dim, block_size] uint8 codes; k_bias, v_bias int32 [num_blocks, heads]."""

    def __init__(self, num_blocks, heads, head_dim, block_size=64, fmt=E4M3, device="cuda"):
        z = lambda *shape, dtype=torch.uint8: torch.zeros(*shape, dtype=dtype, device=device)  # noqa: E731
        self._set(z(num_blocks, heads, block_size, head_dim), z(num_blocks, heads, head_dim, block_size),
                  z(num_blocks, heads, dtype=torch.int32), z(num_blocks, heads, dtype=torch.int32), fmt)

    @classmethod
    def from_tensors(cls, k, v, k_bias, v_bias, fmt=E4M3):
        """A cache over the caller's tensors."""
        self = cls.__new__(cls)
        self._set(k, v, k_bias, v_bias, fmt)
        return self

    def _set(self, k, v, k_bias, v_bias, fmt):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a 4-D uint8 tensor of FP8 codes")
        nb, heads, bs, d = k.shape
        if bs not in BLOCK_SIZES or d not in HEAD_DIMS:
            raise ValueError(f"block sizes are {BLOCK_SIZES} and head dimensions {HEAD_DIMS}, got {bs} and {d}")
        if fmt not in (E4M3, E5M2):
            raise ValueError(f"fmt is E4M3 or E5M2, got {fmt!r}")
        if nb < 1 or heads < 1:
            raise ValueError("a cache has at least one block and one head")
        _need_kind(k, "k", torch.uint8)
        _need_kind(v, "v", torch.uint8, shape=(nb, heads, d, bs))
        for t, name in ((k_bias, "k_bias"), (v_bias, "v_bias")):
            _need_kind(t, name, torch.int32, shape=(nb, heads))
        _places(k.device, (k, "k"), (v, "v"), (k_bias, "k_bias"), (v_bias, "v_bias"))
        self.k, self.v, self.k_bias, self.v_bias, self.fmt = k, v, k_bias, v_bias, fmt
        self.num_blocks, self.heads, self.block_size, self.head_dim = nb, heads, bs, d
        self.device = k.device
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_bias.data_ptr(), v_bias.data_ptr(), nb, heads, bs, d,
                                    int(fmt), 0)
        self._ref = ctypes.byref(self._struct)


class KVBatch:
    """A ragged batch: cu_tokens [batch + 1], lens [batch], block_table [batch,
    width], all int32 on the device; max_new and max_len bound the new tokens
    and the lengths, `tokens` is the packed tensors' row count (the host's
    numbers: the device arrays are not read here)."""

    def __init__(self, cu_tokens, lens, block_table, max_new, max_len, tokens):
        _need_kind(lens, "lens", torch.int32)
        if lens.dim() != 1:
            raise ValueError("lens must be 1-D")
        n = lens.shape[0]
        _need_kind(cu_tokens, "cu_tokens", torch.int32, shape=(n + 1,))
        _need_kind(block_table, "block_table", torch.int32)
        if block_table.dim() != 2 or block_table.shape[0] != n:
            raise ValueError(f"block_table must be [{n}, width], got {tuple(block_table.shape)}")
        _places(lens.device, (cu_tokens, "cu_tokens"), (lens, "lens"), (block_table, "block_table"))
        for v, name in ((max_new, "max_new"), (max_len, "max_len"), (tokens, "tokens")):
            if not 0 <= int(v) < 1 << 31:
                raise ValueError(f"{name} is out of range: {v}")
        self.cu_tokens, self.lens, self.block_table = cu_tokens, lens, block_table
        self.batch, self.tokens, self.max_new, self.max_len = n, int(tokens), int(max_new), int(max_len)
        self.device = lens.device
        self._struct = _BatchStruct(cu_tokens.data_ptr(), lens.data_ptr(), block_table.data_ptr(), n,
                                    block_table.shape[1], self.tokens, self.max_new, self.max_len, 0)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def from_lists(cls, new, lens, tables, device="cuda"):
        """From host lists: new tokens and length of each sequence, and its
        block numbers (padded here with -1, no block)."""
        if not len(new) == len(lens) == len(tables):
            raise ValueError("new, lens and tables have one entry for each sequence")
        if any(not 0 <= n <= m for n, m in zip(new, lens)):
            raise ValueError("a sequence's new tokens are among its length")
        width = max([len(t) for t in tables] + [1])
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).to(device)  # noqa: E731
        table = i32([list(t) + [-1] * (width - len(t)) for t in tables]).reshape(len(new), width)
        return cls(i32(cu), i32(list(lens)).reshape(-1), table, max([0, *new]), max([0, *lens]), cu[-1])

    def positions(self):
        """The position of each row of the packed tensors, int32 [tokens], from
        what the device arrays hold now (rows behind the last sequence count on)."""
        t = torch.arange(self.tokens, dtype=torch.int32, device=self.device)
        if self.batch == 0:
            return t
        i = torch.searchsorted(self.cu_tokens[1:], t, right=True).clamp_(max=self.batch - 1)
        return t + (self.lens - self.cu_tokens[1:])[i]


def _opt(t):
    return 0 if t is None else t.data_ptr()


def _pair(cache, batch):
    if not isinstance(cache, KVCache) or not isinstance(batch, KVBatch):
        raise ValueError("cache is a KVCache and batch a KVBatch")
    if cache.device != batch.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    if batch.max_len > batch.block_table.shape[1] * cache.block_size:
        raise ValueError(f"lengths up to {batch.max_len} do not fit {batch.block_table.shape[1]} blocks of "
                         f"{cache.block_size}")


def _head_rows(t, name, tokens, heads, d, device, dtype=None):
    """Row stride in elements of [tokens, heads, d] rows with packed heads."""
    if not isinstance(t, torch.Tensor) or t.shape != (tokens, heads, d):
        raise ValueError(f"{name} must be a [{tokens}, {heads}, {d}] tensor, got "
                         f"{tuple(t.shape) if isinstance(t, torch.Tensor) else type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor on {device}, got {t.device}")
    row, head, one = t.stride()
    if tokens and (one != 1 or (heads > 1 and head != d)):
        raise ValueError(f"{name}: the heads of a row must be contiguous, got strides {t.stride()}")
    return row if tokens > 1 else heads * d


def _packed(t, most=(1 << 63) - 1):
    """t, or a copy whose rows the kernels can read: heads side by side, rows that
    do not overlap and are at most `most` elements apart, on 16-byte boundaries."""
    if isinstance(t, torch.Tensor) and t.dim() == 3:
        row, head, one = t.stride()
        n, d = t.shape[1:]
        if one != 1 or head != d or not n * d <= row <= most or row * t.element_size() % 16 or t.data_ptr() % 16:
            return _aligned(t)
    return t


def kv_append(cache, batch, k, v, q=None, rope=None, rope_pairs=False, q_out=None, stream=None):
    """Writes the batch's new keys and values into the cache (fp8_kv_append).
    k, v: [tokens, heads, head_dim] bf16 or float32, rows any stride apart (a
    slice of the fused product's rows).  rope: (cos, sin), float32 [positions,
    head_dim / 2], rotates keys and queries, dimension j with j + head_dim / 2,
    or 2j with 2j + 1 (rope_pairs).  q: optional [tokens, q_heads, head_dim] of
    k's type; returns them, rotated, in bf16 (q_out if given), else None."""
    _pair(cache, batch)
    T, H, D, dev = batch.tokens, cache.heads, cache.head_dim, cache.device
    dt = _dtype_code(k)
    ks = _head_rows(k, "k", T, H, D, dev)
    vs = _head_rows(v, "v", T, H, D, dev, k.dtype)
    qs = heads = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a [tokens, q_heads, head_dim] tensor")
        heads = q.shape[1]
        qs = _head_rows(q, "q", T, heads, D, dev, k.dtype)
        if q_out is not None:
            _need_kind(q_out, "q_out", torch.bfloat16, shape=(T, heads, D))
            _need_place(q_out, "q_out", dev)
        else:
            q_out = _empty((T, heads, D), torch.bfloat16, dev, stream)
    elif q_out is not None:
        raise ValueError("q_out without q")
    cos = sin = None
    if rope is not None:
        cos, sin = rope
        for t, name in ((cos, "cos"), (sin, "sin")):
            _need_kind(t, name, torch.float32)
            if t.dim() != 2 or t.shape[1] != D // 2 or t.shape != cos.shape:
                raise ValueError(f"{name} must be [positions, {D // 2}], got {tuple(t.shape)}")
            if t.shape[0] < batch.max_len:
                raise ValueError(f"{name} holds {t.shape[0]} positions, the batch up to {batch.max_len}")
            _need_place(t, name, dev)
    _check("fp8_kv_append",
           lib.fp8_kv_append(cache._ref, batch._ref, k.data_ptr(), ks, v.data_ptr(), vs, dt, _opt(q), qs, heads, _opt(q_out),
                             _opt(cos), _opt(sin), 0 if cos is None else cos.shape[0], int(bool(rope_pairs)),
                             _stream(stream)))
    return q_out


def kv_read(cache, batch, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """(k, v) [tokens, heads, head_dim] of the batch's last tokens of every
    sequence, as bf16 or float32 (fp8_kv_read); new = lens reads all of them."""
    _pair(cache, batch)
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"outputs are bfloat16 or float32, got {dtype}")
    shape, dev = (batch.tokens, cache.heads, cache.head_dim), cache.device
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is not None:
            _need_kind(t, name, dtype, shape=shape)
            _need_place(t, name, dev)
    k_out = _empty(shape, dtype, dev, stream) if k_out is None else k_out
    v_out = _empty(shape, dtype, dev, stream) if v_out is None else v_out
    _check("fp8_kv_read", lib.fp8_kv_read(cache._ref, batch._ref, _dtype_code(k_out), k_out.data_ptr(), v_out.data_ptr(),
                                          _stream(stream)))
    return k_out, v_out


def attention_workspace_bytes(cache, batch, q_heads):
    """Workspace bytes of kv_attention (fp8_kv_attention_workspace_bytes; 0:
    none).  Grows with the batch's bounds, not with the device's lengths."""
    _pair(cache, batch)
    n = lib.fp8_kv_attention_workspace_bytes(cache._ref, batch._ref, int(q_heads))
    if n < 0:
        raise Fp8Error("fp8_kv_attention_workspace_bytes", n)
    return n


def attention_workspace(cache, batch, q_heads, stream=None):
    """A workspace of that size, or None."""
    n = attention_workspace_bytes(cache, batch, q_heads)
    return _empty(n, torch.uint8, cache.device, stream) if n else None


def kv_attention(cache, batch, q, scale=None, causal=True, window=0, out=None, lse=None, return_lse=False,
                 workspace=None, stream=None):
    """Attention of the new tokens' queries [tokens, q_heads, head_dim] bf16 over
    the cache (fp8_kv_attention): out [tokens, q_heads, head_dim] bf16, or (out,
    lse [tokens, q_heads] float32) with return_lse.  scale: head_dim ** -0.5 by
    default.  window > 0: only the last `window` positions, the query's own
    among them (needs causal).  workspace: optional device tensor of at least
    attention_workspace_bytes(...) bytes, otherwise from torch's allocator."""
    _pair(cache, batch)
    T, D, dev = batch.tokens, cache.head_dim, cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [tokens, q_heads, head_dim] tensor")
    heads = q.shape[1]
    if heads < 1 or heads % cache.heads:
        raise ValueError(f"{heads} query heads over {cache.heads} key heads: a positive multiple is wanted")
    qs = _head_rows(q, "q", T, heads, D, dev, torch.bfloat16)
    if window < 0 or (window and not causal):
        raise ValueError("a window is positive and needs causal")
    window = min(int(window), 0x7FFFFFFF)   # past every position, and what the library's 32 bits hold
    if out is not None:
        _need_kind(out, "out", torch.bfloat16, shape=(T, heads, D))
        _need_place(out, "out", dev)
    if lse is not None:
        _need_kind(lse, "lse", torch.float32, shape=(T, heads))
        _need_place(lse, "lse", dev)
    need = attention_workspace_bytes(cache, batch, heads)
    if workspace is not None:
        _need_place(workspace, "workspace", dev)
    elif need:
        workspace = _empty(need, torch.uint8, dev, stream)
    out = _empty((T, heads, D), torch.bfloat16, dev, stream) if out is None else out
    if lse is None and return_lse:
        lse = _empty((T, heads), torch.float32, dev, stream)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("fp8_kv_attention",
           lib.fp8_kv_attention(cache._ref, batch._ref, q.data_ptr(), qs, heads,
                                float(D ** -0.5 if scale is None else scale), int(bool(causal)), window, out.data_ptr(),
                                _opt(lse), _opt(workspace), nbytes, _stream(stream)))
    return (out, lse) if return_lse else out
