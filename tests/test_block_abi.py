"""The entry points of include/fp8lin_block.h without a GPU: exported, bound,
and every bad argument refused on the host with the documented status, before
any HIP call.  The Python wrappers' own refusals likewise."""
import ctypes
import os
import re

import pytest
import torch

import fp8_precision_linear_amd as fl
from fp8_precision_linear_amd import attention as fa
from fp8_precision_linear_amd import decoder, norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = fl.lib
P = ctypes.c_void_p
A, MIS, MISW = 256, 264, 258        # fake addresses: aligned, 8 bytes off, 2 bytes off


def status(name):
    return {v: k for k, v in fl.STATUS.items()}["FP8_ERR_" + name]


def test_every_declared_function_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8lin_block.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp8_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 9
    for n in names:
        assert hasattr(L, n) and n in fl.SIGNATURES, n


def caller(fn, names, ok):
    def call(**kw):
        a = dict(zip(names, ok))
        for k, v in kw.items():
            assert k in a, k
            a[k] = v
        return fn(*a.values())
    return call


FWD = ["x", "xt", "r", "rt", "w", "wt", "rows", "d", "eps", "h", "rstd"]
FWD_OK = [A, 1, A, 0, A, 1, 4, 64, 1e-5, A, A]
KINDS = {"fwd": (L.fp8_rmsnorm_fwd, FWD + ["y", "amax", "stream"], FWD_OK + [A, A, None]),
         "cast": (L.fp8_rmsnorm_cast, FWD + ["bias", "fmt", "y", "amax", "stream"], FWD_OK + [A, 0, A, A, None]),
         "quantize": (L.fp8_rmsnorm_quantize, FWD + ["fmt", "margin", "y", "row_amax", "amax", "bias", "stream"],
                      FWD_OK + [0, 0, A, A, A, A, None])}


@pytest.mark.parametrize("kind", list(KINDS))
def test_norm_forward_checks(kind):
    call = caller(*KINDS[kind])
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=32772), dict(d=16385), dict(d=-4)):
        assert call(**bad) == status("SIZE"), bad
    for bad in (dict(xt=2), dict(rt=-1), dict(wt=5)):
        assert call(**bad) == status("DTYPE"), bad
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(h=None)):
        assert call(**bad) == status("NULL"), bad
    for bad in (dict(x=MIS), dict(w=MIS), dict(y=MIS), dict(r=MIS), dict(h=MIS), dict(rstd=MISW), dict(amax=MISW)):
        assert call(**bad) == status("ALIGN"), bad
    if kind != "fwd":
        assert call(fmt=2) == status("FORMAT") and call(fmt=7) == status("FORMAT")
        assert call(bias=None) == status("NULL") and call(bias=MISW) == status("ALIGN")
    if kind == "quantize":
        assert call(margin=65) == call(margin=-65) == status("MARGIN")
        assert call(rstd=None) == call(row_amax=None) == call(amax=None) == status("NULL")
        assert call(row_amax=MISW) == status("ALIGN")
    else:
        assert call(rows=0, x=None, w=None, y=None, h=None, amax=None) == 0   # nothing to write


def test_norm_backward_checks():
    names = ["dy", "yt", "h", "ht", "w", "wt", "rstd", "dh", "rows", "d", "dx", "dw", "amax", "ws", "bytes", "stream"]
    need = L.fp8_rmsnorm_bwd_workspace_bytes(4, 64)
    call = caller(L.fp8_rmsnorm_bwd, names, [A, 1, A, 0, A, 1, A, A, 4, 64, A, A, A, A, need, None])
    assert need > 0
    for rows, d in ((-1, 64), (4, 0), (4, 40000), (4, 16387), (1 << 31, 4)):
        assert L.fp8_rmsnorm_bwd_workspace_bytes(rows, d) == status("SIZE")
        assert call(rows=rows, d=d) == status("SIZE")
    assert call(bytes=need - 1) == status("SIZE")
    for bad in (dict(yt=3), dict(ht=-1), dict(wt=9)):
        assert call(**bad) == status("DTYPE")
    for k in ("dy", "h", "w", "rstd", "dx", "dw", "ws"):
        assert call(**{k: None}) == status("NULL"), k
    for k in ("dy", "h", "w", "dh", "dx", "dw", "ws"):
        assert call(**{k: MIS}) == status("ALIGN"), k
    assert call(rstd=MISW) == call(amax=MISW) == status("ALIGN")


def structs(**kw):
    c = fa._CacheStruct(A, A, A, A, 8, 2, 64, 128, 0, 0)
    b = fa._BatchStruct(A, A, A, 3, 4, 5, 2, 200, 0)
    for k, v in kw.items():
        if any(k == f[0] for f in c._fields_):
            setattr(c, k, v)
        else:
            setattr(b, k, v)
    return ctypes.byref(c), ctypes.byref(b)


def append(q=A, heads=4, dtype=1, k=A, ks=1024, v=A, vs=1024, qs=1024, q_out=A, cos=A, sin=A, rows=200, pairs=0, **kw):
    c, b = structs(**kw)
    return L.fp8_kv_append(c, b, k, ks, v, vs, dtype, q, qs, heads, q_out, cos, sin, rows, pairs, None)


def attend(q=A, qs=512, heads=4, scale=0.1, causal=1, window=0, out=A, lse=A, ws=A, nbytes=1 << 40, **kw):
    c, b = structs(**kw)
    return L.fp8_kv_attention(c, b, q, qs, heads, scale, causal, window, out, lse, ws, nbytes, None)


def read(dtype=0, k_out=A, v_out=A, **kw):
    c, b = structs(**kw)
    return L.fp8_kv_read(c, b, dtype, k_out, v_out, None)


@pytest.mark.parametrize("call", [append, attend, read], ids=["append", "attention", "read"])
def test_cache_and_batch_checks(call):
    for bad in (dict(num_blocks=0), dict(num_blocks=-1), dict(block_size=48), dict(block_size=8), dict(head_dim=96),
                dict(head_dim=512), dict(batch=-1), dict(table_width=-1), dict(tokens=-1), dict(max_new=-1),
                dict(max_len=-1), dict(max_len=257), dict(max_len=(1 << 30) + 1)):
        assert call(**bad) == status("SIZE"), bad
    assert call(fmt=2) == status("FORMAT")
    for k in ("k_bias", "v_bias", "cu_tokens", "lens", "block_table"):
        assert call(**{k: None}) == status("NULL"), k
        assert call(**{k: MISW}) == status("ALIGN"), k
    # nothing to do: nothing else is looked at
    for empty in (dict(batch=0), dict(tokens=0), dict(max_new=0)):
        assert call(cu_tokens=None, lens=None, block_table=None, **empty) == 0


def test_null_structs():
    c, b = structs()
    assert L.fp8_kv_read(None, b, 0, A, A, None) == L.fp8_kv_read(c, None, 0, A, A, None) == status("NULL")
    assert L.fp8_kv_attention_workspace_bytes(None, b, 4) == status("NULL")


def test_append_checks():
    assert append(dtype=2) == status("DTYPE")
    assert append(heads=0) == status("SIZE")
    for k in ("k", "v", "q_out"):
        assert append(**{k: None}) == status("NULL"), k
        assert append(**{k: MIS}) == status("ALIGN"), k
    assert append(q=MIS) == status("ALIGN")
    assert append(cos=None) == append(sin=None) == status("NULL")
    assert append(cos=MIS) == append(sin=MIS) == status("ALIGN")
    assert append(rows=199) == status("SIZE")
    for k in ("ks", "vs", "qs"):
        assert append(**{k: 100}) == status("SIZE"), k          # rows overlap
        assert append(**{k: 1026}) == status("ALIGN"), k        # rows not on 16 bytes
    assert append(batch=1 << 30, max_new=100) == status("SIZE")   # too many workgroups
    assert read(dtype=3) == status("DTYPE")
    assert read(k_out=MIS) == read(v_out=MIS) == status("ALIGN")
    assert read(k_out=None, v_out=None) == 0


def test_attention_checks():
    assert attend(heads=3) == attend(heads=0) == attend(heads=-2) == status("SIZE")
    assert attend(window=-1) == attend(window=5, causal=0) == status("SIZE")
    assert attend(scale=float("nan")) == attend(scale=float("inf")) == status("SIZE")
    assert attend(q=None) == attend(out=None) == status("NULL")
    assert attend(q=MIS) == attend(out=MIS) == attend(lse=MISW) == attend(ws=MIS) == status("ALIGN")
    assert attend(qs=100) == status("SIZE") and attend(qs=516) == status("ALIGN")
    c, b = structs(max_len=100000, table_width=2000)
    need = L.fp8_kv_attention_workspace_bytes(c, b, 4)
    assert need > 0
    assert attend(max_len=100000, table_width=2000, nbytes=need - 1) == status("SIZE")
    assert attend(max_len=100000, table_width=2000, ws=None, nbytes=0) == status("NULL")
    assert L.fp8_kv_attention_workspace_bytes(*structs(), 4) == 0    # short sequences: none


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on a real device")
def test_valid_calls_without_a_device_report_no_device():
    for kind in KINDS:
        assert caller(*KINDS[kind])() == status("DEVICE")
    assert append() == attend() == read() == status("DEVICE")


def test_norm_wrappers_refuse():
    x, w = torch.zeros(2, 8), torch.ones(8)
    with pytest.raises(ValueError, match="CUDA"):
        norm.rmsnorm_fwd(x, w)
    with pytest.raises(ValueError, match="do not match"):
        norm.rmsnorm_fwd(x, torch.ones(9))
    with pytest.raises(ValueError, match="eps"):
        norm.rmsnorm_fwd(x, w, eps=-1.0)
    with pytest.raises(ValueError, match="eps"):
        norm.rmsnorm_fwd(x, w, eps=float("nan"))
    with pytest.raises(ValueError, match="residual"):
        norm.rmsnorm_fwd(x, w, residual=torch.zeros(3, 8))
    with pytest.raises(ValueError, match="residual"):
        norm.rmsnorm_fwd(x, w, h=torch.zeros(2, 8))
    with pytest.raises(TypeError):
        norm.rmsnorm_fwd(x.half(), w)
    with pytest.raises(ValueError, match="elements"):
        norm.rmsnorm_fwd(torch.zeros(1, 16385), torch.zeros(16385))
    with pytest.raises(ValueError, match="do not match"):
        norm.rmsnorm_bwd(torch.zeros(2, 9), x, w, torch.zeros(2))
    with pytest.raises(ValueError, match="rstd"):
        norm.rmsnorm_bwd(x, x, w, torch.zeros(3))
    with pytest.raises(fl.Fp8Error):
        norm.rmsnorm_bwd_workspace_bytes(-1, 8)


def test_attention_wrappers_refuse():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        fa.KVCache(2, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="block sizes"):
        fa.KVCache(2, 2, 96, device="cpu")
    with pytest.raises(ValueError, match="E4M3 or E5M2"):
        fa.KVCache(2, 2, 64, fmt=fl.E3M4, device="cpu")
    with pytest.raises(ValueError, match="at least one"):
        fa.KVCache(0, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="v must have shape"):
        fa.KVCache.from_tensors(u8(2, 2, 64, 128), u8(2, 2, 64, 128), i32(2, 2), i32(2, 2))
    with pytest.raises(ValueError, match="k_bias"):
        fa.KVCache.from_tensors(u8(2, 2, 64, 128), u8(2, 2, 128, 64), i32(2, 3), i32(2, 2))
    with pytest.raises(ValueError, match="cu_tokens"):
        fa.KVBatch(i32(3), i32(3), i32(3, 1), 1, 1, 3)
    with pytest.raises(ValueError, match="block_table"):
        fa.KVBatch(i32(4), i32(3), i32(2, 1), 1, 1, 3)
    with pytest.raises(ValueError, match="among its length"):
        fa.KVBatch.from_lists([3], [2], [[0]], device="cpu")
    with pytest.raises(ValueError, match="one entry"):
        fa.KVBatch.from_lists([1, 1], [2], [[0]], device="cpu")
    with pytest.raises(ValueError, match="KVCache"):
        fa.kv_attention(None, None, torch.zeros(1, 1, 64))


def test_decoder_refuses():
    z = torch.zeros
    with pytest.raises(ValueError, match="do not fit"):
        decoder.FP8DecoderLayer(z(64), z(100, 64), z(64, 64), z(64), z(128, 64), z(64, 64), 1, 1, 64)
    with pytest.raises(ValueError, match="chain"):
        decoder.FP8DecoderLayer(z(64), z(192, 64), z(64, 64), z(64), z(128, 64), z(64, 60), 1, 1, 64)
