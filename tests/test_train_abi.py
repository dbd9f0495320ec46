"""The entry points of include/fp8lin_train.h without a GPU: exported, bound,
and every bad argument refused on the host with the documented status, before
any HIP call.  The Python wrappers' own refusals likewise."""
import ctypes
import os
import re

import pytest
import torch

import fp8_precision_linear_amd as fl
from fp8_precision_linear_amd import embedding as em
from fp8_precision_linear_amd import qk_norm as qn
from fp8_precision_linear_amd import self_attention as sa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = fl.lib
A, MIS, MISW = 256, 264, 258        # fake addresses: aligned, 8 bytes off, 2 bytes off


def status(name):
    return {v: k for k, v in fl.STATUS.items()}["FP8_ERR_" + name]


def test_every_declared_function_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8lin_train.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp8_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 9
    for n in names:
        assert hasattr(L, n) and n in fl.SIGNATURES, n


def caller(fn, **ok):
    def call(**kw):
        assert all(k in ok for k in kw), kw
        return fn(*{**ok, **kw}.values())
    return call


def refused(call, name, *bads):
    for bad in bads:
        assert call(**bad) == status(name), (name, bad)


def each(keys, value):
    return [{k: value} for k in keys.split()]


def test_embedding_checks():
    call = caller(L.fp8_embedding_fwd, ids=A, bits=64, tokens=4, table=A, tt=1, vocab=10, d=8, scale=1.0, out=A, ot=0,
                  stream=None)
    refused(call, "DTYPE", dict(bits=16), dict(tt=2), dict(ot=-1))
    refused(call, "SIZE", dict(tokens=-1), dict(vocab=-1), dict(d=0), dict(d=(1 << 24) + 1), dict(vocab=1 << 31),
            dict(tokens=1 << 31), dict(tokens=1 << 30, d=1 << 20))
    refused(call, "NULL", *each("ids table out", None))
    refused(call, "ALIGN", *each("table out", MIS), dict(ids=260), dict(ids=MISW, bits=32))
    assert call(tokens=0, ids=None, table=None, out=None) == 0
    need = L.fp8_embedding_bwd_workspace_bytes(4, 10, 8)
    assert need > 0
    call = caller(L.fp8_embedding_bwd, dout=A, dt=1, ids=A, bits=64, tokens=4, vocab=10, d=8, scale=1.0, acc=0, dtable=A,
                  ws=A, nbytes=need, stream=None)
    refused(call, "DTYPE", dict(bits=0), dict(dt=5))
    refused(call, "SIZE", dict(tokens=-1), dict(vocab=-2), dict(d=-1), dict(nbytes=need - 1))
    refused(call, "NULL", *each("ids dout dtable ws", None))
    refused(call, "ALIGN", *each("dout dtable ws", MIS))
    assert call(vocab=0, dtable=None) == call(tokens=0, acc=1, dtable=None) == 0
    for bad in ((-1, 10, 8), (4, -1, 8), (4, 10, 0), (1 << 31, 10, 8)):
        assert L.fp8_embedding_bwd_workspace_bytes(*bad) == status("SIZE")


QK = dict(x=A, xt=1, x_stride=512, tokens=5, q_heads=4, kv_heads=2, head_dim=64, wq=A, wk=A, wt=1, eps=1e-5, positions=A,
          cos=A, sin=A, rows=9, pairs=0)


def qk_refusals(call):
    refused(call, "SIZE", dict(tokens=-1), dict(q_heads=0), dict(kv_heads=-1), dict(head_dim=96), dict(x_stride=511),
            dict(eps=-1.0), dict(eps=float("nan")), dict(rows=0), dict(rows=4, positions=None), dict(q_heads=1 << 30))
    refused(call, "DTYPE", dict(xt=2), dict(wt=3))
    refused(call, "NULL", *each("x wq wk cos sin", None))
    refused(call, "ALIGN", *each("x wq wk cos sin", MIS), dict(positions=MISW), dict(x_stride=513))


def test_qk_checks():
    call = caller(L.fp8_qk_norm_rope_fwd, **QK, y=A, stream=None)
    qk_refusals(call)
    refused(call, "NULL", dict(y=None))
    refused(call, "ALIGN", dict(y=MIS))
    assert call(tokens=0, x=None, y=None) == 0
    need = L.fp8_qk_norm_rope_bwd_workspace_bytes(5, 4, 2, 64)
    assert need > 0
    call = caller(L.fp8_qk_norm_rope_bwd, dq=A, dqs=256, dk=A, dks=128, dv=A, dvs=128, **QK, dx=A, dwq=A, dwk=A, ws=A,
                  nbytes=need, stream=None)
    qk_refusals(call)
    refused(call, "SIZE", dict(nbytes=need - 1), dict(dqs=255), dict(dks=127), dict(dvs=64))
    refused(call, "NULL", *each("dq dk dv dx dwq dwk ws", None))
    refused(call, "ALIGN", *each("dq dk dv dx ws", MIS), dict(dwq=MISW), dict(dwk=MISW), dict(dqs=257))
    assert call(tokens=0, wq=None, wk=None, dq=None, dx=None, ws=None, nbytes=0) == 0
    for bad in ((-1, 4, 2, 64), (5, 0, 2, 64), (5, 4, 0, 64), (5, 4, 2, 80)):
        assert L.fp8_qk_norm_rope_bwd_workspace_bytes(*bad) == status("SIZE")


def seqs(**kw):
    s = dict(cu=A, batch=3, tokens=50, max_len=30, pad=0)
    s.update(kw)
    return ctypes.byref(sa._SeqsStruct(*s.values()))


HEADS = dict(q_heads=4, kv_heads=2, head_dim=64)
MASK = dict(scale=0.1, causal=1, window=0)


def attention_refusals(call):
    refused(call, "NULL", dict(seqs=None), dict(seqs=seqs(cu=None)))
    refused(call, "SIZE", *(dict(seqs=seqs(**bad)) for bad in (dict(batch=-1), dict(tokens=-1), dict(max_len=-1),
                                                               dict(max_len=(1 << 30) + 1))))
    refused(call, "SIZE", dict(q_heads=3), dict(q_heads=0), dict(kv_heads=0), dict(head_dim=32), dict(window=-1),
            dict(window=5, causal=0), dict(scale=float("inf")), dict(scale=float("nan")), dict(qs=255), dict(ks=100),
            dict(vs=64), dict(qs=(1 << 24) + 8), dict(vs=1 << 32))
    refused(call, "NULL", *each("q k v out lse", None))
    refused(call, "ALIGN", *each("q k v out", MIS), dict(lse=MISW), dict(qs=260), dict(seqs=seqs(cu=MISW)))
    for empty in (dict(batch=0), dict(tokens=0), dict(max_len=0)):
        assert call(seqs=seqs(**empty), q=None, out=None) == 0


def test_attention_checks():
    rows = dict(q=A, qs=256, k=A, ks=128, v=A, vs=128)
    attention_refusals(caller(L.fp8_attention_fwd, **rows, seqs=seqs(), **HEADS, **MASK, out=A, lse=A, stream=None))
    need = L.fp8_attention_bwd_workspace_bytes(seqs(), 4, 2, 64)
    assert need > 0 and L.fp8_attention_bwd_workspace_bytes(seqs(batch=0), 4, 2, 64) == 0
    call = caller(L.fp8_attention_bwd, dout=A, gs=256, **rows, out=A, lse=A, seqs=seqs(), **HEADS, **MASK, dq=A, dqs=256,
                  dk=A, dks=128, dv=A, dvs=128, ws=A, nbytes=need, stream=None)
    attention_refusals(call)
    refused(call, "SIZE", dict(nbytes=need - 1), dict(gs=128), dict(dqs=255), dict(dks=1), dict(dvs=1 << 30))
    refused(call, "NULL", *each("dout dq dk dv ws", None))
    refused(call, "ALIGN", *each("dout dq dk dv ws", MIS), dict(dks=132))
    for bad in ((3, 2, 64), (4, 0, 64), (4, 2, 65)):
        assert L.fp8_attention_bwd_workspace_bytes(seqs(), *bad) == status("SIZE")


# ------------------------------------------------------------------ the Python wrappers
def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_embedding_wrappers_refuse():
    ids, table = torch.zeros(4, dtype=torch.int64), torch.zeros(9, 8)
    for bad in ((ids.float(), table), (None, table), (ids, table[0]), (ids, None), (ids, table[:, :0]), (ids, table)):
        with pytest.raises(ValueError):     # (the last: not on the GPU)
            em.embedding_fwd(*bad)
    with pytest.raises(TypeError):
        em.embedding_fwd(ids, table.half())
    with pytest.raises(TypeError):
        em.embedding_fwd(ids, table, dtype=torch.float16)
    for bad in (dict(dout=torch.zeros(3, 8)), dict(dout=None), dict(accumulate=True), dict(ids=ids.to(torch.int16)), {}):
        with pytest.raises(ValueError):
            em.embedding_bwd(**{**dict(dout=torch.zeros(4, 8), ids=ids, vocab=9), **bad})
    with pytest.raises(fl.Fp8Error):
        em.embedding_bwd(torch.zeros(4, 8), ids, -1)


def test_qk_wrappers_refuse():
    x, w = torch.zeros(5, 8, 64), torch.ones(64)
    for a in ((x[0], 4, 2), (x, 4, 3), (x, 8, 0), (x[..., :32], 4, 2), (None, 4, 2), (x, 4, 2)):
        with pytest.raises(ValueError):
            qn.qk_norm_rope_fwd(*a)
    with pytest.raises(ValueError):
        qn.qk_norm_rope_fwd(x, 4, 2, eps=-1.0)
    with pytest.raises(TypeError):
        qn.qk_norm_rope_fwd(x.half(), 4, 2)
    with pytest.raises(ValueError):
        qn.qk_norm_rope_bwd(bf(5, 4, 64), bf(5, 2, 64)[0], bf(5, 2, 64), x, w, w)
    with pytest.raises(fl.Fp8Error):
        qn.qk_norm_rope_bwd_workspace_bytes(5, 4, 2, 63)


def test_attention_wrappers_refuse():
    with pytest.raises(ValueError):
        sa.Sequences.from_lists([3, -1], device="cpu")
    with pytest.raises(ValueError):
        sa.Sequences.from_lists([3, 1], device="cpu")       # not on the GPU
    with pytest.raises(ValueError):
        sa.Sequences(torch.zeros(3), 1, 1)
    with pytest.raises(ValueError):
        sa.attention_fwd(bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), None)
