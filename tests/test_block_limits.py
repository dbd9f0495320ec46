"""The bounds of a batch that come from the host: max_new is only an upper
bound, so however large it is given, launches and workspaces go by the tokens
and lengths that can exist; sizes that 32-bit row numbers cannot hold are
refused before any HIP call."""
import ctypes

import pytest

import fp8_precision_linear_amd as fl
from fp8_precision_linear_amd import attention as fa

L = fl.lib
A = 256        # a fake address
SIZE = {v: k for k, v in fl.STATUS.items()}["FP8_ERR_SIZE"]
BIG = (1 << 31) - 1


def structs(heads=8, batch=3, width=1 << 20, tokens=5, max_new=2, max_len=200):
    return (ctypes.byref(fa._CacheStruct(A, A, A, A, 8, heads, 64, 128, 0, 0)),
            ctypes.byref(fa._BatchStruct(A, A, A, batch, width, tokens, max_new, max_len, 0)))


def workspace(q_heads, **kw):
    return L.fp8_kv_attention_workspace_bytes(*structs(**kw), q_heads)


@pytest.mark.parametrize("kw", [dict(tokens=5), dict(tokens=5, max_len=100000), dict(tokens=1000, max_len=3),
                                dict(tokens=40, max_len=5000, batch=1)])
def test_loose_max_new(kw):
    """A looser bound changes nothing past what tokens and max_len allow."""
    real = min(kw["tokens"], kw.get("max_len", 200))
    want = workspace(64, max_new=real, **kw)
    assert want >= 0
    for loose in (real + 1, 1 << 20, 1 << 27, BIG):
        assert workspace(64, max_new=loose, **kw) == want, loose


def attend(q_heads, **kw):
    c, b = structs(**kw)
    return L.fp8_kv_attention(c, b, A, 1 << 20, q_heads, 0.1, 1, 0, A, A, A, 1 << 60, None)


@pytest.mark.parametrize("kw,q_heads", [
    (dict(heads=1, batch=1, tokens=BIG, max_new=BIG, max_len=1 << 26), 256),
    (dict(heads=1, batch=1, tokens=1 << 24, max_new=1 << 24, max_len=1 << 24), 128),
    (dict(heads=1, batch=1, tokens=1 << 20, max_new=1 << 20, max_len=1 << 25), 1 << 11),
])
def test_rows_past_32_bits(kw, q_heads):
    """Rows of a key head are tokens times query heads a key head."""
    assert workspace(q_heads, **kw) == SIZE
    assert attend(q_heads, **kw) == SIZE


def test_the_largest_rows():
    n = (1 << 24) - 8                       # times 128: just below 2^31 - 128
    kw = dict(heads=1, batch=1, tokens=n, max_new=n, max_len=1 << 24)
    assert workspace(128, **kw) >= 0
