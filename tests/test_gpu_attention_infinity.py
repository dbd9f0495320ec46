"""Infinity codes among the cached values (E5M2 has them; a caller's own cache
may hold some): an output whose token and dimension a query sees is NaN, as for
a NaN code, wherever the token lies in its tile and whoever else sees it; the
other queries and dimensions do not notice."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu, say
from test_gpu_attention import NAN_CODE, build, check, store

pytestmark = pytest.mark.gpu
E5M2 = 1


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    from fp8_precision_linear_amd import attention
    return attention


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("new,length,window", [(1, 400, 0), (3, 400, 0), (3, 300, 20), (100, 250, 0), (90, 400, 30),
                                               (1, 2500, 0)])
def test_seen_infinities_make_nan(fa, D, bs, new, length, window):
    H, Hq = 1, 2
    for seed, qscale in ((1, 1.0), (2, 30.0)):
        rng = np.random.default_rng(seed + length)
        cache, tables, k, v, kb, vb = build(fa, rng, [length], H, D, bs, E5M2)
        given = v.copy()
        # one sign a dimension, both in one, in whole tiles and in the last
        for p, dims, codes in ((70, slice(5, D, 9), 0x7C), (length - 20, slice(6, D, 11), 0xFC),
                               (length - 2, slice(7, D, 13), 0x7C), (75, slice(5, D, 18), 0xFC)):
            given[tables[0][p // bs], :, dims, p % bs] = codes
            v[tables[0][p // bs], :, dims, p % bs] = NAN_CODE
        store(cache, k, given, kb, vb)
        q = torch.from_numpy(rng.standard_normal((new, Hq, D)).astype(np.float32) * qscale).to(torch.bfloat16).cuda()
        say("infinity codes", D, bs, new, length, window, qscale)
        out, lse = fa.kv_attention(cache, fa.KVBatch.from_lists([new], [length], tables), q, window=window,
                                   return_lse=True)
        check(out, lse, q, [0, new], [new], [length], tables, k, v, kb, vb, bs, E5M2, D ** -0.5, True, window,
              (D, bs, new, length, window, qscale))


@pytest.mark.parametrize("code", [0x7C, 0xFC, NAN_CODE])
@pytest.mark.parametrize("new,length,window", [(1, 400, 0), (3, 300, 20), (100, 250, 0), (90, 400, 30), (1, 2500, 0)])
def test_infinite_and_nan_keys(fa, new, length, window, code):
    """A logit of +infinity or NaN makes the whole output NaN, one of -infinity
    has no weight; queries that do not see the key do not notice."""
    H, Hq, D, bs = 1, 2, 64, 32
    rng = np.random.default_rng(length + code)
    cache, tables, k, v, kb, vb = build(fa, rng, [length], H, D, bs, E5M2)
    for p in (70, length - 15):
        k[tables[0][p // bs], :, p % bs, 9] = code
    store(cache, k, v, kb, vb)
    q = torch.from_numpy(rng.standard_normal((new, Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    say("infinite keys", new, length, window, code)
    out, lse = fa.kv_attention(cache, fa.KVBatch.from_lists([new], [length], tables), q, window=window, return_lse=True)
    check(out, lse, q, [0, new], [new], [length], tables, k, v, kb, vb, bs, E5M2, D ** -0.5, True, window, (new, code))
    qn, gone = q.cpu().double().numpy(), np.isnan(out.cpu().float().numpy()).all(-1)
    for i in range(new):
        at = length - new + i
        sees = any(p <= at and (not window or p > at - window) for p in (70, length - 15))
        for a in range(Hq):
            assert gone[i, a] == (sees and (code == NAN_CODE or (qn[i, a, 9] > 0) == (code == 0x7C)))
            assert np.isnan(lse[i, a].item()) == gone[i, a]
