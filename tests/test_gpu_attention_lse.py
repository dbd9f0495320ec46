"""The logarithm of the sum, to its last bit: keys of zeros give logits of zero,
so lse = ln(keys seen).  Every step before the last is exact then (powers of two
and whole numbers below 2^24), so only the rounding to fp32 is left: 2^-24 of
the value, and 2^-45 where the value itself is zero."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, say
from test_gpu_kv_cache import tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    from fp8_precision_linear_amd import attention
    return attention


@pytest.mark.parametrize("H,Hq,D,bs", [(1, 2, 64, 16), (2, 8, 128, 64), (1, 4, 256, 128)])
@pytest.mark.parametrize("new", [1, 7, 150])
def test_counts(fa, H, Hq, D, bs, new):
    rng = np.random.default_rng(new + D)
    lens = [max(new, n) for n in (1, 2, 3, 5, 11, 63, 100, 151, 700, 1501, 5003)]
    tables, nb = tables_for(rng, lens, bs)
    cache = fa.KVCache(nb, H, D, block_size=bs)
    q = torch.randn(new * len(lens), Hq, D, device="cuda").to(torch.bfloat16)
    for batches in ([list(range(len(lens)))], [[i] for i in range(len(lens))]):
        for rows in batches:
            some = [lens[i] for i in rows]
            say("lse", H, Hq, D, bs, new, some)
            batch = fa.KVBatch.from_lists([new] * len(some), some, [tables[i] for i in rows])
            out, lse = fa.kv_attention(cache, batch, q[:new * len(some)], return_lse=True)
            assert (out == 0).all()
            seen = np.concatenate([np.arange(n - new + 1, n + 1) for n in some])
            want = np.log(seen.astype(float))[:, None]
            assert np.all(np.abs(lse.cpu().double().numpy() - want) <= 2.0 ** -24 * want + 2.0 ** -45)
