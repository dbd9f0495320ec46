"""A NaN value that a query sees makes its output NaN also where the keys are
split and the part that holds it counts for nothing beside the others (weights
below 2^-149 of the largest): as 0 * NaN does within a part.

The logits (base 2) are 0 for the first half of the keys and 512 for the other,
exactly; the outputs are the plain mean of the latter's values, to bf16's
rounding and 2^-11 of the magnitudes (the probabilities' fp16)."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu, say
from test_gpu_attention import NAN_CODE, store
from test_gpu_attention_large_logits import LN2
from test_gpu_kv_cache import tables_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,length,H,Hq,D,bs", [(1, 2000, 1, 2, 64, 64), (2, 1700, 1, 16, 128, 64),
                                                  (2, 1700, 60, 60, 64, 32), (40, 700, 1, 1, 64, 64),
                                                  (34, 4500, 1, 1, 64, 32)])
@pytest.mark.parametrize("dead", [3, 130, None])
def test_nan_in_a_part_of_no_weight(new, length, H, Hq, D, bs, dead):
    need_gpu()
    from fp8_precision_linear_amd import attention as fa
    rng = np.random.default_rng(length)
    tables, nb = tables_for(rng, [length], bs)
    at = np.arange(length)
    blk = np.array(tables[0])[at // bs]
    k = np.zeros((nb, H, bs, D))
    k[blk, :, at % bs, 0] = np.where(at < length // 2, 0.0, 8.0)[:, None]
    v = ref.encode_fp8(rng.standard_normal((nb, H, D, bs)), 0)
    if dead is not None:
        v[tables[0][dead // bs], :, 5::9, dead % bs] = NAN_CODE
    cache = fa.KVCache(nb, H, D, block_size=bs)
    store(cache, ref.encode_fp8(k, 0), v, np.zeros((nb, H), np.int32), np.zeros((nb, H), np.int32))
    q = torch.zeros(new, Hq, D)
    q[..., 0] = 64.0
    say("NaN in a part of no weight", new, length, H, Hq, D, bs, dead)
    out = fa.kv_attention(cache, fa.KVBatch.from_lists([new], [length], tables), q.to(torch.bfloat16).cuda(),
                          scale=float(LN2)).cpu().double().numpy()
    val = ref.code_values(0)[v[blk, :, :, at % bs]]
    bad = np.zeros(D, bool)
    bad[5::9] = dead is not None
    assert np.array_equal(np.isnan(out), np.broadcast_to(bad, out.shape))
    for i in range(new):
        vis = val[length // 2:length - new + i + 1]
        for a in range(Hq):
            vv = vis[:, a * H // Hq]
            bound = 2.0 ** -8 * np.abs(vv.mean(0)) + 2.0 ** -10 * np.abs(vv).mean(0)
            assert np.all(np.abs(out[i, a] - vv.mean(0))[~bad] <= bound[~bad]), (i, a)
