"""max_new given far looser than the batch needs: the same cache, read-back,
outputs and sums, bit for bit, as with the bound that tokens and max_len set."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, say
from test_gpu_attention import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,lens,Hq", [([1, 1], [300, 40], 8), ([70, 3], [200, 2000], 2), ([2, 1], [5, 2000], 128)])
def test_loose_max_new(new, lens, Hq):
    need_gpu()
    from fp8_precision_linear_amd import attention as fa
    H, D, bs, T = 2, 64, 32, sum(new)
    results = []
    x = torch.randn(T, 2 * H + Hq, D, device="cuda")
    for bound in (T, 1000, 1 << 24, (1 << 31) - 1):
        cache, tables, *_ = build(fa, np.random.default_rng(4), lens, H, D, bs, 0)
        b = fa.KVBatch.from_lists(new, lens, tables)
        batch = fa.KVBatch(b.cu_tokens, b.lens, b.block_table, max_new=bound, max_len=b.max_len, tokens=T)
        say("loose max_new", new, lens, Hq, bound)
        q = fa.kv_append(cache, batch, x[:, :H], x[:, H:2 * H], q=x[:, 2 * H:])
        results.append((q, cache.k, cache.v, cache.k_bias, cache.v_bias, *fa.kv_read(cache, batch),
                        *fa.kv_attention(cache, batch, q, return_lse=True)))
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
