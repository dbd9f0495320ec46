"""A window that passes 32 bits sees everything, as any window longer than the
sequence does."""
import sys

import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from test_gpu_attention import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,length", [(1, 300), (80, 200)])
def test_windows_past_32_bits(new, length):
    need_gpu()
    from fp8_precision_linear_amd import attention as fa
    rng = np.random.default_rng(1)
    cache, tables, *_ = build(fa, rng, [length], 1, 64, 64, 0)
    batch = fa.KVBatch.from_lists([new], [length], tables)
    q = torch.randn(new, 2, 64, device="cuda").to(torch.bfloat16)
    want = fa.kv_attention(cache, batch, q)
    for window in ((1 << 31) - 1, 1 << 31, (1 << 32) + 5, sys.maxsize):
        assert torch.equal(fa.kv_attention(cache, batch, q, window=window), want), window
