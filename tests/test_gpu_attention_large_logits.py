"""fp8_kv_attention where logits are so large that fp32 holds them in steps of
1/8 to 256 (base 2): the softmax sees their exact differences.

The logits are exact by construction: t_j = T + u n_j with u the fp32 step of T
and small whole n_j, from two products in different dimensions, and the factor
scale * log2(e) is 1.  So the probabilities have no error from the logits, and
the bound is the outputs' bf16 rounding, 2^-8 of the value, sum_j p_j |v_j|
times 2^-11 (the probabilities' fp16) + 2^-16 (exp2, sums, the base of e against
that of 2), and 2^-24 of the largest value a key (fp16 below its normal
range).  lse: 2^-22 of it, a few roundings of a number of its size."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu, say
from test_gpu_attention import store
from test_gpu_kv_cache import tables_for

pytestmark = pytest.mark.gpu
LN2 = np.float32(0.6931472)


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    assert LN2 * np.float32(1.44269504) == np.float32(1.0)
    from fp8_precision_linear_amd import attention
    return attention


def run(fa, e, sign, n, L, H, Hq, D, bs, window=0, rise=None, fmt=0):
    """n new tokens on L in all.  rise (a, b): all keys of a tile of 64 have the
    same logit, a steps more every b tiles; otherwise it varies by up to four."""
    rng = np.random.default_rng(1000 * e + n + L + bs + (sign > 0))
    T, u = sign * 1.5 * 2.0 ** e, 2.0 ** (e - 23)
    tables, nb = tables_for(rng, [L], bs)
    steps = rng.integers(-4, 5, (nb, H, bs)).astype(float)
    if rise:
        for i, b in enumerate(tables[0]):
            steps[b] = rise[0] * ((i * bs + np.arange(bs)) // 64 // rise[1])
    keys = np.zeros((nb, H, bs, D))
    keys[..., 0], keys[..., D - 1] = 1.0, steps
    k = ref.encode_fp8(keys, fmt)
    v = ref.encode_fp8(rng.standard_normal((nb, H, D, bs)) * ref.FMT_MAX[fmt] / 5, fmt)
    kb, vb = np.zeros((nb, H), np.int32), np.full((nb, H), ref.EMAX[fmt], np.int32)
    cache = fa.KVCache(nb, H, D, block_size=bs, fmt=fmt)
    store(cache, k, v, kb, vb)
    q = torch.zeros(n, Hq, D)
    q[..., 0], q[..., D - 1] = T, u
    q = q.to(torch.bfloat16).cuda()
    assert q[0, 0, 0].item() == T and q[0, 0, D - 1].item() == u
    say("large logits", e, sign, n, L, H, Hq, D, bs, window, rise)
    out, lse = fa.kv_attention(cache, fa.KVBatch.from_lists([n], [L], tables), q, scale=float(LN2), window=window,
                               return_lse=True)
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    at = np.arange(L)
    blk = np.array(tables[0])[at // bs]
    val = ref.code_values(fmt)[v[blk, :, :, at % bs]] * 2.0 ** -float(ref.EMAX[fmt])      # [L, H, D]
    t = T + u * steps[blk, :, at % bs]                                                    # [L, H]
    for i in range(n):
        pos = L - n + i
        see = (at <= pos) & ((at > pos - window) if window else True)
        for a in range(Hq):
            s, vv = t[see, a * H // Hq], val[see, a * H // Hq]
            p = np.exp((s - s.max()) * float(LN2))
            want_lse = s.max() * float(LN2) + np.log(p.sum())
            p /= p.sum()
            want, mag = p @ vv, p @ np.abs(vv)
            bound = 2.0 ** -8 * np.abs(want) + mag * (2.0 ** -11 + 2.0 ** -16) + see.sum() * 2.0 ** -24 * np.abs(vv).max()
            assert np.all(np.abs(out[i, a] - want) <= bound), (i, a, out[i, a][:4], want[:4])
            assert abs(lse[i, a] - want_lse) <= 2.0 ** -22 * abs(want_lse), (i, a)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("e", range(20, 32))
def test_every_binade(fa, e, sign):
    """One visible key, and several tiles of them for the same wave, in the
    kernel of few rows and in that of many."""
    for n, L, H, Hq, D, bs in ((3, 40, 2, 4, 64, 32), (3, 400, 1, 2, 128, 64), (2, 600, 1, 1, 64, 16),
                               (90, 90, 1, 2, 64, 32), (70, 250, 1, 2, 128, 64), (40, 250, 1, 1, 256, 16)):
        run(fa, e, sign, n, L, H, Hq, D, bs, window=1)
        run(fa, e, sign, n, L, H, Hq, D, bs)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("e", range(20, 32))
@pytest.mark.parametrize("rise", [1, 2, 4])
def test_rising_tiles(fa, rise, e, sign):
    """Every tile that a wave takes passes the one before by a few steps (the
    waves of the kernel of few rows take every fourth)."""
    run(fa, e, sign, 2, 780, 1, 1, 64, 64, rise=(rise, 4))
    run(fa, e, sign, 1, 780, 1, 2, 128, 16, rise=(rise, 4))
    run(fa, e, sign, 40, 256, 1, 1, 64, 64, rise=(rise, 1))
    run(fa, e, sign, 35, 250, 1, 1, 128, 32, rise=(rise, 1))
