"""Batches that hold prompts beside single tokens and drafts on long caches, as
a server that admits prompts while it decodes makes them: right for every
sequence (test_gpu_attention's bound), and not slower by far than the same
sequences in calls of their own."""
import pytest
import torch

from gpu_util import need_gpu, say
from test_gpu_attention import run

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    from fp8_precision_linear_amd import attention
    return attention


@pytest.mark.parametrize("seqs", [
    [(60, 300), (1, 6000), (2, 4500), (0, 100), (3, 50)],
    [(1, 5000), (1, 40), (90, 90)],
    [(40, 5000), (1, 4200), (33, 33), (32, 4300), (8, 8)],
    [(70, 4500)] + [(1, 30 * i + 1) for i in range(70)],
])
@pytest.mark.parametrize("H,Hq,D,bs,fmt", [(2, 8, 64, 64, E4M3), (1, 1, 64, 16, E4M3), (1, 16, 128, 32, E5M2),
                                           (1, 32, 64, 128, E4M3), (1, 40, 64, 64, E4M3), (1, 4, 256, 64, E4M3)])
def test_mixed(fa, seqs, H, Hq, D, bs, fmt):
    if Hq * D > 1100 and len(seqs) > 10:
        seqs = seqs[:30]
    run(fa, len(seqs) + Hq, seqs, H, Hq, D, bs, fmt)


@pytest.mark.parametrize("window", [100, 4096, 4500])
def test_mixed_windows(fa, window):
    run(fa, window, [(60, 300), (1, 6000), (2, 4500), (100, 5000)], 1, 4, 64, 64, E4M3, window=window)


def test_mixed_not_causal(fa):
    run(fa, 3, [(60, 300), (1, 5000), (3, 4500)], 1, 4, 64, 32, E4M3, causal=False)


# where both kernels take their share: whole row tiles fill the chip (so that no
# chunk needs a workspace, but the even shares do) and one cache is long
SHAPES = [
    ([(300, 300), (1, 6500), (0, 5), (31, 4000), (1, 1), (33, 40), (2, 64), (32, 2000), (1, 65), (0, 0), (5, 5),
      (1, 1500)], 16, 16, 64, 64, E4M3),
    ([(512, 512), (16, 6500), (1, 6500), (17, 300), (0, 9), (3, 3), (1, 33), (2, 100)], 8, 16, 128, 32, E4M3),
    ([(1, 6500), (256, 700), (4, 5000), (5, 77), (1, 1), (0, 4), (3, 1600), (1, 300)], 4, 32, 256, 64, E5M2),
    ([(1, 100), (512, 512), (16, 20), (1, 7000), (2, 130), (0, 3), (15, 15), (1, 6000)], 8, 16, 64, 16, E5M2),
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5000), (True, 70), (False, 0)])
def test_both_kernels(fa, shape, causal, window):
    seqs, H, Hq, D, bs, fmt = SHAPES[shape]
    new, lens = [n for n, _ in seqs], [m for _, m in seqs]
    width = max(-(-m // bs) for m in lens)
    batch = fa.KVBatch.from_lists(new, lens, [[0] * width] * len(seqs))
    assert fa.attention_workspace_bytes(fa.KVCache(1, H, D, block_size=bs, fmt=fmt), batch, Hq) > 0
    alone = [max(new)] * len(seqs)   # no room for a sequence of few rows: one kernel, which does not split here
    batch = fa.KVBatch.from_lists(alone, [max(n, a) for n, a in zip(lens, alone)], [[0] * width] * len(seqs))
    assert fa.attention_workspace_bytes(fa.KVCache(1, H, D, block_size=bs, fmt=fmt), batch, Hq) == 0
    run(fa, 50 + shape, seqs, H, Hq, D, bs, fmt, causal=causal, window=window)


def time_of(f):
    f()
    best = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(4):
            f()
        b.record()
        b.synchronize()
        best.append(a.elapsed_time(b))
    return min(best)


def test_a_long_cache_beside_a_prompt_is_split(fa):
    """512 tokens of a new prompt and one token on 131071 cached, 64 heads on 8:
    both calls of their own take some 75 us, and one kernel for both 2400.  Three
    times as long is far above what one call may cost more than two."""
    H, Hq, D, bs = 8, 64, 128, 64
    cache = fa.KVCache(131072 // bs + 8, H, D, block_size=bs)
    cache.k.random_(0, 100), cache.v.random_(0, 100)
    tables = [list(range(8)), list(range(8, 8 + 131072 // bs))]
    q = torch.randn(513, Hq, D, device="cuda").to(torch.bfloat16)
    both = fa.KVBatch.from_lists([512, 1], [512, 131071], tables)
    prompt, token = (fa.KVBatch.from_lists([n], [m], [t]) for n, m, t in ((512, 512, tables[0]), (1, 131071, tables[1])))
    say("a long cache beside a prompt")
    apart = time_of(lambda: (fa.kv_attention(cache, prompt, q[:512]), fa.kv_attention(cache, token, q[512:])))
    assert time_of(lambda: fa.kv_attention(cache, both, q)) < 3 * apart
