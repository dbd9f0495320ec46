"""Batches whose grid is larger than one launch may be (2^32 lanes): a ragged
batch with one long sequence has a workgroup for every block that any sequence
might touch.  Each result equals that of the same sequences in calls that fit
one launch."""
import pytest
import torch

from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    from fp8_precision_linear_amd import attention
    return attention


def tables(lens, bs):
    out, at = [], 0
    for n in lens:
        used = -(-n // bs)
        out.append(list(range(at, at + used)))
        at += used
    return out, at


def noise(cache):
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (cache.k, cache.v):
        t.copy_(torch.randint(0, 127, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (cache.k_bias, cache.v_bias):
        t.copy_(torch.randint(2, 9, t.shape, generator=g, device="cuda", dtype=torch.int32))


def test_read(fa):
    bs, H, D = 16, 8, 64
    lens = [5] * 60 + [131072] + [9] * 67        # 128 * 8193 * 8 * 2 workgroups of 256 lanes
    t, nb = tables(lens, bs)
    cache = fa.KVCache(nb, H, D, block_size=bs)
    noise(cache)
    say("read", len(lens), max(lens))
    k, v = fa.kv_read(cache, fa.KVBatch.from_lists(lens, lens, t))
    at = 0
    for part in (slice(0, 60), slice(60, 61), slice(61, 128)):
        some = lens[part]
        for got, want in zip((k, v), fa.kv_read(cache, fa.KVBatch.from_lists(some, some, t[part]))):
            assert torch.equal(got[at:at + sum(some)], want)
        at += sum(some)


def test_append(fa):
    bs, H, D = 16, 1, 64
    lens = [1] * 2000 + [131072] + [1] * 47      # 2048 * (8193 + queries') workgroups of 256 lanes
    t, nb = tables(lens, bs)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(sum(lens), 3 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    one, parts = (fa.KVCache(nb, H, D, block_size=bs) for _ in range(2))
    say("append", len(lens), max(lens))
    q = fa.kv_append(one, fa.KVBatch.from_lists(lens, lens, t), x[:, :H], x[:, H:2 * H], q=x[:, 2 * H:])
    at = 0
    for part in (slice(0, 2000), slice(2000, 2001), slice(2001, 2048)):
        some = lens[part]
        rows = x[at:at + sum(some)]
        want = fa.kv_append(parts, fa.KVBatch.from_lists(some, some, t[part]), rows[:, :H], rows[:, H:2 * H],
                            q=rows[:, 2 * H:])
        assert torch.equal(q[at:at + sum(some)], want)
        at += sum(some)
    for a, b in zip((one.k, one.v, one.k_bias, one.v_bias), (parts.k, parts.v, parts.k_bias, parts.v_bias)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("new", [1, 40])
def test_attention(fa, new):
    """2^24 workgroups of 256 lanes and a few more, nearly all of sequences
    without a new token; the kernel of few rows, and that of many."""
    bs, H, D, B = 16, 64, 64, (1 << 18) + 3
    cache = fa.KVCache(12, H, D, block_size=bs)
    noise(cache)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, lens, table = i32(B + 1), i32(B), i32(B, 3)
    busy = [0, 1 << 17, B - 1]
    some = [[0, 1, 2], [3, 4, 5], [6, 7, 8]]
    for n, i in enumerate(busy):
        cu[i + 1:] = (n + 1) * new
        lens[i] = 41 + n
        table[i] = torch.tensor(some[n], dtype=torch.int32)
    q = torch.randn(3 * new, H, D, device="cuda").to(torch.bfloat16)
    say("attention", new, B)
    out, lse = fa.kv_attention(cache, fa.KVBatch(cu, lens, table, max_new=new, max_len=43, tokens=3 * new), q,
                               return_lse=True)
    want, want_lse = fa.kv_attention(cache, fa.KVBatch.from_lists([new] * 3, [41, 42, 43], some), q, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
