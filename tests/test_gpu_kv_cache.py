"""The paged FP8 cache: fp8_kv_append and fp8_kv_read against their
definitions, bit for bit (rotation in fp32 with every product and sum rounded,
codes and scales exact)."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    from fp8_precision_linear_amd import attention
    return attention


def tables_for(rng, lens, bs, spare=3):
    used = [-(-n // bs) for n in lens]
    order = rng.permutation(sum(used) + spare)
    out, at = [], 0
    for u in used:
        out.append([int(b) for b in order[at:at + u]])
        at += u
    return out, len(order)


def filled_cache(fa, rng, nb, H, D, bs, fmt):
    """A cache with something in every slot, NaN codes among it."""
    c = fa.KVCache(nb, H, D, block_size=bs, fmt=fmt)
    for t in (c.k, c.v):
        t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape, dtype=np.uint8)))
    for t in (c.k_bias, c.v_bias):
        t.copy_(torch.from_numpy(rng.integers(3, 9, t.shape).astype(np.int32)))
    return c


def snapshot(c):
    return [t.cpu().numpy().copy() for t in (c.k, c.v, c.k_bias, c.v_bias)]


def rope_tables(n, D):
    inv = 10000.0 ** (-np.arange(0, D, 2) / D)
    a = np.arange(n)[:, None] * inv
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


CASES = [  # (new, len) of each sequence, heads, query heads, D, block size, fmt, dtype, rope
    ([(1, 1)], 1, 1, 64, 16, E4M3, "f32", None),
    ([(1, 17), (1, 64), (1, 65)], 2, 6, 128, 64, E4M3, "f32", "halves"),
    ([(5, 5), (0, 9), (33, 40), (0, 0)], 3, 3, 64, 16, E5M2, "bf16", "pairs"),
    ([(70, 200), (1, 33), (129, 129)], 2, 2, 128, 32, E4M3, "bf16", "halves"),
    ([(300, 301)], 1, 8, 256, 128, E4M3, "f32", "halves"),
    ([(64, 64), (63, 127), (65, 129)], 2, 4, 64, 64, E5M2, "f32", "pairs"),
    ([(2, 130)], 4, 4, 256, 64, E4M3, "bf16", None),
    ([(500, 500)], 2, 2, 64, 128, E5M2, "bf16", None),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_append_and_read(fa, case):
    seqs, H, Hq, D, bs, fmt, dt, rope = case
    rng = np.random.default_rng(len(seqs) * 100 + D + bs)
    new, lens = [n for n, _ in seqs], [m for _, m in seqs]
    T = sum(new)
    tables, nb = tables_for(rng, lens, bs)
    cache = filled_cache(fa, rng, nb, H, D, bs, fmt)
    k0, v0, kb0, vb0 = snapshot(cache)
    batch = fa.KVBatch.from_lists(new, lens, tables)
    # a fused product's rows: queries, keys, values side by side
    x = torch.from_numpy(rng.standard_normal((T, Hq + 2 * H, D)).astype(np.float32))
    x[:, Hq:Hq + H, ::7] *= 20
    x[: T // 3] *= 1e-3            # later tokens of a block may need a smaller bias
    if dt == "bf16":
        x = x.to(torch.bfloat16)
    xd = x.cuda()
    cs = rope_tables(max(lens) + 3, D) if rope else None
    say("append", seqs, H, Hq, D, bs, fmt, dt, rope)
    q = fa.kv_append(cache, batch, xd[:, Hq:Hq + H], xd[:, Hq + H:], q=xd[:, :Hq],
                     rope=None if cs is None else tuple(torch.from_numpy(t).cuda() for t in cs),
                     rope_pairs=rope == "pairs")
    torch.cuda.synchronize()
    xn = x.float().numpy()
    first, spans, pos = 0, [], []
    for n, m in seqs:
        spans.append((first, n, m))
        pos += list(range(m - n, m))
        first += n
    pos = np.array(pos, dtype=int)
    turn = (lambda t: t) if cs is None else (lambda t: ref.rotate(t, pos, *cs, rope == "pairs"))
    kr = turn(xn[:, Hq:Hq + H])
    ref.append(k0, kb0, kr, spans, tables, bs, fmt, False)
    ref.append(v0, vb0, xn[:, Hq + H:], spans, tables, bs, fmt, True)
    k1, v1, kb1, vb1 = snapshot(cache)
    assert np.array_equal(kb1, kb0) and np.array_equal(vb1, vb0)
    assert np.array_equal(k1, k0) and np.array_equal(v1, v0)
    assert torch.equal(q.cpu(), ref.bf16(turn(xn[:, :Hq])))
    # the same tokens again: nothing changes
    fa.kv_append(cache, batch, xd[:, Hq:Hq + H], xd[:, Hq + H:],
                 rope=None if cs is None else tuple(torch.from_numpy(t).cuda() for t in cs), rope_pairs=rope == "pairs")
    for a, b in zip(snapshot(cache), (k0, v0, kb0, vb0)):
        assert np.array_equal(a, b)
    # read back: the new tokens, then whole sequences
    for dtype in (torch.bfloat16, torch.float32):
        for cnt in (new, lens):
            b2 = fa.KVBatch.from_lists(cnt, lens, tables)
            kk, vv = fa.kv_read(cache, b2, dtype=dtype)
            at = 0
            for i, (n, m) in enumerate(zip(cnt, lens)):
                for got, codes, bias, values in ((kk, k0, kb0, False), (vv, v0, vb0, True)):
                    want = ref.gather(codes, bias, tables[i], m, bs, fmt, values)[m - n:]
                    g = got[at:at + n].cpu()
                    w = torch.from_numpy(want.astype(np.float32)).to(dtype)
                    assert torch.equal(g.isnan(), w.isnan())
                    assert torch.equal(g.nan_to_num(1.0), w.nan_to_num(1.0))
                at += n


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_values_that_move_the_scale(fa, fmt):
    """Zeros, infinities, NaN and tiny values; a block that grows token by
    token, whose scale falls and whose old tokens are coded again."""
    rng = np.random.default_rng(3)
    H, D, bs = 2, 64, 16
    tables = [[2, 0]]
    cache = fa.KVCache(3, H, D, block_size=bs, fmt=fmt)
    k0, v0, kb0, vb0 = snapshot(cache)
    rows = [np.zeros((H, D)), 1e-42 * np.ones((H, D)), rng.standard_normal((H, D)) * 1e-6, rng.standard_normal((H, D)),
            rng.standard_normal((H, D)) * 50, np.where(rng.random((H, D)) < 0.1, np.inf, rng.standard_normal((H, D))),
            np.where(rng.random((H, D)) < 0.1, np.nan, 1e4 * rng.standard_normal((H, D))), np.full((H, D), -np.inf),
            np.full((H, D), np.nan), rng.standard_normal((H, D)) * 3e38, rng.standard_normal((H, D)) * 1e-20]
    rows += [rng.standard_normal((H, D)) * 2.0 ** int(e) for e in rng.integers(-40, 40, 12)]
    for p, x in enumerate(rows):
        x = np.asarray(x).astype(np.float32)[None]
        xd = torch.from_numpy(x).cuda()
        batch = fa.KVBatch.from_lists([1], [p + 1], tables)
        fa.kv_append(cache, batch, xd, xd)
        ref.append(k0, kb0, x, [(0, 1, p + 1)], tables, bs, fmt, False)
        ref.append(v0, vb0, x, [(0, 1, p + 1)], tables, bs, fmt, True)
        for a, b, what in zip(snapshot(cache), (k0, v0, kb0, vb0), ("k", "v", "k_bias", "v_bias")):
            assert np.array_equal(a, b), (p, what)


def test_blocks_that_are_not_there(fa):
    """Table entries outside the cache are skipped by the write and read as
    zeros; lengths and counts past their bounds stay within the buffers."""
    rng = np.random.default_rng(8)
    H, D, bs = 2, 64, 16
    cache = filled_cache(fa, rng, 4, H, D, bs, E4M3)
    before = snapshot(cache)
    tables = [[1, -1, 99, 3]]
    batch = fa.KVBatch.from_lists([50], [50], tables)
    x = torch.from_numpy(rng.standard_normal((50, H, D)).astype(np.float32)).cuda()
    fa.kv_append(cache, batch, x, x)
    k0, v0, kb0, vb0 = before
    ref.append(k0, kb0, x.cpu().numpy(), [(0, 50, 50)], tables, bs, E4M3, False)
    ref.append(v0, vb0, x.cpu().numpy(), [(0, 50, 50)], tables, bs, E4M3, True)
    for a, b in zip(snapshot(cache), (k0, v0, kb0, vb0)):
        assert np.array_equal(a, b)
    k, v = fa.kv_read(cache, batch)
    assert (k[16:48] == 0).all() and (v[16:48] == 0).all() and (k[:16] != 0).any() and (k[48:] != 0).any()
    # device arrays that disagree with the host's bounds
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    wild = fa.KVBatch(i32([-5, 1 << 30]), i32([1 << 30]), i32(tables), max_new=50, max_len=64, tokens=50)
    k2, v2 = fa.kv_read(cache, wild)
    fa.kv_append(cache, wild, x, x)
    down = fa.KVBatch(i32([40, 3]), i32([-7]), i32(tables), max_new=50, max_len=64, tokens=50)
    fa.kv_append(cache, down, x, x)
    torch.cuda.synchronize()


def test_many_sequences(fa):
    """Hundreds of single tokens at once."""
    rng = np.random.default_rng(12)
    H, D, bs, B = 2, 128, 32, 301
    lens = [int(n) for n in rng.integers(1, 200, B)]
    tables, nb = tables_for(rng, lens, bs)
    cache = filled_cache(fa, rng, nb, H, D, bs, E4M3)
    k0, v0, kb0, vb0 = snapshot(cache)
    batch = fa.KVBatch.from_lists([1] * B, lens, tables)
    x = torch.from_numpy(rng.standard_normal((B, H, D)).astype(np.float32)).cuda()
    fa.kv_append(cache, batch, x, x)
    spans = [(i, 1, m) for i, m in enumerate(lens)]
    ref.append(k0, kb0, x.cpu().numpy(), spans, tables, bs, E4M3, False)
    ref.append(v0, vb0, x.cpu().numpy(), spans, tables, bs, E4M3, True)
    for a, b in zip(snapshot(cache), (k0, v0, kb0, vb0)):
        assert np.array_equal(a, b)


def test_nothing_to_do(fa):
    cache = fa.KVCache(2, 2, 64)
    for new, lens in (([], []), ([0], [0]), ([0, 0], [10, 3])):
        batch = fa.KVBatch.from_lists(new, lens, [[0]] * len(new))
        x = torch.empty(0, 2, 64, device="cuda")
        q = fa.kv_append(cache, batch, x, x, q=x)
        k, v = fa.kv_read(cache, batch)
        assert q.shape == k.shape == v.shape == (0, 2, 64)
