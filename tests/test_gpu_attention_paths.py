"""Paths of fp8_kv_attention that only long or many sequences take, against the
64-bit form with test_gpu_attention's bound: chunks of more than 64 tiles, more
than 64 sequences that share the workgroups, joins of few and of many parts, a
negative scale."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu, say
from test_gpu_attention import build, check, run

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    from fp8_precision_linear_amd import attention
    return attention


def heads_of(codes, bias, table, n, bs, fmt, values, h):
    """[n, D] float64 of one head of a sequence."""
    at = np.arange(n)
    blk = np.array(table)[at // bs]
    c = codes[blk, h, :, at % bs] if values else codes[blk, h, at % bs]
    return ref.code_values(fmt)[c] * 2.0 ** -bias[blk, h].astype(np.float64)[:, None]


@pytest.mark.parametrize("new,length,H,Hq,D,bs,window", [
    (512, 9000, 4, 64, 64, 64, 0),      # two chunks of 71 tiles
    (512, 9000, 4, 64, 64, 16, 0),
    (1024, 4097, 4, 64, 64, 64, 0),     # one of 65
    (1024, 4097, 4, 64, 64, 16, 0),
    (1024, 8300, 4, 64, 128, 128, 0),   # 64 + 64 + 2
    (1024, 8300, 4, 64, 64, 32, 5000),
])
def test_chunks_of_many_tiles(fa, new, length, H, Hq, D, bs, window):
    rng = np.random.default_rng(length + bs)
    cache, tables, k, v, kb, vb = build(fa, rng, [length], H, D, bs, E4M3)
    q = torch.from_numpy(rng.standard_normal((new, Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    say("chunks of many tiles", new, length, H, Hq, D, bs, window)
    out, lse = fa.kv_attention(cache, fa.KVBatch.from_lists([new], [length], tables), q, window=window, return_lse=True)
    qn, out, lse = (t.cpu().double().numpy() for t in (q, out, lse))
    picks = [(0, 0), (new - 1, Hq - 1)] + [(int(rng.integers(new)), int(rng.integers(Hq))) for _ in range(38)]
    for t, a in picks:
        h = a * H // Hq
        kk, vv = (heads_of(c, b, tables[0], length, bs, E4M3, x, h)[:, None] for c, b, x in ((k, kb, False), (v, vb, True)))
        o, s, mag, big = ref.attend(qn[t:t + 1, a:a + 1], kk, vv, [length - new + t], D ** -0.5, True, window)
        bound = 2.0 ** -8 * np.abs(o) + mag * (2.0 ** -11 + big[..., None] * 2.0 ** -19 + 2.0 ** -18) \
            + length * 2.0 ** -30 * np.abs(vv).max()
        assert np.all(np.abs(out[t, a] - o[0, 0]) <= bound[0, 0]), (t, a)
        assert abs(lse[t, a] - s[0, 0]) <= big[0, 0] * 2.0 ** -19 + 2.0 ** -18 * (1 + abs(s[0, 0])), (t, a)


@pytest.mark.parametrize("count,longest", [(65, 1700), (65, 20000), (130, 2000), (200, 1600)])
@pytest.mark.parametrize("H,Hq,D,bs", [(2, 8, 64, 64), (1, 3, 128, 16)])
def test_many_sequences(fa, count, longest, H, Hq, D, bs):
    """Ragged single tokens, some sequences without one, one much longer, first
    or last or between."""
    rng = np.random.default_rng(count + longest + D)
    lens = [int(n) for n in rng.integers(1, 1500, count)]
    new = [int(n) for n in rng.random(count) > 0.15]
    at = (0, count - 1, count // 2)[(count + D) % 3]
    lens[at], new[at] = longest, 1
    run(fa, count + D, list(zip(new, lens)), H, Hq, D, bs, E4M3)


def test_two_row_blocks_of_many_sequences(fa):
    run(fa, 3, [(2, 100 + 40 * i) for i in range(70)], 1, 16, 128, 64, E5M2)
    run(fa, 4, [(2, 100 + 40 * i) for i in range(40)], 1, 16, 256, 64, E4M3)


def test_join_of_many_chunks(fa):
    """More than 16 chunks of the kernel of many rows."""
    run(fa, 5, [(40, 5000), (3, 5), (1, 4000)], 1, 2, 64, 64, E4M3)
    run(fa, 6, [(34, 4500)], 1, 1, 256, 16, E5M2)


@pytest.mark.parametrize("seqs,H,Hq,D,bs", [([(1, 300), (3, 65)], 2, 4, 64, 32), ([(100, 250), (1, 64)], 1, 2, 128, 64),
                                            ([(1, 2000)], 1, 4, 64, 64)])
def test_negative_scale(fa, seqs, H, Hq, D, bs):
    """The same as the negated queries at the positive scale."""
    rng = np.random.default_rng(H + D)
    new, lens = [n for n, _ in seqs], [m for _, m in seqs]
    cache, tables, k, v, kb, vb = build(fa, rng, lens, H, D, bs, E4M3)
    batch = fa.KVBatch.from_lists(new, lens, tables)
    q = torch.from_numpy(rng.standard_normal((sum(new), Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    say("negative scale", seqs)
    out, lse = fa.kv_attention(cache, batch, q, scale=-0.2, return_lse=True)
    check(out, lse, -q, np.cumsum([0] + new), new, lens, tables, k, v, kb, vb, bs, E4M3, 0.2, True, 0, seqs)
