"""fp8_kv_attention against its definition in 64 bits.

Bound for one output: its bf16 rounding, 2^-8 of the value, and
sum_j p_j |v_j| times
  2^-11            the probability's fp16 rounding
  B * 2^-19        the logit's error: sums of up to 256 fp32 products of
                   magnitude B = scale * max_j sum_d |q_d k_jd| in all
  2^-18            exp2, the sum of the probabilities, the joins
plus what fp16 loses below its normal range, 2^-30 of the largest value a key.
lse: B * 2^-19 + 2^-18 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu, say
from test_gpu_kv_cache import tables_for

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1
NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def fa():
    need_gpu()
    from fp8_precision_linear_amd import attention
    return attention


def build(fa, rng, lens, H, D, bs, fmt, spread=2, spare=2):
    """A cache of normal values whose unused slots hold NaN codes."""
    tables, nb = tables_for(rng, lens, bs, spare)
    cache = fa.KVCache(nb, H, D, block_size=bs, fmt=fmt)
    k = ref.encode_fp8(rng.standard_normal((nb, H, bs, D)) * ref.FMT_MAX[fmt] / 5, fmt)
    v = ref.encode_fp8(rng.standard_normal((nb, H, D, bs)) * ref.FMT_MAX[fmt] / 5, fmt)
    e = ref.EMAX[fmt] - 1
    kb = rng.integers(e - spread, e + 1, (nb, H)).astype(np.int32)
    vb = rng.integers(e - spread, e + 1, (nb, H)).astype(np.int32)
    used = np.zeros((nb, bs), bool)
    for t, n in zip(tables, lens):
        for p in range(n):
            used[t[p // bs], p % bs] = True
    k = np.where(used[:, None, :, None], k, NAN_CODE).astype(np.uint8)
    v = np.where(used[:, None, None, :], v, NAN_CODE).astype(np.uint8)
    store(cache, k, v, kb, vb)
    return cache, tables, k, v, kb, vb


def store(cache, k, v, kb, vb):
    for t, a in ((cache.k, k), (cache.v, v), (cache.k_bias, kb), (cache.v_bias, vb)):
        t.copy_(torch.from_numpy(a))


def check(out, lse, q, cu, new, lens, tables, k, v, kb, vb, bs, fmt, scale, causal, window, what):
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    q = q.cpu().double().numpy()
    for i, (n, m) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        kk = ref.gather(k, kb, tables[i], m, bs, fmt, False)
        vv = ref.gather(v, vb, tables[i], m, bs, fmt, True)
        o, s, mag, big = ref.attend(q[cu[i]:cu[i] + n], kk, vv, np.arange(m - n, m), scale, causal, window)
        got, gl = out[cu[i]:cu[i] + n], lse[cu[i]:cu[i] + n]
        top = np.abs(np.nan_to_num(vv)).max() if m else 0.0
        bound = 2.0 ** -8 * np.abs(o) + mag * (2.0 ** -11 + big[..., None] * 2.0 ** -19 + 2.0 ** -18) + m * 2.0 ** -30 * top
        bad = np.isnan(o)
        assert np.array_equal(np.isnan(got), bad), (what, i, "NaN")
        err = np.abs(np.where(bad, 0, got - np.where(bad, 0, o)))
        assert np.all(err <= np.where(bad, 0, bound) + 1e-30), (what, i, float(np.nanmax(err / (bound + 1e-30))))
        gone = np.isneginf(s)
        assert np.array_equal(np.isneginf(gl), gone), (what, i, "lse")
        ok = ~gone & ~np.isnan(s)
        assert np.all(np.abs(gl - s)[ok] <= (big * 2.0 ** -19 + 2.0 ** -18 * (1 + np.abs(s)))[ok]), (what, i, "lse")


def run(fa, seed, seqs, H, Hq, D, bs, fmt, causal=True, window=0, scale=None, spread=2, change=None, qscale=1.0):
    rng = np.random.default_rng(seed)
    new, lens = [n for n, _ in seqs], [m for _, m in seqs]
    cache, tables, k, v, kb, vb = build(fa, rng, lens, H, D, bs, fmt, spread)
    if change:
        change(rng, tables, k, v, kb, vb)
        store(cache, k, v, kb, vb)
    batch = fa.KVBatch.from_lists(new, lens, tables)
    T = sum(new)
    q = torch.from_numpy(rng.standard_normal((T, Hq + 1, D)).astype(np.float32) * qscale).to(torch.bfloat16).cuda()[:, :Hq]
    say("attention", seqs, H, Hq, D, bs, fmt, causal, window)
    out, lse = fa.kv_attention(cache, batch, q, causal=causal, window=window, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    cu = np.cumsum([0] + new)
    check(out, lse, q, cu, new, lens, tables, k, v, kb, vb, bs, fmt, D ** -0.5 if scale is None else scale, causal,
          window, (seqs, H, Hq, D, bs, fmt, causal, window))
    again = fa.kv_attention(cache, batch, q, causal=causal, window=window, scale=scale, return_lse=True)
    assert torch.equal(again[0].view(torch.int16), out.view(torch.int16)), "same inputs, same bits"
    assert torch.equal(again[1].view(torch.int32), lse.view(torch.int32))
    return out, lse


# single tokens and short drafts: every length around the tiles and blocks
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_single_tokens(fa, D, bs):
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 257, 320, 700]
    run(fa, D + bs, [(1, n) for n in lens], 2, 8, D, bs, E4M3 if bs < 64 else E5M2)


@pytest.mark.parametrize("H,Hq", [(1, 1), (3, 3), (1, 16), (1, 17), (2, 6), (1, 40), (4, 128)])
def test_head_layouts(fa, H, Hq):
    run(fa, H * 50 + Hq, [(1, 100), (1, 333), (1, 1)], H, Hq, 128, 64, E4M3)


@pytest.mark.parametrize("n", [2, 3, 4, 8, 16, 33])
def test_drafts(fa, n):
    run(fa, n, [(n, n), (n, n + 70), (1, 300), (max(1, n - 1), 128)], 2, 8, 64, 32, E5M2)


# prompts: whole, on top of a past, ragged, rows past the last tile
@pytest.mark.parametrize("D,bs,fmt", [(64, 16, E4M3), (128, 64, E4M3), (128, 32, E5M2), (256, 128, E4M3), (64, 128, E5M2)])
def test_prompts(fa, D, bs, fmt):
    run(fa, D + bs, [(130, 130), (40, 200), (1, 77), (0, 50), (65, 65), (0, 0)], 2, 4, D, bs, fmt)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1000])
def test_window(fa, window):
    run(fa, window, [(1, 300), (1, 64), (3, 129), (1, 1)], 2, 4, 64, 32, E4M3, window=window)
    run(fa, window, [(90, 300), (70, 70)], 1, 4, 128, 64, E4M3, window=window)


def test_not_causal(fa):
    run(fa, 1, [(5, 40), (1, 100), (3, 3)], 2, 4, 64, 16, E4M3, causal=False)
    run(fa, 2, [(150, 170), (70, 300)], 1, 2, 128, 64, E4M3, causal=False)


def test_long_splits(fa):
    """One long sequence beside short ones: the split and its join."""
    run(fa, 5, [(1, 5000), (1, 3), (1, 700)], 1, 4, 128, 64, E4M3)
    run(fa, 6, [(2, 4100), (2, 2)], 2, 4, 64, 16, E5M2)
    run(fa, 7, [(40, 3000), (1, 2)], 1, 4, 64, 64, E4M3)
    run(fa, 8, [(1, 5000), (1, 300)], 1, 4, 64, 64, E4M3, window=777)


def test_scales_far_apart(fa):
    """Blocks whose values differ by up to 2^20, in both orders, and keys too;
    large logits (a nearly one-hot softmax) and a scale of zero."""
    def rising(rng, tables, k, v, kb, vb):
        for t in tables:
            for j, b in enumerate(t):
                vb[b] = 20 - 4 * j if j < 6 else 0
    def falling(rng, tables, k, v, kb, vb):
        for t in tables:
            for j, b in enumerate(t):
                vb[b] = -4 + 4 * min(j, 6)
                kb[b] = 7 + (j % 3)
    for change in (rising, falling):
        run(fa, 11, [(1, 400), (1, 100)], 2, 4, 64, 64, E4M3, change=change)
        run(fa, 12, [(80, 400), (60, 100)], 1, 2, 128, 64, E4M3, change=change)
        run(fa, 13, [(1, 400), (20, 390)], 1, 2, 128, 16, E5M2, change=change)
    run(fa, 14, [(1, 500), (3, 70)], 2, 4, 128, 64, E4M3, qscale=30.0)
    run(fa, 15, [(100, 500)], 1, 2, 64, 64, E4M3, qscale=30.0)
    run(fa, 16, [(100, 130), (1, 64)], 1, 2, 64, 64, E4M3, scale=0.0)


def test_blocks_of_zeros(fa):
    """A block of zeros has bias 126; its tokens still count in the softmax."""
    def zero(rng, tables, k, v, kb, vb):
        b = tables[0][1]
        k[b], v[b] = 0, 0
        kb[b], vb[b] = 126, 126
    run(fa, 21, [(1, 200)], 1, 2, 128, 64, E4M3, change=zero)
    run(fa, 22, [(70, 200)], 1, 2, 64, 16, E4M3, change=zero)
    def all_zero(rng, tables, k, v, kb, vb):
        v[:], vb[:] = 0, 126
    run(fa, 23, [(1, 200), (50, 60)], 1, 2, 64, 64, E4M3, change=all_zero)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_nan_values_reach_only_those_who_see_them(fa, fmt):
    """NaN in a value that some queries see and others do not (a later token
    of the same call; one that left the window)."""
    def nan_at(positions, seq=0):
        def change(rng, tables, k, v, kb, vb):
            bs = k.shape[2]
            for p in positions:
                v[tables[seq][p // bs], :, 5::9, p % bs] = NAN_CODE
        return change
    run(fa, 31, [(4, 70)], 1, 4, 64, 16, fmt, change=nan_at([67]))
    run(fa, 32, [(100, 150)], 1, 4, 64, 64, fmt, change=nan_at([90, 149]))
    run(fa, 33, [(100, 150)], 1, 2, 128, 64, fmt, window=20, change=nan_at([30, 90]))
    run(fa, 34, [(3, 150)], 1, 2, 128, 64, fmt, window=20, change=nan_at([10, 129]))


def test_missing_blocks_are_not_seen(fa):
    rng = np.random.default_rng(2)
    H, Hq, D, bs = 1, 2, 64, 32
    lens = [100]
    cache, tables, k, v, kb, vb = build(fa, rng, lens, H, D, bs, E4M3)
    gone = [list(tables[0])]
    gone[0][1] = -1
    for new in (1, 60):
        batch = fa.KVBatch.from_lists([new], lens, gone)
        q = torch.from_numpy(rng.standard_normal((new, Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
        out, lse = fa.kv_attention(cache, batch, q, return_lse=True)
        kk = ref.gather(k, kb, tables[0], 100, bs, E4M3, False)
        vv = ref.gather(v, vb, tables[0], 100, bs, E4M3, True)
        keep = np.r_[0:32, 64:100]
        pos = np.arange(100 - new, 100)
        for t in range(new):
            see = keep[keep <= pos[t]]
            o, s, mag, big = ref.attend(q[t:t + 1].cpu().double().numpy(), kk[see], vv[see], [10 ** 6], D ** -0.5, True, 0)
            assert np.all(np.abs(out[t].cpu().double().numpy() - o[0]) <= 2.0 ** -8 * np.abs(o[0]) + mag[0] * 2.0 ** -10)
            assert np.all(np.abs(lse[t].cpu().double().numpy() - s[0]) <= 1e-4)
    # no block at all: nothing is seen
    batch = fa.KVBatch.from_lists([2], [40], [[-1, 77]])
    out, lse = fa.kv_attention(cache, batch, q[:2], return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_offsets_past_32_bits(fa):
    """A cache of more than 2^32 code bytes: blocks at both ends of it."""
    H, D, bs = 8, 128, 64
    nb = (1 << 32) // (H * D * bs) + 70
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    rng = np.random.default_rng(9)
    cache = fa.KVCache(nb, H, D, block_size=bs)
    tables, lens = [[nb - 1, 0, nb - 3]], [150]
    x = torch.from_numpy(rng.standard_normal((150, 2 * H, D)).astype(np.float32)).cuda()
    batch = fa.KVBatch.from_lists(lens, lens, tables)
    fa.kv_append(cache, batch, x[:, :H], x[:, H:])
    k, v = fa.kv_read(cache, batch, dtype=torch.float32)
    for got, want in ((k, x[:, :H]), (v, x[:, H:])):
        # half a step of E4M3 at the scale of the block: 2^-4 of the value, or of
        # the smallest normal at the bias of a block whose maximum is about 4
        assert ((got - want).abs() <= 2 ** -4 * want.abs() + 2.0 ** -10 * 2.0 ** -5).all()
    q = x[-2:, :H].to(torch.bfloat16)
    b2 = fa.KVBatch.from_lists([2], lens, tables)
    out = fa.kv_attention(cache, b2, q)
    kk, vv = (t.cpu().double().numpy() for t in (k, v))
    o, s, mag, big = ref.attend(q.cpu().double().numpy(), kk, vv, [148, 149], D ** -0.5, True, 0)
    assert np.all(np.abs(out.cpu().double().numpy() - o) <= 2.0 ** -8 * np.abs(o) + mag * 2.0 ** -10)


def test_other_stream_workspace_and_graph(fa):
    rng = np.random.default_rng(77)
    lens = [3000, 500]
    cache, tables, *_ = build(fa, rng, lens, 2, 64, 64, E4M3)
    batch = fa.KVBatch.from_lists([1, 1], lens, tables)
    q = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    want, wl = fa.kv_attention(cache, batch, q, return_lse=True)
    ws = fa.attention_workspace(cache, batch, 8)
    assert ws is not None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, gl = fa.kv_attention(cache, batch, q, return_lse=True, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(gl, wl)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.kv_attention(cache, batch, q, out=out, lse=lse, workspace=ws)
    for _ in range(3):
        q.copy_(torch.randn(2, 8, 64, device="cuda"))
        batch.lens.copy_(torch.randint(1, 500, (2,), device="cuda"))   # lengths are the device's
        g.replay()
        torch.cuda.synchronize()
        want, wl = fa.kv_attention(cache, batch, q, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("n,H,Hq", [(3, 2, 4), (90, 1, 2)])
def test_one_visible_key_takes_all_whatever_its_logit(fa, n, H, Hq):
    """A window of one: out is the token's own value, also where the only logit
    is some -1e33.  Bound: the probability is 1, so the value's bf16 rounding and
    the few fp32 steps are all that is left."""
    D, bs, fmt = 64, 32, E4M3
    rng = np.random.default_rng(n)
    cache, tables, k, v, kb, vb = build(fa, rng, [n], H, D, bs, fmt)
    q = torch.from_numpy(rng.standard_normal((n, Hq, D)).astype(np.float32) * 2.0 ** 110).to(torch.bfloat16).cuda()
    say("one key", n, H, Hq)
    out, lse = fa.kv_attention(cache, fa.KVBatch.from_lists([n], [n], tables), q, window=1, scale=1.0, return_lse=True)
    own = ref.gather(v, vb, tables[0], n, bs, fmt, True)
    keys = ref.gather(k, kb, tables[0], n, bs, fmt, False)
    qd, got, lse = q.cpu().double().numpy(), out.cpu().double().numpy(), lse.cpu().double().numpy()
    low = 0
    for h in range(Hq):
        g = h * H // Hq
        want = own[:, g] if own.shape[0] == n else own[g]
        key = keys[:, g] if keys.shape[0] == n else keys[g]
        assert np.all(np.abs(got[:, h] - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18)), h
        s = (qd[:, h] * key).sum(-1)
        assert np.all(np.abs(lse[:, h] - s) <= 2.0 ** -17 * np.abs(qd[:, h] * key).sum(-1)), h
        low += int((s < -1e32).sum())
    assert low > 0
