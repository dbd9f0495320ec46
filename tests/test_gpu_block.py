"""The layer that trains, with every operator in it, against the same layer in
float64 from the definitions; and the served layer with the same weights.

Bound: as for the decoder layer (test_gpu_decoder.py).  Every product's operands
are rounded to E4M3 (2^-5 rms at the worst place of a binade) and gradients to
E5M2 (2^-4), independently, so a product's output is off by some 2.6% (4% with a
gradient) of its norm, and a gradient at the far end of the layer by a few of
these together: 10% of a result's norm is asked forward, 20% backward."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
VOCAB, D_MODEL, F, HQ, H, D = 300, 256, 384, 4, 2, 64
LENS = [90, 1, 38]


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import attention, block, decoder, self_attention
    return attention, block, decoder, self_attention


def make(block, qk_norm=True, layers=1):
    torch.manual_seed(4)
    m = block.FP8Model(VOCAB, layers, D_MODEL, F, HQ, H, D, 128, qk_norm=qk_norm, embed_scale=2.0, device="cuda")
    with torch.no_grad():
        for name, p in m.named_parameters():
            if p.dim() == 1:
                p.add_(0.1 * torch.randn_like(p))
            elif "embedding" not in name:
                p.copy_(torch.randn_like(p) * p.shape[1] ** -0.5)
            else:
                p.copy_(torch.randn_like(p) * 0.5)
    return m


def reference(w, ids, lens, qk_norm, layers, eps=1e-5):
    """Logits in float64, w: name -> float64 leaf."""
    norm = lambda t, g: t * (t.square().mean(-1, keepdim=True) + eps).rsqrt() * g  # noqa: E731
    h = w["embedding.weight"][ids] * 2.0
    pos = torch.cat([torch.arange(n) for n in lens]).cuda().double()
    inv = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    c, s = (f(pos[:, None] * inv)[:, None] for f in (torch.cos, torch.sin))
    turn = lambda t: torch.cat((t[..., :D // 2] * c - t[..., D // 2:] * s,  # noqa: E731
                                t[..., D // 2:] * c + t[..., :D // 2] * s), -1)
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)]).cuda()
    see = (seq[:, None] == seq[None]) & (pos[None] <= pos[:, None])
    for i in range(layers):
        p = lambda n: w[f"layers.{i}.{n}"]  # noqa: B023, E731
        qkv = (norm(h, p("attn_in.norm_weight")) @ p("attn_in.weight").t()).view(-1, HQ + 2 * H, D)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:]
        if qk_norm:
            q, k = norm(q, p("q_norm")), norm(k, p("k_norm"))
        q, k = turn(q), turn(k)
        k, v = (t.repeat_interleave(HQ // H, 1) for t in (k, v))
        heads = []
        for a in range(HQ):
            sc = (q[:, a] @ k[:, a].t() * D ** -0.5).masked_fill(~see, -torch.inf)
            heads.append(sc.softmax(1) @ v[:, a])
        h = h + torch.cat(heads, 1) @ p("attn_out.weight").t()
        g = norm(h, p("norm_mlp")) @ p("mlp.w1").t()
        g, u = g[:, :F], g[:, F:]
        h = h + (g * torch.sigmoid(g) * u) @ p("mlp.w2").t()
    return norm(h, w["head.norm_weight"]) @ w["head.weight"].t()


@pytest.mark.parametrize("qk_norm,layers", [(True, 1), (False, 1), (True, 2)])
def test_gradients(mods, qk_norm, layers):
    _, block, _, sa = mods
    m = make(block, qk_norm, layers)
    seqs = sa.Sequences.from_lists(LENS)
    ids = torch.randint(0, VOCAB, (seqs.tokens,), device="cuda")
    dout = torch.randn(seqs.tokens, VOCAB, device="cuda")
    logits = m(ids, seqs)
    logits.backward(dout)
    w = {n: p.detach().double().requires_grad_() for n, p in m.named_parameters()}
    want = reference(w, ids, LENS, qk_norm, layers)
    want.backward(dout.double())
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    assert rel(logits, want) < 0.1 * layers
    for n, p in m.named_parameters():
        assert rel(p.grad, w[n].grad) < 0.2 * layers, n


def test_served_layer_is_the_trained_one(mods):
    """Prompts, then single tokens, through the cache, against the packed pass:
    the same FP8 products; only the cache's rounding of keys and values lies
    between them (a fraction of the layer's own FP8 rounding)."""
    fa, block, dec, sa = mods
    m = make(block, layers=2)
    seqs = sa.Sequences.from_lists(LENS)
    ids = torch.randint(0, VOCAB, (seqs.tokens,), device="cuda")
    with torch.no_grad():
        pos = seqs.positions()
        x, h = m.embedding(ids), None
        for layer in m.layers:
            x, h = layer(x, h, seqs, m.rope, pos)
    from fp8_precision_linear_amd.norm import rmsnorm_fwd
    want = rmsnorm_fwd(x, m.head.norm_weight.detach(), residual=h)[0].double()
    served = dec.FP8Decoder([dec.FP8DecoderLayer.from_block(b) for b in m.layers], m.head.norm_weight.detach(), 8, 128,
                            embedding=m.embedding.weight.detach(), embed_scale=2.0)
    tables = [[0, 1], [2], [3]]
    first = [80, 0, 38]                 # the rest token by token
    rows = [torch.arange(n, device="cuda") + sum(LENS[:i]) for i, n in enumerate(LENS)]
    got = torch.zeros_like(want)
    done = [0, 0, 0]
    while done != LENS:
        new = [min(f if a == 0 and f else 1, n - a) for f, a, n in zip(first, done, LENS)]
        at = torch.cat([r[a:a + n] for r, a, n in zip(rows, done, new)])
        done = [a + n for a, n in zip(done, new)]
        got[at] = served(ids[at], fa.KVBatch.from_lists(new, done, tables)).double()
    assert ((got - want).norm() / want.norm()).item() < 0.1


def test_positions(mods):
    fa, _, _, sa = mods
    seqs = sa.Sequences.from_lists([3, 0, 2])
    assert seqs.positions().tolist() == [0, 1, 2, 0, 1]
    batch = fa.KVBatch.from_lists([2, 0, 1], [7, 3, 1], [[0], [1], [2]])
    assert batch.positions().tolist() == [5, 6, 0]
    batch.lens.add_(1)      # from what the arrays hold now
    assert batch.positions().tolist() == [6, 7, 1]
    assert sa.Sequences.from_lists([]).positions().tolist() == []


def test_ids_need_an_embedding(mods):
    fa, block, dec, _ = mods
    m = make(block)
    served = dec.FP8Decoder([dec.FP8DecoderLayer.from_block(m.layers[0])], m.head.norm_weight.detach(), 2, 64)
    with pytest.raises(ValueError):
        served(torch.zeros(1, dtype=torch.int64, device="cuda"), fa.KVBatch.from_lists([1], [1], [[0]]))
    with pytest.raises(ValueError):
        m(torch.zeros(200, dtype=torch.int64, device="cuda"), mods[3].Sequences.from_lists([200]))


def test_command(mods, capsys):
    mods[1].main(["--layers", "1", "--sequences", "2", "--length", "130", "--steps", "2"])
    assert "ms a step" in capsys.readouterr().out
