"""What block.FP8Block trained is what decoder.FP8DecoderLayer serves: its window
among the rest (test_gpu_block.py has the model, the sizes and the bound of 10%)."""
import pytest
import torch

from gpu_util import need_gpu
from test_gpu_block import D_MODEL, F, H, HQ, LENS, VOCAB, D, make

pytestmark = pytest.mark.gpu
WINDOW = 6


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import attention, block, decoder, self_attention
    return attention, block, decoder, self_attention


def packed(m, seqs, ids):
    """Final hidden states of the layers run on packed sequences."""
    from fp8_precision_linear_amd.norm import rmsnorm_fwd
    with torch.no_grad():
        x, h = m.embedding(ids), None
        for layer in m.layers:
            x, h = layer(x, h, seqs, m.rope)
        return rmsnorm_fwd(x, m.head.norm_weight.detach(), residual=h)[0].double()


def served(mods, m, ids):
    """The same through the cache: prompts of half a sequence, then single tokens."""
    fa, _, dec, _ = mods
    model = dec.FP8Decoder([dec.FP8DecoderLayer.from_block(b) for b in m.layers], m.head.norm_weight.detach(), 8, 128,
                           embedding=m.embedding.weight.detach(), embed_scale=2.0)
    rows = [torch.arange(n, device="cuda") + sum(LENS[:i]) for i, n in enumerate(LENS)]
    got = torch.zeros(sum(LENS), D_MODEL, dtype=torch.float64, device="cuda")
    done = [0] * len(LENS)
    while done != LENS:
        new = [min(n // 2 if a == 0 and n > 1 else 1, n - a) for a, n in zip(done, LENS)]
        at = torch.cat([r[a:a + n] for r, a, n in zip(rows, done, new)])
        done = [a + n for a, n in zip(done, new)]
        got[at] = model(ids[at], fa.KVBatch.from_lists(new, done, [[0, 1], [2], [3]])).double()
    return got


def rel(a, b):
    return ((a - b).norm() / b.norm()).item()


@pytest.mark.parametrize("qk_norm", [True, False])
def test_window_is_served(mods, qk_norm):
    m = make(mods[1], qk_norm, layers=2)
    seqs = mods[3].Sequences.from_lists(LENS)
    ids = torch.randint(0, VOCAB, (seqs.tokens,), device="cuda")
    full = packed(m, seqs, ids)
    for layer in m.layers:
        layer.window = WINDOW
    want = packed(m, seqs, ids)
    assert rel(full, want) > 0.2      # (so that the next line tells the two apart)
    assert rel(served(mods, m, ids), want) < 0.1
    # a call's own window goes before the layer's
    one = mods[2].FP8DecoderLayer.from_block(m.layers[0])
    x = torch.randn(40, D_MODEL, device="cuda").to(torch.bfloat16)
    batch = mods[0].KVBatch.from_lists([40], [40], [[0]])
    out = {w: one(x, None, one.cache(1), batch, m.rope, **({} if w is None else {"window": w}))[0] for w in (None, WINDOW, 0)}
    assert torch.equal(out[None], out[WINDOW]) and not torch.equal(out[None], out[0])


def test_model_takes_a_window(mods):
    m = make(mods[1], layers=2)
    w = mods[1].FP8Model(VOCAB, 2, D_MODEL, F, HQ, H, D, 128, embed_scale=2.0, window=WINDOW, device="cuda")
    w.load_state_dict(m.state_dict())
    assert [b.window for b in w.layers] == [WINDOW] * 2
    seqs = mods[3].Sequences.from_lists(LENS)
    ids = torch.randint(0, VOCAB, (seqs.tokens,), device="cuda")
    for layer in m.layers:
        layer.window = WINDOW
    with torch.no_grad():
        assert torch.equal(m(ids, seqs), w(ids, seqs))
