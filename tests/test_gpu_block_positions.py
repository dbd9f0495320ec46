"""Layers whose rotation table is shorter than their sequences."""
import pytest
import torch

from gpu_util import need_gpu
from test_gpu_block import D_MODEL, D, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import attention, block, decoder, self_attention
    return attention, block, decoder, self_attention


@pytest.mark.parametrize("qk_norm", [True, False])
def test_decoder_refuses_positions_past_its_table(mods, qk_norm):
    """With norms of queries and keys as without; the cache keeps what it has."""
    fa, block, dec, _ = mods
    m = make(block, qk_norm)
    layer = dec.FP8DecoderLayer.from_block(m.layers[0])
    cache, rope = layer.cache(1), dec.rope_tables(10, D)
    x = torch.randn(1, D_MODEL, device="cuda").to(torch.bfloat16)
    last = fa.KVBatch.from_lists([1], [10], [[0]])
    layer(x, None, cache, last, rope)                    # position 9, the table's last
    before = [t.clone() for t in (cache.k, cache.v)]
    past = fa.KVBatch.from_lists([1], [11], [[0]])
    for more in ({}, {"positions": past.positions()}):
        with pytest.raises(ValueError):
            layer(x, None, cache, past, rope, **more)
    assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
    model = dec.FP8Decoder([layer], m.head.norm_weight.detach(), 1, 10)
    with pytest.raises(ValueError):
        model(x, past)


def test_block_refuses_positions_past_its_table(mods):
    _, block, dec, sa = mods
    m = make(block)
    x = torch.randn(20, D_MODEL, device="cuda").to(torch.bfloat16)
    seqs = sa.Sequences.from_lists([7, 13])
    y = m.layers[0](x, None, seqs, dec.rope_tables(13, D))[0]
    for more in ({}, {"positions": seqs.positions()}):
        with pytest.raises(ValueError):
            m.layers[0](x, None, seqs, dec.rope_tables(12, D), **more)
    # a loose bound is none on the positions: no sequence is longer than all rows
    loose = sa.Sequences(seqs.cu_tokens, max_len=1 << 30, tokens=20)
    got = m.layers[0](x, None, loose, dec.rope_tables(20, D))[0]
    assert ((got.double() - y.double()).norm() / y.double().norm()).item() < 0.05
