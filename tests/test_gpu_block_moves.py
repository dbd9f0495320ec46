"""A model that is built on the host and moved."""
import pytest
import torch

from gpu_util import need_gpu
from test_gpu_block import D_MODEL, F, H, HQ, VOCAB, D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import block, self_attention
    return block, self_attention


def test_model_moves_with_its_table(mods):
    """Built on the host, then moved: the table is where the weights are, and
    stays float32."""
    block, sa = mods
    torch.manual_seed(5)
    m = block.FP8Model(VOCAB, 1, D_MODEL, F, HQ, H, D, 64)
    table = [t.clone() for t in m.rope]
    names = list(m.state_dict())
    m = m.to("cuda")
    assert all(t.is_cuda and t.dtype == torch.float32 for t in m.rope)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(m.rope, table))
    assert names == list(m.state_dict())
    logits = m(torch.randint(0, VOCAB, (30,), device="cuda"), sa.Sequences.from_lists([20, 10]))
    logits.sum().backward()
    assert bool(logits.isfinite().all()) and all(p.grad is not None for p in m.parameters())
    assert all(t.dtype == torch.float32 for t in m.to(torch.bfloat16).rope)
    # without contents, then with: the tables are made (each a rounding of the same number in 64 bits: a step of 2^-24)
    m = block.FP8Model(VOCAB, 1, D_MODEL, F, HQ, H, D, 64, device="meta").to_empty(device="cuda")
    assert all((a.cpu() - b).abs().max().item() <= 2.0 ** -24 for a, b in zip(m.rope, table))
