"""Attention over packed sequences and its gradients against their 64-bit forms
(seq_ref.py has the bounds)."""
import pytest
import torch

import seq_ref
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    need_gpu()
    from fp8_precision_linear_amd import self_attention
    return self_attention


def inputs(lens, Hq, H, D, seed, std=1.0):
    """Fused rows, their views q, k, v, and dout."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    x = (torch.randn(T, Hq + 2 * H, D, generator=g, device="cuda") * std).to(torch.bfloat16)
    dout = torch.randn(T, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], dout


def check(sa, lens, Hq, H, D, causal=True, window=0, scale=None, seed=0, std=1.0):
    what = f"lens {lens} heads {Hq}/{H} of {D} causal {causal} window {window} scale {scale}"
    say(what)
    q, k, v, dout = inputs(lens, Hq, H, D, seed, std)
    seqs = sa.Sequences.from_lists(lens)
    s = D ** -0.5 if scale is None else scale
    out, lse = sa.attention_fwd(q, k, v, seqs, scale=scale, causal=causal, window=window)
    seq_ref.inside({"out": out, "lse": lse}, seq_ref.forward(q, k, v, lens, s, causal, window), what)
    dq, dk, dv = sa.attention_bwd(dout, q, k, v, out, lse, seqs, scale=scale, causal=causal, window=window)
    want = seq_ref.backward(dout, q, k, v, out, lse, lens, s, causal, window)
    seq_ref.inside({"dq": dq, "dk": dk, "dv": dv}, want, what)


HEADS = [(2, 2, 64), (4, 2, 128), (4, 1, 256), (16, 1, 64), (3, 3, 128)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", [[1], [31, 0, 33, 1], [128], [129, 64, 0, 1, 200], [513]])
def test_causal(sa, heads, lens):
    check(sa, lens, *heads)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", [[1, 2], [65, 0, 127], [300]])
def test_everything_seen(sa, heads, lens):
    check(sa, lens, *heads, causal=False)


@pytest.mark.parametrize("heads", HEADS[:3])
@pytest.mark.parametrize("window", [1, 31, 64, 100, 1 << 31, 1 << 40])
def test_window(sa, heads, window):
    check(sa, [200, 3, 333], *heads, window=window)


@pytest.mark.parametrize("scale", [0.3, -0.1, 0.0])
def test_scales(sa, scale):
    check(sa, [150, 20], 4, 2, 64, scale=scale)
    check(sa, [150, 20], 4, 2, 128, scale=scale, causal=False)


@pytest.mark.parametrize("heads", [(8, 1, 128), (2, 2, 64), (8, 2, 256)])
def test_long(sa, heads):
    """Many tiles, and walks over the queries that are cut into chunks."""
    check(sa, [1500, 700], *heads)


def test_running_maximum_moves(sa):
    """Logits that grow along the keys, by far more than one tile's step."""
    check(sa, [400], 2, 2, 128, std=3.0)
    q, k, v, dout = inputs([600], 2, 2, 64, 5)
    k = (k * torch.linspace(0.1, 6, 600, device="cuda")[:, None, None]).to(torch.bfloat16)
    seqs = sa.Sequences.from_lists([600])
    out, lse = sa.attention_fwd(q, k, v, seqs)
    seq_ref.inside({"out": out, "lse": lse}, seq_ref.forward(q, k, v, [600], 0.125), "growing logits")
    got = dict(zip(("dq", "dk", "dv"), sa.attention_bwd(dout, q, k, v, out, lse, seqs)))
    seq_ref.inside(got, seq_ref.backward(dout, q, k, v, out, lse, [600], 0.125), "growing logits")
