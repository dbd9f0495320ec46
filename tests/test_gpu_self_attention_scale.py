"""Attention over packed sequences at the ends of its scale: 0 makes every logit
of finite numbers 0, and 0 times NaN or infinity NaN."""
import pytest
import torch

import seq_ref
from gpu_util import need_gpu, say
from test_gpu_self_attention import inputs
from test_gpu_self_attention_edges import both, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    need_gpu()
    from fp8_precision_linear_amd import self_attention
    return self_attention


@pytest.mark.parametrize("heads", [(2, 2, 64), (4, 2, 128), (2, 1, 256)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("at", [0, 69, 70, 149])
def test_scale_of_zero(sa, heads, bad, at):
    say("scale 0", heads, bad, at)
    Hq, H, D = heads
    lens = [70, 80]
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, dout = inputs(lens, Hq, H, D, 40)
    clean = both(sa, q, k, v, dout, seqs, scale=0.0)
    q = q.clone()
    q[at, 1, D - 3] = bad
    out, lse, dq, dk, dv = both(sa, q, k, v, dout, seqs, scale=0.0)
    assert bool(out[at, 1].isnan().all()) and bool(lse[at, 1].isnan()) and bool(dq[at, 1].isnan().all())
    b, first = 1 // (Hq // H), 0 if at < 70 else 70
    seen = torch.zeros(150, dtype=torch.bool, device="cuda")
    seen[first:at + 1] = True
    assert bool(dk[seen, b].isnan().all()) and bool(dv[seen, b].isnan().all())
    for got, want in zip((out, lse, dq), clean):
        other = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
        other[at, 1] = False
        assert same((got[other],), (want[other],))
    for got, want in zip((dk, dv), clean[3:]):
        other = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
        other[seen, b] = False
        assert same((got[other],), (want[other],))


@pytest.mark.parametrize("scale", [2.0 ** 100, -2.0 ** 100, 2.0 ** -140])
def test_far_scales(sa, scale):
    """Logits of the usual size from keys that make up for the scale, and of none."""
    q, k, v, _ = inputs([90], 2, 2, 64, 41)
    k = (k.double() * 0.125 / abs(scale)).to(torch.bfloat16) if scale > 1 or scale < 0 else k
    out, lse = sa.attention_fwd(q, k, v, sa.Sequences.from_lists([90]), scale=scale)
    seq_ref.inside({"out": out, "lse": lse}, seq_ref.forward(q, k, v, [90], scale), f"scale {scale}")
