"""Sequences whose lengths are rewritten around the autograd function."""
import pytest
import torch

import seq_ref
from gpu_util import need_gpu
from test_gpu_self_attention import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    need_gpu()
    from fp8_precision_linear_amd import self_attention
    return self_attention


def test_lengths_rewritten_before_the_backward_pass(sa):
    """The gradients would be other sequences': refused, as any saved tensor's
    rewriting is."""
    q, k, v, dout = (t.contiguous() for t in inputs([100], 2, 2, 64, 1))
    leaves = [t.requires_grad_() for t in (q, k, v)]
    cu = torch.tensor([0, 60, 100], dtype=torch.int32, device="cuda")
    seqs = sa.Sequences(cu, 100, 100, whole=True)
    out = sa.attention(*leaves, seqs)
    cu[1] = 30                                           # the next micro-batch's
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(dout)
    # as they are now they are right for the next pass
    for t in leaves:
        t.grad = None
    out = sa.attention(*leaves, seqs)
    out.backward(dout)
    o, lse = sa.attention_fwd(q.detach(), k.detach(), v.detach(), seqs)
    want = seq_ref.backward(dout, q.detach(), k.detach(), v.detach(), o, lse, [30, 70], 0.125)
    seq_ref.inside({n: t.grad for n, t in zip(("dq", "dk", "dv"), leaves)}, want, "rewritten")


def test_lengths_made_in_inference_mode(sa):
    """A plan made there has no versions, and trains all the same."""
    q, k, v, dout = (t.contiguous() for t in inputs([50], 2, 2, 64, 2))
    with torch.inference_mode():
        seqs = sa.Sequences.from_lists([30, 20])
    grads = []
    for s in (seqs, sa.Sequences.from_lists([30, 20])):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        sa.attention(*leaves, s).backward(dout)
        grads.append([t.grad for t in leaves])
    assert all(torch.equal(a, b) for a, b in zip(*grads))
