"""The outputs of the autograd function of the head norms, changed in place."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    need_gpu()
    from fp8_precision_linear_amd import qk_norm
    return qk_norm


def test_head_norms_in_place(qn):
    """Outputs are tensors of their own to autograd: one may be scaled in place."""
    T, Hq, H, D = 9, 4, 2, 64
    x, w = torch.randn(T, Hq + 2 * H, D, device="cuda"), torch.ones(D, device="cuda")
    dy = [torch.randn(T, n, D, device="cuda").to(torch.bfloat16) for n in (Hq, H, H)]
    grads = []
    for in_place in (False, True):
        leaves = [t.clone().requires_grad_() for t in (x, w, w)]
        q, k, v = qn.qk_norm_rope(leaves[0], Hq, H, *leaves[1:])
        if in_place:
            q.mul_(0.5)
            v.neg_()
        else:
            q, v = q * 0.5, -v
        torch.autograd.backward((q, k, v), dy)
        grads.append([q.detach(), k.detach(), v.detach(), *(t.grad for t in leaves)])
    assert all(torch.equal(a, b) for a, b in zip(*grads))
