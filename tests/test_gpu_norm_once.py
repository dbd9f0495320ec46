"""A second derivative through the norm's autograd functions is refused: their
backward passes are kernels that autograd does not see into."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kind", ["norm", "norm and linear"])
def test_second_derivatives_are_refused(kind, residual):
    need_gpu()
    from fp8_precision_linear_amd import norm
    x = torch.randn(16, 128, device="cuda").requires_grad_()
    r = torch.randn(16, 128, device="cuda").requires_grad_() if residual else None
    if kind == "norm":
        w = torch.ones(128, device="cuda").requires_grad_()
        y = norm.RMSNormFunction.apply(x, r, w, 1e-5)
    else:
        y = norm.FP8NormLinear(128, 64, device="cuda")(x, r)
    y = y[0] if residual else y
    dx, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.square().sum().backward()
