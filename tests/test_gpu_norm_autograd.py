"""The norm's autograd functions: what the backward pass reads is held by
autograd, so a change of it in between is refused and nothing outlives its
graph; gradients with and without a residual and accumulated into weight.grad."""
import gc
import weakref

import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import norm
    import fp8_precision_linear_amd as fl
    return fl, norm


def tensors(seed, rows=48, d=256):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, d, generator=g).cuda()
    r = torch.randn(rows, d, generator=g).to(torch.bfloat16).cuda()
    return x.requires_grad_(), r.requires_grad_()


def layer_of(norm, seed=0, d=256, out=128):
    torch.manual_seed(seed)
    layer = norm.FP8NormLinear(d, out, eps=EPS, device="cuda")
    with torch.no_grad():
        layer.norm_weight.add_(0.1 * torch.randn(d, device="cuda"))
    return layer


def test_changed_residual_stream_is_refused(mods):
    _, norm = mods
    x, r = tensors(1)
    y, h = layer_of(norm)(x, r)
    h.add_(1.0)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_changed_input_is_refused(mods):
    _, norm = mods
    x, _ = tensors(2)
    z = x * 2.0
    y = layer_of(norm)(z)
    z.mul_(3.0)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_changed_norm_weight_is_refused(mods):
    _, norm = mods
    x, r = tensors(3)
    layer = layer_of(norm)
    y, _ = layer(x, r)
    with torch.no_grad():
        layer.norm_weight.mul_(2.0)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


@pytest.mark.parametrize("residual", [False, True])
def test_a_dropped_graph_frees_its_tensors(mods, residual):
    _, norm = mods
    layer = layer_of(norm)
    x, r = tensors(4, rows=4096)
    x = x.detach()
    layer(x, r if residual else None)   # workspaces
    gc.collect()
    gc.disable()
    try:
        before = torch.cuda.memory_allocated()
        out = layer(x, r if residual else None)
        kept = weakref.ref(out[1] if residual else out)
        del out
        assert kept() is None and torch.cuda.memory_allocated() == before
    finally:
        gc.enable()


@pytest.mark.parametrize("residual", [False, True])
def test_gradients(mods, residual):
    """Bit for bit those of the calls the layer stands for."""
    fl, norm = mods
    x, r = tensors(5)
    layer = layer_of(norm)
    gy, gh = torch.randn(48, 128, device="cuda"), torch.randn(48, 256, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        w, wn = layer.weight.detach(), layer.norm_weight.detach()
        n8, bn, _, h, rstd = norm.rmsnorm_quantize(x, wn, fl.E4M3, residual=r if residual else None, eps=EPS)
        w8, bw, _ = fl.quantize(w, fl.E4M3)
        dy8, bdy, _ = fl.quantize(gy, fl.E5M2)
        dn = fl.scaled_gemm_auto(fl.OP_DGRAD, dy8, fl.E5M2, bdy, w8, fl.E4M3, bw)
        dw = fl.scaled_gemm_auto(fl.OP_WGRAD, dy8, fl.E5M2, bdy, n8, fl.E4M3, bn)
        dx, dwn = norm.rmsnorm_bwd(dn, h, wn, rstd, dh=gh if residual else None)
    if residual:
        torch.autograd.backward(list(layer(x, r)), [gy, gh])
        assert torch.equal(r.grad, dx)
    else:
        layer(x).backward(gy)
    assert torch.equal(x.grad, dx.to(x.dtype))
    assert torch.equal(layer.weight.grad, dw) and torch.equal(layer.norm_weight.grad, dwn)


def test_norm_function_without_residual(mods):
    """Against the 64-bit gradient: E = 2^-18 of the terms (sums and products in
    fp32) and the rounding of dy, given in bf16, is none."""
    _, norm = mods
    x, _ = tensors(6)
    w = (1 + 0.1 * torch.randn(256, device="cuda")).requires_grad_()
    gy = torch.randn(48, 256, device="cuda").to(torch.bfloat16)
    norm.RMSNormFunction.apply(x, None, w, EPS).backward(gy)
    xd, wd, dy = (t.detach().double().cpu().numpy() for t in (x, w, gy))
    rs = 1 / np.sqrt((xd * xd).mean(1) + EPS)
    dx, dw = ref.norm_grads(dy, xd, wd, rs, None)
    g, xh = np.abs(dy * wd), np.abs(xd * rs[:, None])
    terms = rs[:, None] * (g + xh * (g * xh).mean(1, keepdims=True))
    assert np.all(np.abs(x.grad.double().cpu().numpy() - dx) <= 2.0 ** -17 * terms)
    assert np.all(np.abs(w.grad.double().cpu().numpy() - dw) <= 2.0 ** -17 * (np.abs(dy) * xh).sum(0))


@pytest.mark.parametrize("residual", [False, True])
def test_accumulation_into_weight_grad(mods, residual):
    """fuse_wgrad_accumulation: three passes add up as fp8_scaled_gemm_accumulate
    does, the norm's weight as autograd adds."""
    fl, norm = mods
    plain, fused = layer_of(norm, 7), layer_of(norm, 7)
    fused.state.fuse_wgrad_accumulation = True
    assert torch.equal(plain.weight, fused.weight)
    each = []
    for k in range(3):
        gy = torch.randn(48, 128, device="cuda")
        for layer in (plain, fused):
            x, r = tensors(20 + k)
            y = layer(x, r)[0] if residual else layer(x)
            y.backward(gy)
        each.append(plain.weight.grad)
        plain.weight.grad = None
        if k == 0:
            first = fused.weight.grad
    assert fused.weight.grad is first
    want = (each[0] + each[1]) + each[2]
    # the accumulating product rounds each sum once, as autograd does
    assert torch.allclose(first, want, rtol=0, atol=2.0 ** -22 * float(torch.stack(each).abs().max() * 3))
    assert torch.equal(plain.norm_weight.grad, fused.norm_weight.grad)


def test_second_backward(mods):
    """Of a retained graph: the gradients again; of a freed one: autograd's error."""
    _, norm = mods
    x, r = tensors(8)
    layer = layer_of(norm)
    gy = torch.randn(48, 128, device="cuda")
    y, h = layer(x, r)
    y.backward(gy, retain_graph=True)
    once = [t.grad.clone() for t in (x, r, layer.weight, layer.norm_weight)]
    for t in (x, r, layer.weight, layer.norm_weight):
        t.grad = None
    y.backward(gy)
    for t, g in zip((x, r, layer.weight, layer.norm_weight), once):
        assert torch.equal(t.grad, g)
    with pytest.raises(RuntimeError, match="second time"):
        y.backward(gy)
