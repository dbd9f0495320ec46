"""RMS norm with the residual's addition (fp8_rmsnorm_*) against its definition
in 64 bits.

Bounds.  A row's sum of squares is a chain of at most 32 fused additions a
lane and a tree of at most 10 more, so rstd is within (42 / 2 + 4) 2^-24 <
2^-19 of the definition, relative; y adds two roundings: 2^-18 = E.  bf16 adds
2^-8 of the value.  A code must lie between the codes of y (1 - E) and
y (1 + E).  Gradients: sums and products again within E of the sum of their
terms' magnitudes; dw sums at most 64 terms in a row: 2 E."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
E = 2.0 ** -18
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (1, 8192), (3, 4), (5, 7), (2, 64), (130, 768), (17, 1000), (9, 1026), (4, 2048), (33, 2052),
          (6, 4096), (3, 4099), (7, 5120), (2, 8191), (2, 8196), (3, 16384), (2, 16383), (2, 32768),
          (9, 1021), (6, 2047), (5, 4097), (3, 8190), (2, 2), (3, 3)]


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import norm
    import fp8_precision_linear_amd as fl
    return fl, norm


def make(rows, d, xt, rt, wt, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * rows + d)
    x = torch.randn(rows, d, generator=g).to(xt)
    r = None if rt is None else (torch.randn(rows, d, generator=g) * 3).to(rt)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(wt)
    if r is not None and d > 3:
        r[:, d // 3] *= 30   # a strong column
    return x, r, w


def dev(t):
    return None if t is None else t.cuda()


def check_codes(codes, y, bias, fmt, what):
    got = ref.code_values(fmt)[codes]
    s = 2.0 ** bias
    a, b = ref.round_fp8(y * s * (1 - E), fmt), ref.round_fp8(y * s * (1 + E), fmt)
    assert np.all((got >= np.minimum(a, b)) & (got <= np.maximum(a, b))), what


TYPES = [(F32, BF, F32), (BF, BF, BF), (BF, F32, F32), (F32, None, BF), (BF, None, F32), (F32, F32, F32)]


@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward(mods, rows, d):
    fl, norm = mods
    for i, (xt, rt, wt) in enumerate(TYPES):
        say("norm", rows, d, xt, rt, wt)
        x, r, w = make(rows, d, xt, rt, wt, i)
        h64 = ref.norm_h(x, r)
        y64, rstd64 = ref.norm_y(h64, w.double().numpy(), EPS)
        fmt = (fl.E4M3, fl.E5M2)[i % 2]
        am = torch.empty(1, device="cuda")
        y, h, rstd = norm.rmsnorm_fwd(dev(x), dev(w), residual=dev(r), eps=EPS, amax=am)
        assert h.dtype == (xt if rt is None else rt) and np.array_equal(h.cpu().double().numpy(), h64)
        assert np.all(np.abs(rstd.cpu().double().numpy() - rstd64) <= E / 2 * rstd64)
        assert np.all(np.abs(y.cpu().double().numpy() - y64) <= (2.0 ** -8 * (1 + E) + E) * np.abs(y64) + 2.0 ** -133)
        assert am.item() == y.float().abs().max().item()
        # at a given bias, with the amax of the fp32 values
        bias = torch.tensor([3 - 2 * i], dtype=torch.int32, device="cuda")
        c, h2, rstd2 = norm.rmsnorm_cast(dev(x), dev(w), bias, fmt, residual=dev(r), eps=EPS, amax=am)
        check_codes(c.cpu().numpy(), y64, int(bias), fmt, (rows, d, "cast"))
        assert abs(am.item() - np.abs(y64).max()) <= E * np.abs(y64).max()
        assert torch.equal(h2, h) and torch.equal(rstd2, rstd)
        # current scaling
        rmax = torch.empty(rows, device="cuda")
        q, b, a, h3, rstd3 = norm.rmsnorm_quantize(dev(x), dev(w), fmt, residual=dev(r), eps=EPS, margin=i - 2,
                                                   row_amax=rmax)
        assert torch.equal(h3, h) and torch.equal(rstd3, rstd)
        assert a.item() == am.item() == rmax.max().item()
        assert np.all(np.abs(rmax.cpu().double().numpy() - np.abs(y64).max(1)) <= E * np.abs(y64).max(1))
        assert int(b) == ref.bias_of(a.item(), fmt) - (i - 2)
        check_codes(q.cpu().numpy(), y64, int(b), fmt, (rows, d, "quantize"))
        # the same codes as the cast at that bias
        c2, _, _ = norm.rmsnorm_cast(dev(x), dev(w), b, fmt, residual=dev(r), eps=EPS)
        assert torch.equal(c2, q)


@pytest.mark.parametrize("rows,d", SHAPES)
def test_backward(mods, rows, d):
    fl, norm = mods
    for i, (yt, ht, wt, with_dh) in enumerate([(F32, BF, F32, True), (BF, BF, BF, False), (F32, F32, F32, True),
                                               (BF, F32, F32, False)]):
        say("norm gradient", rows, d, yt, ht, with_dh)
        h, dh, w = make(rows, d, ht, ht if with_dh else None, wt, 50 + i)
        dy = make(rows, d, yt, None, wt, 90 + i)[0]
        h64, w64, dy64 = h.double().numpy(), w.double().numpy(), dy.double().numpy()
        rstd = torch.from_numpy(1 / np.sqrt((h64 * h64).mean(1) + EPS)).float()
        r64 = rstd.double().numpy()
        dx64, dw64 = ref.norm_grads(dy64, h64, w64, r64, None if dh is None else dh.double().numpy())
        am = torch.empty(1, device="cuda")
        dx, dw = norm.rmsnorm_bwd(dev(dy), dev(h), dev(w), dev(rstd), dh=dev(dh), amax=am)
        g, xh = np.abs(dy64 * w64), np.abs(h64 * r64[:, None])
        terms = r64[:, None] * (g + xh * (g * xh).mean(1, keepdims=True)) + (0 if dh is None else dh.double().abs().numpy())
        bound = E * terms + (2.0 ** -8 * np.abs(dx64) if ht == BF else 0) + 2.0 ** -133
        assert np.all(np.abs(dx.cpu().double().numpy() - dx64) <= bound), (rows, d, i)
        assert np.all(np.abs(dw.cpu().double().numpy() - dw64) <= 2 * E * (np.abs(dy64) * xh).sum(0) + 1e-30)
        assert am.item() == dx.float().abs().max().item()
        # the same bits again, and with dx written over dh
        over = dev(dh).clone() if dh is not None else None
        dx2, dw2 = norm.rmsnorm_bwd(dev(dy), dev(h), dev(w), dev(rstd), dh=over, dx=over)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_many_rows(mods):
    """More rows than workgroups, an odd number of them."""
    fl, norm = mods
    for rows, d in ((9001, 256), (2500, 1100)):
        x, r, w = make(rows, d, F32, BF, F32)
        h64 = ref.norm_h(x, r)
        y64, r64 = ref.norm_y(h64, w.double().numpy(), EPS)
        q, b, a, h, rstd = norm.rmsnorm_quantize(dev(x), dev(w), fl.E4M3, residual=dev(r), eps=EPS)
        check_codes(q.cpu().numpy(), y64, int(b), fl.E4M3, rows)
        dy = torch.randn(rows, d)
        dx, dw = norm.rmsnorm_bwd(dev(dy), h, dev(w), rstd)
        dx64, dw64 = ref.norm_grads(dy.double().numpy(), h64, w.double().numpy(), rstd.cpu().double().numpy(), None)
        assert np.all(np.abs(dw.cpu().double().numpy() - dw64)
                      <= 2 * E * (np.abs(dy.double().numpy() * h64 * r64[:, None])).sum(0))


def test_gradient_against_differences(mods):
    """Central differences of the definition in 64 bits, along random
    directions: step 1e-5 of values of scale 1, so the differences themselves
    are good to about 1e-9 of the terms; the kernel to E of them."""
    fl, norm = mods
    rng = np.random.default_rng(4)
    rows, d = 6, 97
    h, w, dy = rng.standard_normal((rows, d)), 1 + 0.2 * rng.standard_normal(d), rng.standard_normal((rows, d))
    h, w, dy = (v.astype(np.float32).astype(np.float64) for v in (h, w, dy))
    loss = lambda hh, ww: (ref.norm_y(hh, ww, EPS)[0] * dy).sum()  # noqa: E731
    t = lambda v: torch.from_numpy(v.astype(np.float32)).cuda()  # noqa: E731
    rstd = t(1 / np.sqrt((h * h).mean(1) + EPS))
    dx, dw = norm.rmsnorm_bwd(t(dy), t(h), t(w), rstd)
    dx, dw = dx.cpu().double().numpy(), dw.cpu().double().numpy()
    for _ in range(5):
        u, v = rng.standard_normal((rows, d)), rng.standard_normal(d)
        s = 1e-5
        want = (loss(h + s * u, w) - loss(h - s * u, w)) / (2 * s)
        assert abs((dx * u).sum() - want) <= 4 * E * np.abs(u * dy).sum() * 3
        want = (loss(h, w + s * v) - loss(h, w - s * v)) / (2 * s)
        assert abs((dw * v).sum() - want) <= 4 * E * np.abs(v).sum() * np.abs(dy).sum(0).max()


def test_special_values(mods):
    """Zeros, infinities, NaN, a row whose squares overflow, tiny rows."""
    fl, norm = mods
    x = torch.randn(6, 64)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1e30
    x[4] *= 1e-30
    w = torch.ones(64)
    y, _, rstd = norm.rmsnorm_fwd(x.cuda(), w.cuda(), eps=EPS)
    y, rstd = y.float().cpu(), rstd.cpu()
    assert torch.equal(y[0], torch.zeros(64)) and abs(rstd[0].item() * EPS ** 0.5 - 1) < 1e-5
    assert y[1].isnan().all()
    assert y[2, 7].isnan() and (y[2, :7] == 0).all()   # rstd = 0, inf * 0
    assert rstd[3] == 0 and (y[3] == 0).all()
    assert torch.allclose(y[4], x[4] * EPS ** -0.5, rtol=2 ** -7)
    b = torch.zeros(1, dtype=torch.int32, device="cuda")
    c, _, _ = norm.rmsnorm_cast(x.cuda(), w.cuda(), b, fl.E4M3, eps=EPS)
    assert (c[1] & 0x7F == 0x7F).all() and int(c[2, 7]) & 0x7F == 0x7F
    _, bias, amax, _, _ = norm.rmsnorm_quantize(x.cuda(), w.cuda(), fl.E4M3, eps=EPS)
    assert amax.isnan().item() and int(bias) == 0   # as fp8_amax and fp8_compute_bias have it
    # biases far outside the conversion's own range
    for bb in (-200, -127, 126, 127, 160):
        b.fill_(bb)
        v = torch.ldexp(torch.randn(4, 64), torch.tensor(max(-120, min(120, -bb))))
        r1 = torch.ones(4, 64)
        c, h, rs = norm.rmsnorm_cast(v.cuda(), w.cuda(), b, fl.E4M3, eps=EPS)
        y64, _ = ref.norm_y(v.double().numpy(), np.ones(64), EPS)
        check_codes(c.cpu().numpy(), y64, bb, fl.E4M3, bb)
        del r1


def test_empty(mods):
    fl, norm = mods
    x, w = torch.empty(0, 128, device="cuda"), torch.ones(128, device="cuda")
    am = torch.full((1,), 7.0, device="cuda")
    y, h, rstd = norm.rmsnorm_fwd(x, w, amax=am)
    assert y.shape == (0, 128) and am.item() == 0
    q, b, a, _, _ = norm.rmsnorm_quantize(x, w, fl.E4M3)
    assert int(b) == 0 and a.item() == 0
    dx, dw = norm.rmsnorm_bwd(x, x, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 128) and torch.equal(dw, torch.zeros_like(dw))


def test_other_stream_and_graph(mods):
    """On a stream of the caller's, and replayed from a graph on new inputs."""
    fl, norm = mods
    s = torch.cuda.Stream()
    x, r, w = (dev(t) for t in make(300, 1024, F32, BF, F32))
    want = norm.rmsnorm_quantize(x, w, fl.E4M3, residual=r)
    s.wait_stream(torch.cuda.current_stream())
    got = norm.rmsnorm_quantize(x, w, fl.E4M3, residual=r, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    dy = torch.randn(300, 1024, device="cuda")
    outs = dict(out=torch.empty_like(want[0]), bias=torch.empty_like(want[1]), amax=torch.empty_like(want[2]),
                h=torch.empty_like(want[3]), rstd=torch.empty_like(want[4]), row_amax=torch.empty(300, device="cuda"))
    dx, dw = torch.empty(300, 1024, dtype=BF, device="cuda"), torch.empty(1024, device="cuda")
    ws = torch.empty(norm.rmsnorm_bwd_workspace_bytes(300, 1024), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm.rmsnorm_quantize(x, w, fl.E4M3, residual=r, **outs)
        norm.rmsnorm_bwd(dy, outs["h"], w, outs["rstd"], dx=dx, dw=dw, workspace=ws)
    for k in range(3):
        x.copy_(torch.randn(300, 1024, device="cuda") * (k + 1))
        g.replay()
        torch.cuda.synchronize()
        want = norm.rmsnorm_quantize(x, w, fl.E4M3, residual=r)
        wx, ww = norm.rmsnorm_bwd(dy, want[3], w, want[4])
        for a, b in zip((outs["out"], outs["bias"], outs["amax"], outs["h"], outs["rstd"], dx, dw), (*want, wx, ww)):
            assert torch.equal(a, b)


def test_modules(mods):
    """The autograd forms: gradients reach x, residual and both weights; the
    fused norm and FP8 linear equals the norm, then the product of its codes."""
    fl, norm = mods
    x, r, w = (dev(t) for t in make(96, 256, F32, BF, F32))
    x.requires_grad_(), r.requires_grad_(), w.requires_grad_()
    y, h = norm.RMSNormFunction.apply(x, r, w, EPS)
    gy, gh = torch.randn(96, 256, device="cuda").to(BF), torch.randn(96, 256, device="cuda").to(BF)
    torch.autograd.backward([y, h], [gy, gh])
    _, h1, rstd = norm.rmsnorm_fwd(x.detach(), w.detach(), residual=r.detach(), eps=EPS)
    dx, dw = norm.rmsnorm_bwd(gy, h1, w.detach(), rstd, dh=gh)
    assert torch.equal(x.grad, dx.float()) and torch.equal(r.grad, dx) and torch.equal(w.grad, dw)

    layer = norm.FP8NormLinear(256, 128, eps=EPS, device="cuda")
    with torch.no_grad():
        layer.norm_weight.copy_(w)
    x.grad = r.grad = None
    y, h = layer(x, r)
    q, b, _, h2, _ = norm.rmsnorm_quantize(x.detach(), layer.norm_weight.detach(), fl.E4M3, residual=r.detach(), eps=EPS)
    w8, bw, _ = fl.quantize(layer.weight.detach(), fl.E4M3)
    assert torch.equal(h, h2) and torch.equal(y, fl.scaled_gemm_auto(fl.OP_FWD, q, fl.E4M3, b, w8, fl.E4M3, bw))
    gy = torch.randn(96, 128, device="cuda")
    torch.autograd.backward([y, h], [gy, gh])
    # against the gradients in 64 bits: FP8 gradients are good to the formats'
    # half steps (2^-3 for dy in E5M2, 2^-4 for the others), averaged over sums
    h64 = h.detach().double()
    rs = (h64.square().mean(1, keepdim=True) + EPS).rsqrt()
    n64 = h64 * rs * layer.norm_weight.detach().double()
    dn = gy.double() @ layer.weight.detach().double()
    want = ref.norm_grads(dn.cpu().numpy(), h64.cpu().numpy(), layer.norm_weight.detach().double().cpu().numpy(),
                          rs[:, 0].cpu().numpy(), gh.double().cpu().numpy())
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    assert rel(r.grad.double().cpu().numpy(), want[0]) < 0.15
    assert rel(layer.norm_weight.grad.double().cpu().numpy(), want[1]) < 0.15
    assert rel(layer.weight.grad.double().cpu().numpy(), (gy.double().t() @ n64).cpu().numpy()) < 0.15
