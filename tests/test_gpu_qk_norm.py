"""Norms of queries and keys with the rotation, and their gradients, against
their 64-bit forms.

Bounds, relative to magnitudes before cancellation.  h = 2^-8 is half a step of
bf16 (none for an fp32 dx), u = 2^-20 covers the fp32 arithmetic: a sum of at most
256 squares or products (2^-24 * 8 by the tree of the lanes' sums), a root, four
products, one sum.  With c, s the angles, a rotated element's magnitude is
|a c| + |b s|.
  y   h |y| + u M,  M the rotation of |n|
  dx  h |dx| + u rstd (|g| + |xhat| mean |g xhat|), g from the rotated magnitudes
  dw  2^-18 sum |dn xhat|   (a lane adds up to some 100 terms in fp32)"""
import pytest
import torch

from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
H8, U = 2.0 ** -8, 2.0 ** -20
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def qn():
    need_gpu()
    from fp8_precision_linear_amd import qk_norm
    return qk_norm


def tables(positions, D):
    inv = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def turn(x, c, s, pairs, magnitude=False):
    """x [T, heads, D] rotated by c, s [T, D / 2]; or its magnitudes."""
    D = x.shape[-1]
    c, s = c[:, None], s[:, None]
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :D // 2], x[..., D // 2:])
    if magnitude:
        lo, hi = a.abs() * c.abs() + b.abs() * s.abs(), b.abs() * c.abs() + a.abs() * s.abs()
    else:
        lo, hi = a * c - b * s, b * c + a * s
    return torch.stack((lo, hi), -1).flatten(-2) if pairs else torch.cat((lo, hi), -1)


def make(T, Hq, H, D, xt, norm, wt=torch.float32, strided=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T)
    n = Hq + 2 * H
    x = torch.randn(T, n + (2 if strided else 0), D, generator=g, device="cuda").to(xt)[:, :n]
    w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(wt) for _ in range(2)] if norm else [None, None]
    dy = [torch.randn(T, k, D, generator=g, device="cuda").to(torch.bfloat16) for k in (Hq, H, H)]
    pos = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32)
    return x, w, dy, pos


def check(qn, T, Hq, H, D, xt=torch.float32, rope="halves", norm=True, wt=torch.float32, strided=False, positions=True,
          eps=1e-5):
    say(T, Hq, H, D, xt, rope, norm, wt, strided, positions)
    x, (wq, wk), (dq, dk, dv), pos = make(T, Hq, H, D, xt, norm, wt, strided)
    rows = 50 if positions else T + 3
    table = tables(rows, D) if rope != "none" else None
    at = pos.long() if positions else torch.arange(T, device="cuda")
    one, zero = torch.ones(T, D // 2, dtype=torch.float64, device="cuda"), torch.zeros(T, D // 2, dtype=torch.float64, device="cuda")
    c, s = (table[0].double()[at], table[1].double()[at]) if table else (one, zero)
    pairs = rope == "pairs"
    more = dict(wq=wq, wk=wk, eps=eps, rope=table, positions=pos if positions else None, rope_pairs=pairs)
    q, k, v = qn.qk_norm_rope_fwd(x, Hq, H, **more)
    dx, dwq, dwk = qn.qk_norm_rope_bwd(dq, dk, dv, x, **more)
    assert torch.equal(v, x[:, Hq + H:].to(torch.bfloat16))
    assert torch.equal(dx[:, Hq + H:], dv.to(xt))
    hx = H8 if xt == torch.bfloat16 else 2.0 ** -24
    for name, got, grad, dy, xs, w, dw in (("q", q, dx[:, :Hq], dq, x[:, :Hq], wq, dwq),
                                           ("k", k, dx[:, Hq:Hq + H], dk, x[:, Hq:Hq + H], wk, dwk)):
        xs, dy = xs.double(), dy.double()
        dn, dm = turn(dy, c, -s, pairs), turn(dy, c, s, pairs, magnitude=True)
        if w is None:
            n, r = xs, None
            want, bound = dn, hx * dn.abs() + U * dm
        else:
            r = (xs.square().mean(2, keepdim=True) + eps).pow(-0.5)
            xhat = xs * r
            n = xhat * w.double()
            g, gm = dn * w.double(), dm * w.double().abs()
            want = r * (g - xhat * (g * xhat).mean(2, keepdim=True))
            bound = hx * want.abs() + U * r * (gm + xhat.abs() * (gm * xhat.abs()).mean(2, keepdim=True))
            off = (dw.double() - (dn * xhat).sum((0, 1))).abs()
            assert bool((off <= 2.0 ** -18 * (dm * xhat.abs()).sum((0, 1)) + TINY).all()), "dw" + name
        y = turn(n, c, s, pairs)
        assert bool(((got.double() - y).abs() <= H8 * y.abs() + U * turn(n, c, s, pairs, magnitude=True) + TINY).all()), name
        assert bool(((grad.double() - want).abs() <= bound + TINY).all()), "d" + name


SHAPES = [(4, 2, 64), (3, 1, 128), (5, 5, 256), (40, 40, 128), (64, 8, 128), (16, 1, 64), (1, 1, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 131])
def test_shapes(qn, shape, T):
    check(qn, T, *shape)


@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rope", ["none", "halves", "pairs"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_kinds(qn, xt, rope, norm, D):
    check(qn, 37, 6, 2, D, xt, rope, norm, wt=torch.bfloat16 if D == 64 else torch.float32)


def test_strided_rows_and_own_positions(qn):
    check(qn, 29, 4, 2, 128, strided=True)
    check(qn, 29, 4, 2, 64, torch.bfloat16, strided=True, positions=False)


def test_many_tokens(qn):
    """More items than the backward's workgroups hold at once."""
    check(qn, 3001, 12, 12, 64)


def test_positions_past_the_table(qn):
    """They count as the table's first and last."""
    x, (wq, wk), _, _ = make(4, 2, 1, 64, torch.float32, True)
    table = tables(10, 64)
    pos = torch.tensor([-3, 0, 9, 1 << 30], dtype=torch.int32, device="cuda")
    q, _, _ = qn.qk_norm_rope_fwd(x, 2, 1, wq, wk, rope=table, positions=pos)
    want, _, _ = qn.qk_norm_rope_fwd(x, 2, 1, wq, wk, rope=table, positions=pos.clamp(0, 9))
    assert torch.equal(q, want)


def test_no_tokens(qn):
    x, (wq, wk), dy, pos = make(0, 2, 1, 64, torch.float32, True)
    q, k, v = qn.qk_norm_rope_fwd(x, 2, 1, wq, wk, rope=tables(3, 64))
    assert q.shape == (0, 2, 64) and k.shape == v.shape == (0, 1, 64)
    dx, dwq, dwk = qn.qk_norm_rope_bwd(*dy, x, wq, wk)
    assert dx.shape == x.shape and not dwq.any() and not dwk.any()


def test_nan_stays_in_its_head(qn):
    x, (wq, wk), dy, pos = make(5, 4, 2, 128, torch.float32, True)
    x[2, 1, 7] = float("nan")
    x[3, 7, 0] = float("inf")      # a value
    q, k, v = qn.qk_norm_rope_fwd(x, 4, 2, wq, wk, rope=tables(50, 128), positions=pos)
    bad = q.isnan().any(2)
    assert bool(bad[2, 1]) and int(bad.sum()) == 1 and not k.isnan().any() and int(v.isinf().sum()) == 1
    dx, dwq, dwk = qn.qk_norm_rope_bwd(*dy, x, wq, wk, rope=tables(50, 128), positions=pos)
    assert int(dx.isnan().any(2).sum()) == 1 and bool(dwq.isnan().any()) and bool(dwk.isfinite().all())


def test_autograd(qn):
    """Gradients of the function against differences of its 64-bit form."""
    x, (wq, wk), (dq, dk, dv), pos = make(3, 2, 1, 64, torch.float32, True)
    leaves = [t.clone().requires_grad_() for t in (x, wq, wk)]
    table = tables(50, 64)
    q, k, v = qn.qk_norm_rope(*leaves[:1], 2, 1, *leaves[1:], rope=table, positions=pos)
    torch.autograd.backward((q, k, v), (dq, dk, dv))
    c, s = table[0].double()[pos.long()], table[1].double()[pos.long()]

    def loss(x, wq, wk):
        total = (x[:, 3:] * dv.double()).sum()
        for xs, w, dy in ((x[:, :2], wq, dq), (x[:, 2:3], wk, dk)):
            n = xs * (xs.square().mean(2, keepdim=True) + 1e-5).pow(-0.5) * w
            total = total + (turn(n, c, s, False) * dy.double()).sum()
        return total.item()
    at = [t.double() for t in (x, wq, wk)]
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, leaf in enumerate(leaves):
        way = torch.randn(leaf.shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-4     # a central difference: off by some 1e-8 of the third derivative
        up = loss(*[t + step * way if j == i else t for j, t in enumerate(at)])
        down = loss(*[t - step * way if j == i else t for j, t in enumerate(at)])
        got = (leaf.grad.double() * way).sum().item()
        assert abs(got - (up - down) / (2 * step)) <= 1e-5 * (leaf.grad.double() * way).abs().sum().item() + 1e-6


def test_graph_and_streams(qn):
    """Both directions captured and replayed, and on two other streams at once:
    the eager calls' bits."""
    T, Hq, H, D = 333, 6, 2, 128
    x, (wq, wk), dy, pos = make(T, Hq, H, D, torch.bfloat16, True)
    more = dict(wq=wq, wk=wk, rope=tables(50, D), positions=pos)

    def both(stream=None):
        y = qn.qk_norm_rope_fwd(x, Hq, H, **more, stream=stream)
        return (*y, *qn.qk_norm_rope_bwd(*dy, x, **more, stream=stream))
    want = both()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [both(s) for _ in range(2) for s in sides]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = both()
    for r in range(3):
        new, _, more_dy, _ = make(T, Hq, H, D, torch.bfloat16, True, seed=1 + r)
        for a, b in zip((x, *dy), (new, *more_dy)):
            a.copy_(b)
        pos.add_(1)
        want = both()
        torch.cuda.synchronize()
        for t in outs:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), r


def test_offsets_past_32_bits(qn):
    """Rows 2^23 elements apart."""
    T, Hq, H, D, row = 300, 2, 1, 64, 1 << 23
    say("rows", row, "apart")
    x, (wq, wk), dy, pos = make(T, Hq, H, D, torch.bfloat16, True)
    more = dict(wq=wq, wk=wk, rope=tables(50, D), positions=pos)
    want = (*qn.qk_norm_rope_fwd(x, Hq, H, **more), *qn.qk_norm_rope_bwd(*dy, x, **more))
    wide = torch.empty(T * row, dtype=torch.bfloat16, device="cuda").view(T, row)
    far, at = [], 0
    for t in (x, *dy):
        n = t.shape[1]
        far.append(wide[:, at:at + n * D].unflatten(1, (n, D)))
        far[-1].copy_(t)
        at += n * D
    got = (*qn.qk_norm_rope_fwd(far[0], Hq, H, **more), *qn.qk_norm_rope_bwd(*far[1:], far[0], **more))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
