"""Attention over packed sequences at its edges: what is not seen has no
influence, rows of no sequence stay as they are, any arrays stay within the
buffers, and calls on other streams, from graphs and at the same time give the
same bits."""
import pytest
import torch

import seq_ref
from gpu_util import need_gpu, say
from test_gpu_self_attention import inputs

pytestmark = pytest.mark.gpu
SHAPES = [(2, 2, 64), (4, 2, 128), (2, 1, 256)]
GRADS = ("dq", "dk", "dv")


@pytest.fixture(scope="module")
def sa():
    need_gpu()
    from fp8_precision_linear_amd import self_attention
    return self_attention


def both(sa, q, k, v, dout, seqs, **kw):
    out, lse = sa.attention_fwd(q, k, v, seqs, **kw)
    return (out, lse, *sa.attention_bwd(dout, q, k, v, out, lse, seqs, **kw))


def same(a, b):
    """The same bits, NaN included."""
    return all(torch.equal(x.contiguous().view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                           y.contiguous().view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32)) for x, y in zip(a, b))


def inside(lens, Hq, D, q, k, v, dout, out, lse, *grads):
    T = sum(lens)
    q, k, v, dout = (t[:T] for t in (q, k, v, dout))
    seq_ref.inside({"out": out, "lse": lse}, seq_ref.forward(q, k, v, lens, D ** -0.5), "forward")
    seq_ref.inside(dict(zip(GRADS, grads)), seq_ref.backward(dout, q, k, v, out, lse, lens, D ** -0.5), "backward")


@pytest.mark.parametrize("heads", SHAPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("at", [0, 70, 199, 200, 299])
def test_unseen_nan_has_no_influence(sa, heads, bad, at):
    """One token of k, v, q or dout is bad: rows that do not see it (earlier
    ones, other sequences) keep their bits, and those that do are not finite."""
    say("unseen", heads, bad, at)
    Hq, H, D = heads
    lens = [200, 100, 0, 65]
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, dout = inputs(lens, Hq, H, D, 3)
    clean = both(sa, q, k, v, dout, seqs)
    lo, hi = (0, 200) if at < 200 else (200, 300)
    T = sum(lens)
    after = torch.zeros(T, dtype=torch.bool, device="cuda")
    after[at:hi] = True                  # the queries that see token `at`
    before = torch.zeros_like(after)
    before[lo:at + 1] = True             # the keys that query `at` sees
    for name in ("k", "v", "q", "dout"):
        t = {n: x.clone() for n, x in (("q", q), ("k", k), ("v", v), ("dout", dout))}
        t[name][at, 0, 5] = bad
        got = dict(zip(("out", "lse", *GRADS), both(sa, t["q"], t["k"], t["v"], t["dout"], seqs)))
        want = dict(zip(("out", "lse", *GRADS), clean))
        group = slice(0, Hq // H) if name in ("k", "v") else slice(0, 1)
        if name in ("k", "v"):           # reaches the queries after it, and through them every key these see
            rows = {"out": after, "lse": after if name == "k" else ~after & after, "dq": after}
            keys = torch.zeros_like(after)
            keys[lo:hi] = True
            rows["dk"] = rows["dv"] = keys
        else:                            # reaches its own row, and the keys that this sees
            own = torch.zeros_like(after)
            own[at] = True
            rows = {"dq": own, "dk": before, "dv": before, "out": own, "lse": own}
            if name == "dout":
                rows["out"] = rows["lse"] = ~own & own
        for n, reached in rows.items():
            heads_of = group if n in ("out", "lse", "dq") else slice(0, 1)
            other = torch.ones(got[n].shape[:2], dtype=torch.bool, device="cuda")
            other[:, heads_of] = ~reached[:, None]
            assert same((got[n][other],), (want[n][other],)), (name, n)
        # and what does see it says so
        if name in ("q", "dout"):
            assert not bool(got["dq"][at, 0].isfinite().all()) and not bool(got["dk"][at, 0].isfinite().all()), name
        elif name == "v" or bad != bad:   # (an infinite key may be a logit of -inf: a weight of zero)
            assert not bool(got["out"][at, 0].isfinite().all()) and not bool(got["dq"][at, 0].isfinite().all()), name


@pytest.mark.parametrize("heads", SHAPES)
def test_seen_infinite_value_is_nan_in_its_dimension(sa, heads):
    Hq, H, D = heads
    lens = [300]
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, _ = inputs(lens, Hq, H, D, 4)
    v[100, 0, 9] = float("inf")
    out, lse = sa.attention_fwd(q, k, v, seqs)
    assert bool(out[100:, 0, 9].isnan().all()) and bool(lse.isfinite().all())
    out[100:, :Hq // H, 9] = 0
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("heads", SHAPES)
def test_window_hides_nan(sa, heads):
    """A bad key and value behind the window of the queries after it."""
    Hq, H, D = heads
    lens = [400]
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, dout = inputs(lens, Hq, H, D, 5)
    clean = both(sa, q, k, v, dout, seqs, window=50)
    k, v = k.clone(), v.clone()
    k[100], v[100] = float("nan"), float("inf")
    got = both(sa, q, k, v, dout, seqs, window=50)
    for n, a, b in zip(("out", "lse", "dq"), got, clean):
        assert same((a[:100], a[150:]), (b[:100], b[150:])), n
    for a, b in zip(got[3:], clean[3:]):    # keys that queries 100 .. 149 do not see
        assert same((a[:51], a[150:]), (b[:51], b[150:]))


@pytest.mark.parametrize("heads", SHAPES)
def test_rows_of_no_sequence_stay(sa, heads):
    Hq, H, D = heads
    lens = [70, 33]
    q, k, v, dout = inputs([*lens, 50], Hq, H, D, 6)
    T = q.shape[0]
    cu = torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda")
    seqs = sa.Sequences(cu, max_len=100, tokens=T)       # (a loose bound)
    o = [torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, Hq), 7.0, device="cuda")]
    g = [torch.full((T, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (Hq, H, H)]
    sa.attention_fwd(q, k, v, seqs, out=o[0], lse=o[1])
    sa.attention_bwd(dout, q, k, v, *o, seqs, dq=g[0], dk=g[1], dv=g[2])
    for t in (*o, *g):
        assert bool((t[103:] == 7.0).all()) and bool((t[:103] != 7.0).any())
    # (other bounds than the lengths' own cut the work differently: no bits to compare)
    inside(lens, Hq, D, q, k, v, dout, *[t[:103] for t in (*o, *g)])
    # the autograd function clears them
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    sa.attention(*leaves, seqs).backward(dout)
    for leaf, t in zip(leaves, g):
        assert not leaf.grad[103:].any() and same((leaf.grad[:103],), (t[:103],))


def test_any_arrays_stay_within_the_buffers(sa):
    """cu_tokens that are not what they should be: rows past the tensors do not
    exist, lengths are held to max_len, and nothing outside is written."""
    Hq, H, D, T = 4, 2, 64, 200
    for cu, most in (([0, 300, 900], 1000), ([-50, 20, 1 << 30], 1 << 30), ([150, 10, 190, 5, 250], 100), ([0, 200], 64),
                     ([0, 50, 0, 50, 0, 200, 100], 200)):
        say("arrays", cu, most)
        pad = torch.full((T + 64, Hq + 2 * H, D), 3.0, dtype=torch.bfloat16, device="cuda")
        q, k, v, dout = inputs([T], Hq, H, D, 7)
        seqs = sa.Sequences(torch.tensor(cu, dtype=torch.int32, device="cuda"), max_len=most, tokens=T)
        out, lse = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, Hq, device="cuda")
        sa.attention_fwd(q, k, v, seqs, out=out, lse=lse)
        rows = pad[:T]
        sa.attention_bwd(dout, q, k, v, out, lse, seqs, dq=rows[:, :Hq], dk=rows[:, Hq:Hq + H], dv=rows[:, Hq + H:])
        torch.cuda.synchronize()
        assert bool((pad[T:] == 3.0).all())


def test_length_bound_cuts_sequences(sa):
    q, k, v, dout = inputs([200], 2, 2, 64, 8)
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    got = both(sa, q, k, v, dout, sa.Sequences(cu, max_len=64, tokens=200))
    inside([64], 2, 64, q, k, v, dout, *[t[:64] for t in got])


@pytest.mark.parametrize("heads", SHAPES)
def test_strides_and_outputs_in_one_tensor(sa, heads):
    Hq, H, D = heads
    lens = [130, 70]
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, dout = inputs(lens, Hq, H, D, 9)
    want = both(sa, *(t.contiguous() for t in (q, k, v, dout)), seqs)
    wide = torch.randn(200, Hq + 3, D, device="cuda").to(torch.bfloat16)
    wide[:, :Hq] = dout
    out, lse = sa.attention_fwd(q, k, v, seqs)
    into = torch.zeros(200, Hq + 2 * H + 1, D, dtype=torch.bfloat16, device="cuda")
    got = sa.attention_bwd(wide[:, :Hq], q, k, v, out, lse, seqs, dq=into[:, :Hq], dk=into[:, Hq:Hq + H],
                           dv=into[:, Hq + H:Hq + 2 * H])
    assert same((out, lse, *got), want) and not into[:, -1].any()
    # autograd takes any strides: heads first, and a gradient that is an expanded row
    leaves = [t.transpose(0, 1).contiguous().requires_grad_() for t in (q, k, v)]
    y = sa.attention(*(t.transpose(0, 1) for t in leaves), seqs)
    y.backward(dout[:1].expand_as(dout))
    flat = both(sa, q.contiguous(), k.contiguous(), v.contiguous(), dout[:1].expand_as(dout).contiguous(), seqs)
    assert same([t.grad.transpose(0, 1) for t in leaves], flat[2:])


@pytest.mark.parametrize("heads", SHAPES)
def test_streams_and_repeats(sa, heads):
    """The same bits from another stream, from two calls at once, and again."""
    Hq, H, D = heads
    lens = [300, 129, 1]
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, dout = inputs(lens, Hq, H, D, 10)
    want = both(sa, q, k, v, dout, seqs)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [both(sa, q, k, v, dout, seqs, stream=s) for s in sides for _ in range(2)]
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)


@pytest.mark.parametrize("heads", SHAPES)
def test_graph(sa, heads):
    """Forward and backward captured; replays on new contents, with eager calls
    between them, give the eager calls' bits.  Two graphs, replayed in turn."""
    Hq, H, D = heads
    lens = [200, 77]
    seqs = sa.Sequences.from_lists(lens)
    bufs = [t.contiguous() for t in inputs(lens, Hq, H, D, 11)]
    outs, graphs = [], []
    both(sa, *bufs, seqs)
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(sa, *bufs, seqs))
        graphs.append(g)
    for r in range(4):
        for b, t in zip(bufs, inputs(lens, Hq, H, D, 20 + r)):
            b.copy_(t)
        want = both(sa, *bufs, seqs)
        torch.cuda.synchronize()
        for t in outs[r % 2]:
            t.fill_(3)
        graphs[r % 2].replay()
        torch.cuda.synchronize()
        assert same(outs[r % 2], want), r


def test_autograd_in_a_graph(sa):
    """A training step's forward and backward captured as one graph."""
    lens = [90, 40]
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, dout = (t.contiguous() for t in inputs(lens, 4, 2, 64, 12))
    want = both(sa, q, k, v, dout, seqs)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sa.attention(*leaves, seqs).backward(dout)
    torch.cuda.current_stream().wait_stream(side)
    for t in leaves:
        t.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = sa.attention(*leaves, seqs)
        y.backward(dout)
    for _ in range(3):
        for t in leaves:
            t.grad.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        assert same((y.detach(), *(t.grad for t in leaves)), (want[0], *want[2:]))


def test_second_derivative_is_refused(sa):
    q, k, v, _ = (t.contiguous().requires_grad_() for t in inputs([20], 2, 2, 64, 13))
    y = sa.attention(q, k, v, sa.Sequences.from_lists([20]))
    g, = torch.autograd.grad(y.float().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_gradient_against_differences(sa):
    """Directional derivatives of the 64-bit function: the gradients' own rounding
    (2^-8 of each element's bound) summed along a direction of signs."""
    lens = [70, 33]
    q, k, v, dout = inputs(lens, 4, 2, 64, 14)
    seqs = sa.Sequences.from_lists(lens)
    out, lse, *grads = both(sa, q, k, v, dout, seqs)
    want = seq_ref.backward(dout, q, k, v, out, lse, lens, 0.125)
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = [t.double() for t in (q, k, v)]

    def loss(*xs):
        return (seq_ref.forward(*xs, lens, 0.125)["out"][0] * dout.double()).sum().item()
    step = 1e-3
    for i, name in enumerate(GRADS):
        way = torch.randint(0, 2, xs[i].shape, generator=g, device="cuda").double() * 2 - 1
        up, down = (loss(*[x + s * step * way if j == i else x for j, x in enumerate(xs)]) for s in (1, -1))
        got = (grads[i].double() * way).sum().item()
        # the true gradient's delta has the unrounded out: another 2^-8 sum |dout out| p |k|, inside
        # the bound's own 2^-8 sum |ds| |k| up to a factor of few; errors of random sign add as roots
        slack = 8 * want[name][1].square().sum().sqrt().item() + 1e-4 * (grads[i].double() * way).abs().sum().item()
        assert abs(got - (up - down) / (2 * step)) <= slack, name


def test_huge_logits(sa):
    """Logits of 2^24 and more: the largest key takes all, in every tile order."""
    for D in (64, 128, 256):
        q, k, v, _ = inputs([200], 2, 2, D, 15)
        q, k = q * 2.0 ** 14, k * 2.0 ** 14
        seqs = sa.Sequences.from_lists([200])
        out, lse = sa.attention_fwd(q, k, v, seqs)
        want = seq_ref.forward(q, k, v, [200], D ** -0.5)
        assert bool(((lse.double() - want["lse"][0]).abs() <= 2.0 ** -20 * want["lse"][0].abs() + 1).all())
        s = torch.stack([(q[:, a].double() @ k[:, a].double().t()).masked_fill(~seq_ref.visible(200, True, 0), -torch.inf)
                         for a in range(2)])
        top = s.topk(2, dim=2).values
        # where the largest logit leads by far more than fp32 rounds it, out is its value
        clear = ((top[..., 0] - top[..., 1]) * D ** -0.5 > 2.0 ** -18 * top[..., 0].abs() * D ** -0.5 + 40).t()
        clear[0] = True
        best = s.argmax(2).t()
        vals = torch.stack([v[best[:, a], a] for a in range(2)], 1)
        assert bool(out.isfinite().all()) and torch.equal(out[clear], vals[clear])
