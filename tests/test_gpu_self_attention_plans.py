"""Attention over packed sequences in each of the ways that its work is divided:
two sets of waves, whole tiles, and walks of which those over the queries, or
both, are cut into shares (seq_ref.py has the bounds)."""
import pytest
import torch

import seq_ref
from gpu_util import need_gpu, say
from test_gpu_self_attention import check, inputs
from test_gpu_self_attention_edges import both, inside, same

pytestmark = pytest.mark.gpu

# enough tiles for every head's keys, or only for the queries' heads
WHOLE = [([200] * 20, 32, 32, 64), ([130] * 20, 26, 26, 128), ([150] * 10, 26, 26, 256)]
KEYS_CUT = [([200] * 20, 32, 4, 64), ([200, 1, 0, 310] * 5, 32, 8, 128), ([170] * 10, 32, 4, 256)]


@pytest.fixture(scope="module")
def sa():
    need_gpu()
    from fp8_precision_linear_amd import self_attention
    return self_attention


@pytest.mark.parametrize("shape", WHOLE + KEYS_CUT)
@pytest.mark.parametrize("mask", [{}, {"window": 50}, {"causal": False}])
def test_plans(sa, shape, mask):
    check(sa, *shape, **mask, seed=1)


# long sequences among many short ones, whose tiles are counted through
RAGGED = [([20] * 30 + [2100] + [0, 33] * 15, 32, 32, 64), ([1300] + [3] * 600 + [257, 1] * 2, 2, 2, 64),
          ([5] * 20 + [129, 1800, 130] + [1] * 30, 20, 20, 128), ([2, 2000] + [9] * 30, 12, 12, 256),
          ([3] * 100 + [1500], 4, 2, 128), ([1300] + [3] * 600, 2, 1, 64), ([2] * 300 + [900] + [5] * 300, 1, 1, 64)]


@pytest.mark.parametrize("shape", RAGGED)
@pytest.mark.parametrize("mask", [{}, {"window": 140}, {"causal": False}])
def test_ragged(sa, shape, mask):
    check(sa, *shape, **mask, seed=11)


def test_loose_bounds(sa):
    """No host knowledge of the lengths but their sum: the bound is all rows."""
    lens, Hq, H, D = [60] * 30 + [500] + [0] * 300, 32, 32, 64
    T = sum(lens) + 40
    q, k, v, dout = inputs([T], Hq, H, D, 12)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    seqs = sa.Sequences(cu, max_len=1 << 30, tokens=T)
    got = both(sa, q, k, v, dout, seqs)
    say("loose bounds")
    inside(lens, Hq, D, q, k, v, dout, *[t[:T - 40] for t in got])


@pytest.mark.parametrize("mask", [{}, {"causal": False}])
def test_one_head_of_long_rows(sa, mask):
    """Every walk is cut, most of them several times."""
    check(sa, [2300], 1, 1, 64, **mask, seed=2)


@pytest.mark.parametrize("D", [64, 128])
def test_long_causal_rows(sa, D):
    """More workgroups than CUs, and the last of them by far the longest."""
    check(sa, [2100, 300], 16, 4, D, seed=3)


# workgroups of 64 rows, of 128 with two sets of waves, and with one: by the number
# of tiles, the mask and the length
FORWARD = [([300, 65, 1], 4, 2, 64), ([700], 6, 2, 128), ([500, 64], 4, 4, 256), ([1000], 28, 4, 64), ([900], 30, 30, 128),
           ([700, 600], 20, 5, 256), ([2100], 20, 4, 64), ([2100], 14, 2, 128), ([64, 50], 2, 2, 128)]


@pytest.mark.parametrize("shape", FORWARD)
@pytest.mark.parametrize("mask", [{}, {"window": 33}, {"causal": False}])
def test_forward(sa, shape, mask):
    lens, Hq, H, D = shape
    what = f"{lens} {Hq}/{H} of {D} {mask}"
    say(what)
    q, k, v, _ = inputs(lens, Hq, H, D, 13)
    out, lse = sa.attention_fwd(q, k, v, sa.Sequences.from_lists(lens), **mask)
    seq_ref.inside({"out": out, "lse": lse}, seq_ref.forward(q, k, v, lens, D ** -0.5, **mask), what)


@pytest.mark.parametrize("shape", [WHOLE[0], KEYS_CUT[1], WHOLE[2]])
def test_neighbours_keep_their_bits(sa, shape):
    """A sequence of NaN: the others' results are as without it."""
    lens, Hq, H, D = shape
    say("neighbours", *shape)
    seqs = sa.Sequences.from_lists(lens)
    q, k, v, dout = inputs(lens, Hq, H, D, 4)
    want = both(sa, q, k, v, dout, seqs)
    lo = sum(lens[:3])
    rows = slice(lo, lo + lens[3])
    bad = [t.clone() for t in (q, k, v, dout)]
    for t in bad:
        t[rows] = float("nan")
    got = both(sa, *bad, seqs)
    for a, b in zip(got, want):
        assert same((a[:lo], a[rows.stop:]), (b[:lo], b[rows.stop:])) and bool(a[rows].isnan().all())


@pytest.mark.parametrize("shape", [WHOLE[1], KEYS_CUT[0], ([2100, 300], 16, 4, 64)])
def test_graph(sa, shape):
    """Captured, replayed with eager calls between: the eager calls' bits."""
    lens, Hq, H, D = shape
    seqs = sa.Sequences.from_lists(lens)
    bufs = [t.contiguous() for t in inputs(lens, Hq, H, D, 5)]
    both(sa, *bufs, seqs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = both(sa, *bufs, seqs)
    for r in range(3):
        for b, t in zip(bufs, inputs(lens, Hq, H, D, 6 + r)):
            b.copy_(t)
        want = both(sa, *bufs, seqs)
        torch.cuda.synchronize()
        for t in outs:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert same(outs, want), r


def test_lengths_change_under_a_graph(sa):
    """The lengths are the device's: a graph captured with the bounds of a step
    serves others within them."""
    T, Hq, H, D = 400, 4, 2, 64
    q, k, v, dout = (t.contiguous() for t in inputs([T], Hq, H, D, 9))
    cu = torch.tensor([0, 100, 400, 400], dtype=torch.int32, device="cuda")
    seqs = sa.Sequences(cu, max_len=400, tokens=T)
    both(sa, q, k, v, dout, seqs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = both(sa, q, k, v, dout, seqs)
    for ends in ([0, 400, 400, 400], [0, 1, 2, 399], [0, 130, 257, 400], [0, 0, 0, 0]):
        cu.copy_(torch.tensor(ends, dtype=torch.int32))
        want = both(sa, q, k, v, dout, seqs)
        for t in outs:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        n = ends[-1]
        assert same([t[:n] for t in outs], [t[:n] for t in want]) and all(bool((t[n:] == 3).all()) for t in outs)


def test_offsets_past_32_bits(sa):
    """Rows so far apart that elements lie past 2^32 bytes and 2^31 elements."""
    lens, Hq, H, D = [129, 140], 2, 1, 64
    T, row = sum(lens), 1 << 23
    say("rows", row, "apart")
    q, k, v, dout = inputs(lens, Hq, H, D, 10)
    seqs = sa.Sequences.from_lists(lens)
    want = both(sa, q, k, v, dout, seqs)
    wide = torch.empty(T * row, dtype=torch.bfloat16, device="cuda").view(T, row)
    at = 0
    views = []
    for n in (Hq, H, H, Hq, Hq, H, H):
        views.append(wide[:, at:at + n * D].unflatten(1, (n, D)))
        at += n * D
    for t, x in zip(views, (q, k, v, dout)):
        t.copy_(x)
    out, lse = sa.attention_fwd(*views[:3], seqs)
    sa.attention_bwd(views[3], *views[:3], out, lse, seqs, dq=views[4], dk=views[5], dv=views[6])
    assert same((out, lse, *views[4:]), want)
