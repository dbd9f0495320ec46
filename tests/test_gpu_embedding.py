"""Embedding and its gradient against their 64-bit forms.

Bounds.  Lookup: one fp32 product (2^-24 of the value), one rounding to the
output's type (2^-8 in bf16, none of its own in fp32).  Gradient: an id's rows
are added in fp32 in some order, at most m = (its number of rows) - 1 additions
each off by 2^-24 of a partial sum, which no sum of magnitudes S passes: m 2^-24 S,
and 2^-24 of the result for the scale (2^-23 with `accumulate`, whose addition
rounds once more, of the sum's and the old value's magnitudes)."""
import pytest
import torch

from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def em():
    need_gpu()
    from fp8_precision_linear_amd import embedding
    return embedding


def make_ids(kind, n, vocab, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "random":
        ids = torch.randint(0, vocab, (n,), generator=g)
    elif kind == "one":
        ids = torch.full((n,), vocab - 1)
    elif kind == "few":      # long runs of a few ids, and padding
        ids = torch.randint(0, 3, (n,), generator=g) * ((vocab - 1) // 2)
        ids[torch.rand(n, generator=g) < 0.2] = -1
    elif kind == "text":
        ids = ((vocab + 1) ** torch.rand(n, generator=g, dtype=torch.float64)).long().clamp(max=vocab) - 1
    else:                    # nothing that is a token
        ids = torch.where(torch.rand(n, generator=g) < 0.5, -7, vocab)
    return ids.to(dtype).cuda()


@pytest.mark.parametrize("table_t", list(TYPES))
@pytest.mark.parametrize("out_t", list(TYPES))
@pytest.mark.parametrize("n,vocab,d", [(1, 1, 1), (3, 50, 7), (65, 300, 768), (1000, 97, 1027), (5, 11, 4096)])
def test_lookup(em, table_t, out_t, n, vocab, d):
    say("lookup", table_t, out_t, n, vocab, d)
    g = torch.Generator(device="cuda").manual_seed(n)
    table = torch.randn(vocab, d, generator=g, device="cuda").to(TYPES[table_t])
    for kind, dtype, scale in (("random", torch.int64, 1.0), ("few", torch.int32, 1.7), ("none", torch.int64, 1.0)):
        ids = make_ids(kind, n, vocab, dtype)
        got = em.embedding_fwd(ids, table, scale=scale, dtype=TYPES[out_t]).double()
        there = (ids >= 0) & (ids < vocab)
        want = torch.where(there[:, None], table.double()[ids.clamp(0, vocab - 1).long()] * scale, 0.0)
        half = 2.0 ** -24 + (2.0 ** -8 * (1 + 2.0 ** -20) if out_t == "bf16" else 2.0 ** -24)
        assert bool(((got - want).abs() <= half * want.abs()).all()), kind
        if kind == "none":
            assert not got.any()


def reference(dout, ids, vocab, scale):
    """(sum, sum of magnitudes, rows) of each id, float64."""
    there = (ids >= 0) & (ids < vocab)
    at, rows = ids[there].long(), dout[there].double()
    out = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device="cuda")
    total, count = torch.zeros_like(out), torch.zeros(vocab, dtype=torch.float64, device="cuda")
    out.index_add_(0, at, rows)
    total.index_add_(0, at, rows.abs())
    count.index_add_(0, at, torch.ones(at.shape[0], dtype=torch.float64, device="cuda"))
    return out * scale, total * abs(scale), count[:, None]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("kind", ["random", "one", "few", "text", "none"])
@pytest.mark.parametrize("n,vocab,d", [(1, 1, 1), (31, 513, 7), (33, 40, 768), (1000, 511, 1030), (2048, 50257, 96)])
def test_gradient(em, dt, kind, n, vocab, d):
    say("gradient", dt, kind, n, vocab, d)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    dout = torch.randn(n, d, generator=g, device="cuda").to(TYPES[dt])
    ids = make_ids(kind, n, vocab, torch.int32 if n % 2 else torch.int64)
    want, total, count = reference(dout, ids, vocab, 1.5)
    out = torch.full((vocab, d), 9.0, device="cuda")
    em.embedding_bwd(dout, ids, vocab, scale=1.5, out=out)
    bound = 2.0 ** -24 * ((count - 1).clamp(min=0) * total * (1 + 2.0 ** -10) + want.abs()) + TINY
    assert bool(((out.double() - want).abs() <= bound).all())
    again = em.embedding_bwd(dout, ids, vocab, scale=1.5)
    assert torch.equal(out, again)
    # added to what is there; rows without tokens keep their bits
    old = torch.randn(vocab, d, generator=g, device="cuda")
    acc = old.clone()
    em.embedding_bwd(dout, ids, vocab, scale=1.5, out=acc, accumulate=True)
    assert torch.equal(acc[count[:, 0] == 0], old[count[:, 0] == 0])
    off = (acc.double() - (old.double() + want)).abs()
    assert bool((off <= bound + 2.0 ** -24 * (old.double() + want).abs() + 2.0 ** -46 * total).all())


@pytest.mark.parametrize("n,vocab", [(16384, 32000), (16385, 700), (50000, 300000)])
def test_gradient_of_many_tokens(em, n, vocab):
    """The last size of the one-workgroup sort, and tiles of it."""
    say("many tokens", n, vocab)
    d = 20
    g = torch.Generator(device="cuda").manual_seed(n)
    dout = torch.randn(n, d, generator=g, device="cuda")
    for kind in ("text", "few", "one"):
        ids = make_ids(kind, n, vocab, torch.int64)
        want, total, count = reference(dout, ids, vocab, 1.0)
        got = em.embedding_bwd(dout, ids, vocab).double()
        bound = 2.0 ** -24 * ((count - 1).clamp(min=0) * total * (1 + 2.0 ** -6) + want.abs()) + TINY
        assert bool(((got - want).abs() <= bound).all()), kind


@pytest.mark.parametrize("n", [8192, 8193, 9215, 9216, 20003])
def test_long_runs(em, n):
    """Runs that fill spans of chunks, begin and end inside them, next to short
    ones; rows of an odd length."""
    say("long runs", n)
    d, vocab = 7, 6
    g = torch.Generator(device="cuda").manual_seed(n)
    dout = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
    for cuts in ([n], [1, n], [1023, n - 17], [15, 1024, 2 * 1024 + 1, n - 1024], [n // 3, n // 3 + 1, n // 2]):
        ids = torch.zeros(n, dtype=torch.int32)
        for c in cuts:
            ids[c:] += 1
        ids = ids[torch.randperm(n, generator=torch.Generator().manual_seed(1))].cuda()
        want, total, count = reference(dout, ids, vocab, 1.0)
        got = em.embedding_bwd(dout, ids, vocab).double()
        bound = 2.0 ** -24 * ((count - 1).clamp(min=0) * total * (1 + 2.0 ** -10) + want.abs()) + TINY
        assert bool(((got - want).abs() <= bound).all()), cuts


def test_no_tokens(em):
    out = torch.full((5, 8), 3.0, device="cuda")
    em.embedding_bwd(torch.empty(0, 8, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 5, out=out)
    assert not out.any()
    assert em.embedding_fwd(torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.ones(4, 8, device="cuda")).shape == (0, 3, 8)
    none = em.embedding_bwd(torch.ones(3, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"), 0)
    assert none.shape == (0, 8)


def test_row_order_is_the_tokens(em):
    """Rows whose sum depends on the order: the tokens' own, chunk by chunk."""
    n = 20
    dout = torch.tensor([2.0 ** 24, 1.0] * (n // 2), device="cuda")[:, None].repeat(1, 4)
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    got = em.embedding_bwd(dout, ids, 2)
    s = torch.zeros(4)
    for row in dout.cpu():
        s = s + row
    assert torch.equal(got[0].cpu(), s)


def test_module(em):
    """The layer trains: its gradient is that of 64-bit indexing."""
    torch.manual_seed(1)
    layer = em.Embedding(40, 24, scale=3.0, device="cuda")
    ids = torch.randint(0, 40, (6, 9), device="cuda")
    ids[2, 3:] = -1
    out = layer(ids)
    assert out.shape == (6, 9, 24) and out.dtype == torch.bfloat16
    dout = torch.randn(6, 9, 24, device="cuda").to(torch.bfloat16)
    out.backward(dout)
    want, total, count = reference(dout.reshape(-1, 24), ids.reshape(-1), 40, 3.0)
    assert bool(((layer.weight.grad.double() - want).abs() <= 2.0 ** -24 * (count * total + want.abs()) + TINY).all())


def test_another_stream(em):
    side = torch.cuda.Stream()
    ids = make_ids("text", 700, 1000, torch.int64)
    dout = torch.randn(700, 64, device="cuda")
    want = em.embedding_bwd(dout, ids, 1000)
    side.wait_stream(torch.cuda.current_stream())
    got = em.embedding_bwd(dout, ids, 1000, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_graph(em):
    """Lookup and gradient captured, for the sort of one workgroup and that of
    tiles; replays on new ids, with eager calls between them, give their bits."""
    for n, vocab, d in ((700, 1000, 64), (20000, 500, 20)):
        ids = make_ids("text", n, vocab, torch.int64)
        table, dout = torch.randn(vocab, d, device="cuda"), torch.randn(n, d, device="cuda")
        em.embedding_bwd(dout, ids, vocab)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = (em.embedding_fwd(ids, table, dtype=torch.float32), em.embedding_bwd(dout, ids, vocab))
        for r, kind in enumerate(("few", "one", "random")):
            ids.copy_(make_ids(kind, n, vocab, torch.int64, seed=r))
            want = (em.embedding_fwd(ids, table, dtype=torch.float32), em.embedding_bwd(dout, ids, vocab))
            torch.cuda.synchronize()
            for t in outs:
                t.fill_(3)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), kind


def test_two_calls_at_once(em):
    ids = [make_ids("text", 20000, 700, torch.int64, seed=s) for s in range(2)]
    dout = torch.randn(20000, 96, device="cuda")
    want = [em.embedding_bwd(dout, i, 700) for i in ids]
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [em.embedding_bwd(dout, i, 700, stream=s) for _ in range(2) for i, s in zip(ids, sides)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want * 2))


def test_offsets_past_32_bits(em):
    """A table, and rows of tokens, of more than 2^31 elements."""
    d, vocab = 8192, (1 << 18) + 100
    say("table of", vocab, "rows of", d)
    table = torch.empty(vocab, d, dtype=torch.bfloat16, device="cuda")
    table[-3:] = torch.randn(3, d, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([vocab - 3, vocab - 1, vocab, vocab - 2, vocab - 1], device="cuda")
    got = em.embedding_fwd(ids, table)
    assert torch.equal(got[[0, 1, 3, 4]], table[[vocab - 3, vocab - 1, vocab - 2, vocab - 1]]) and not got[2].any()
    del table
    dout = torch.randn(5, d, device="cuda")
    grad = em.embedding_bwd(dout, ids, vocab)
    assert torch.equal(grad[vocab - 3:], torch.stack((dout[0], dout[3], dout[1] + dout[4])))
    assert not grad[:vocab - 3].any()
    del grad
    many = torch.full((vocab,), -1, dtype=torch.int64, device="cuda")   # tokens: all but some are none
    many[-2:] = torch.tensor([5, 9], device="cuda")
    small = torch.randn(10, d, device="cuda").to(torch.bfloat16)
    out = em.embedding_fwd(many, small)
    assert torch.equal(out[-2:], small[[5, 9]]) and not out[:-2].any()
    out[-2:] = 1.0
    grad = em.embedding_bwd(out, many, 10)
    assert bool((grad[[5, 9]] == 1.0).all()) and not grad[:5].any()
