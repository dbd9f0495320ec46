"""The embedding's gradient past 16384 tokens, where tokens are sorted tile by
tile: both types of rows and of ids, scales, added gradients, ids that are no
tokens, rows of odd lengths, workspaces that held something else.

Bound: test_gpu_embedding.py's.  An id's m rows are added in fp32 in at most
m - 1 additions, each off by 2^-24 of a partial sum: (m - 1) 2^-24 S, enlarged
by 1 + 2^-6 for second order terms (m 2^-24 is at most 2^-8 here); the scale
rounds the result once, and an addition to what is there once more.  The
reference multiplies by what the library's float argument holds: -1.7 in fp32 is
-1.7000000477, 2^-25.1 of it off, which beside the product's own 2^-24 would pass
the bound of an id with one row."""
import pytest
import torch

from gpu_util import need_gpu, say
from test_gpu_embedding import TINY, TYPES, make_ids

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def em():
    need_gpu()
    from fp8_precision_linear_amd import embedding
    return embedding


def reference(dout, ids, vocab, scale):
    """(sum, sum of magnitudes, rows) of each id, float64, added on the host: the
    device's additions to a few ids wait for one another."""
    ids, rows = ids.cpu().long(), dout.cpu().double()
    there = (ids >= 0) & (ids < vocab)
    at, rows = ids[there], rows[there]
    out = torch.zeros(vocab, dout.shape[1], dtype=torch.float64)
    total, count = torch.zeros_like(out), torch.zeros(vocab, dtype=torch.float64)
    out.index_add_(0, at, rows)
    total.index_add_(0, at, rows.abs())
    count.index_add_(0, at, torch.ones(at.shape[0], dtype=torch.float64))
    return (out * scale).cuda(), (total * abs(scale)).cuda(), count[:, None].cuda()


@pytest.mark.parametrize("kind", ["random", "few", "text", "one", "none"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("ids_t", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,vocab,d", [(16385, 511, 7), (33000, 700, 12), (40001, 131073, 5)])
def test_gradient(em, kind, dt, ids_t, n, vocab, d):
    """One, two and two digits of the ids (the largest of them: one past 2^17)."""
    say("tiles", kind, dt, ids_t, n, vocab, d)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    dout = torch.randn(n, d, generator=g, device="cuda").to(TYPES[dt])
    ids = make_ids(kind, n, vocab, ids_t)
    scale = -1.7
    want, total, count = reference(dout, ids, vocab, torch.tensor(scale, dtype=torch.float32).item())
    bound = 2.0 ** -24 * ((count - 1).clamp(min=0) * total * (1 + 2.0 ** -6) + want.abs()) * (1 + 2.0 ** -6) + TINY
    ws = torch.full((em.embedding_bwd_workspace_bytes(n, vocab, d),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((vocab, d), 9.0, device="cuda")
    em.embedding_bwd(dout, ids, vocab, scale=scale, out=out, workspace=ws)
    assert bool(((out.double() - want).abs() <= bound).all())
    old = torch.randn(vocab, d, generator=g, device="cuda")
    acc = old.clone()
    em.embedding_bwd(dout, ids, vocab, scale=scale, out=acc, accumulate=True, workspace=ws)
    none = count[:, 0] == 0
    assert torch.equal(acc[none], old[none])
    # (the old value and the sum, which is off by `bound`, added: one rounding of what results)
    off = (acc.double() - (old.double() + want)).abs()
    assert bool((off <= bound + 2.0 ** -24 * ((old.double() + want).abs() + bound)).all())
    assert torch.equal(em.embedding_bwd(dout, ids, vocab, scale=scale), out)


def test_training_step_of_many_tokens(em):
    """Through the module, whole rows of bf16."""
    n, vocab, d = 32768, 3000, 256
    torch.manual_seed(2)
    layer = em.Embedding(vocab, d, scale=16.0, device="cuda")
    ids = make_ids("text", n, vocab, torch.int64).view(16, n // 16)
    dout = torch.randn(*ids.shape, d, device="cuda").to(torch.bfloat16)
    layer(ids).backward(dout)
    want, total, count = reference(dout.view(n, d), ids.view(n), vocab, 16.0)
    bound = 2.0 ** -24 * (count * total * (1 + 2.0 ** -6) + want.abs()) + TINY
    assert bool(((layer.weight.grad.double() - want).abs() <= bound).all())
