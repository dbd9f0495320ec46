"""Contiguous tensors off 16-byte boundaries through the autograd functions of the
training operators: slices of gradients, of buffers of all parameters."""
import pytest
import torch

from gpu_util import need_gpu, say
from test_gpu_self_attention import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import embedding, qk_norm, self_attention
    return embedding, qk_norm, self_attention


def off(t, elements=1):
    """t's contents in a contiguous tensor `elements` past a 16-byte boundary."""
    flat = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    view = flat[elements:].view(t.shape)
    view.copy_(t)
    assert view.is_contiguous() and view.data_ptr() % 16 != 0
    return view


@pytest.mark.parametrize("d,dtype", [(7, torch.bfloat16), (7, torch.float32), (700, torch.bfloat16)])
def test_embedding_of_pieces(mods, d, dtype):
    """torch.cat hands each piece a slice of its gradient, wherever that starts."""
    em = mods[0]
    say("pieces", d, dtype)
    layer = em.Embedding(50, d, scale=1.5, out_dtype=dtype, device="cuda")
    ids = [torch.randint(0, 50, (n,), device="cuda") for n in (3, 5)]
    dout = torch.randn(8, d, device="cuda").to(dtype)
    torch.cat([layer(i) for i in ids]).backward(dout)
    # two gradients, of sums of at most 5 rows, added: each of these 8 roundings is of 2^-24 of the magnitudes
    at = torch.cat(ids)
    want, total = (torch.zeros(50, d, dtype=torch.float64, device="cuda") for _ in range(2))
    want.index_add_(0, at, dout.double() * 1.5)
    total.index_add_(0, at, dout.double().abs() * 1.5)
    assert bool(((layer.weight.grad.double() - want).abs() <= 8 * 2.0 ** -24 * total).all())


def test_embedding_of_a_flat_buffer(mods):
    """A weight that is a view into a buffer of all parameters."""
    em = mods[0]
    table = torch.randn(40, 24, device="cuda")
    ids = torch.randint(0, 40, (6,), device="cuda")
    got = em.EmbeddingFunction.apply(ids, off(table), 1.0, torch.bfloat16)
    assert torch.equal(got, em.embedding_fwd(ids, table))


def test_head_norms_off_boundaries(mods):
    qn = mods[1]
    T, Hq, H, D = 9, 4, 2, 64
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(T, Hq + 2 * H, D, device="cuda").to(dtype)
        w = [1 + 0.1 * torch.randn(D, device="cuda") for _ in range(2)]
        dy = [torch.randn(T, n, D, device="cuda").to(torch.bfloat16) for n in (Hq, H, H)]
        grads = []
        for moved in (lambda t: t, off):
            leaves = [moved(t).detach().requires_grad_() for t in (x, *w)]
            torch.autograd.backward(qn.qk_norm_rope(leaves[0], Hq, H, *leaves[1:]), [moved(t) for t in dy])
            grads.append([t.grad for t in leaves])
        assert all(torch.equal(a, b) for a, b in zip(*grads)), dtype


def test_attention_off_boundaries(mods):
    sa = mods[2]
    seqs = sa.Sequences.from_lists([40, 25])
    tensors = [t.contiguous() for t in inputs([65], 4, 2, 64, 3)]
    results = []
    for moved in (lambda t: t, off):
        leaves = [moved(t).detach().requires_grad_() for t in tensors[:3]]
        out = sa.attention(*leaves, seqs)
        out.backward(moved(tensors[3]))
        results.append([out.detach(), *(t.grad for t in leaves)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
