"""The decoder layer that runs the norms, the FP8 products, the cache and the
attention together, against the same layer in float64 from the definitions.

Bound: every product's operands are rounded to E4M3 (half a step: 2^-4 of a
value, 2^-5 rms at the worst place of a binade), as are the cached keys and
values.  Errors of single elements are independent, so a product's output is
off by about sqrt(2) 2^-5 / sqrt(3) = 2.6% of its norm, and the layer's output
by a few of these together: 10% of its norm is asked, and that a prompt taken
whole, in chunks and token by token agree to the same."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    need_gpu()
    from fp8_precision_linear_amd import attention, decoder
    return attention, decoder


D_MODEL, F, HQ, H, D = 512, 768, 8, 2, 64


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).cuda()  # noqa: E731
    return dict(norm_attn=1 + 0.1 * torch.randn(D_MODEL, generator=g).cuda(), wqkv=r((HQ + 2 * H) * D, D_MODEL),
                wo=r(D_MODEL, HQ * D), norm_mlp=1 + 0.1 * torch.randn(D_MODEL, generator=g).cuda(),
                w_gate_up=r(2 * F, D_MODEL), w_down=r(D_MODEL, F))


def reference(w, x, eps=1e-5):
    """The layer over one whole sequence x [T, d], float64: x + attention + MLP."""
    w = {k: v.double() for k, v in w.items()}
    x = x.double()
    norm = lambda t, g: t * (t.square().mean(1, keepdim=True) + eps).rsqrt() * g  # noqa: E731
    T = x.shape[0]
    qkv = (norm(x, w["norm_attn"]) @ w["wqkv"].t()).view(T, HQ + 2 * H, D)
    inv = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    ang = torch.arange(T, device="cuda", dtype=torch.float64)[:, None] * inv
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    turn = lambda t: torch.cat((t[..., :D // 2] * c - t[..., D // 2:] * s,  # noqa: E731
                                t[..., D // 2:] * c + t[..., :D // 2] * s), -1)
    q, k, v = turn(qkv[:, :HQ]), turn(qkv[:, HQ:HQ + H]), qkv[:, HQ + H:]
    k, v = (t.repeat_interleave(HQ // H, 1).transpose(0, 1).contiguous() for t in (k, v))
    sc = torch.matmul(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) * D ** -0.5
    sc = sc.masked_fill(torch.ones(T, T, device="cuda", dtype=torch.bool).triu(1), -torch.inf)
    o = torch.matmul(sc.softmax(-1), v).transpose(0, 1).reshape(T, HQ * D)
    h = x + o @ w["wo"].t()
    g = norm(h, w["norm_mlp"]) @ w["w_gate_up"].t()
    g, u = g[:, :F], g[:, F:]
    return h + (g * torch.sigmoid(g) * u) @ w["w_down"].t()


def run(mods, w, seqs, steps):
    """Outputs x + h of every sequence, its tokens taken `steps` at a time."""
    fa, dec = mods
    layer = dec.FP8DecoderLayer(**w, q_heads=HQ, kv_heads=H, head_dim=D)
    per = -(-max(len(s) for s in seqs) // 64)
    cache = layer.cache(per * len(seqs))
    tables = [list(range(i * per, (i + 1) * per)) for i in range(len(seqs))]
    rope = dec.rope_tables(max(len(s) for s in seqs), D)
    done, outs = [0] * len(seqs), [[] for _ in seqs]
    while any(a < len(s) for a, s in zip(done, seqs)):
        new = [min(steps, len(s) - a) for a, s in zip(done, seqs)]
        x = torch.cat([s[a:a + n] for s, a, n in zip(seqs, done, new)])
        done = [a + n for a, n in zip(done, new)]
        batch = fa.KVBatch.from_lists(new, done, tables)
        y, h = layer(x, torch.zeros_like(x), cache, batch, rope)
        at = 0
        for o, n in zip(outs, new):
            o.append(y[at:at + n].double() + h[at:at + n].double())
            at += n
    return [torch.cat(o) for o in outs]


def test_layer(mods):
    w = weights(3)
    g = torch.Generator().manual_seed(5)
    seqs = [torch.randn(n, D_MODEL, generator=g).to(torch.bfloat16).cuda() for n in (130, 37, 1)]
    want = [reference(w, s) for s in seqs]
    outs = {steps: run(mods, w, seqs, steps) for steps in (200, 48, 1)}
    for steps, got in outs.items():
        for a, b, s in zip(got, want, seqs):
            # of what the layer adds to its input
            rel = ((a - b).norm() / (b - s.double()).norm()).item()
            assert rel < 0.1, (steps, len(s), rel)


def test_decoder_command(mods, capsys):
    _, dec = mods
    dec.main(["--layers", "1", "--sequences", "2", "--prompt", "70", "--tokens", "3"])
    assert "ms a token" in capsys.readouterr().out
