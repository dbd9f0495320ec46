"""A decoder layer of the Llama 2 kind that trains on FP8-AMAX products, with
norms of its queries and keys: the norms, the products, the rotation, the
attention and the gated MLP of this package run together, and a model of such
layers from tokens to logits.

    x      = scale * table[ids]             Embedding, bf16
    h      = x + residual
    qkv    = fp8(norm(h))                   FP8NormLinear, float32
    q, k   = rotated norms of the heads     qk_norm_rope, bf16
    o      = attention(q, k, v)             attention, bf16
    a      = fp8(o)                         FP8Linear
    h      = h + a,  n = norm(h)            RMSNormFunction, bf16
    m      = mlp(n)                         FP8SwiGLUMLP
    logits = fp8(norm(m + h))               FP8NormLinear

As in decoder.py a layer returns (m, h), the next one's x and residual.  Batches
are packed sequences of any lengths (self_attention.Sequences).

A backward pass that is captured into a graph must not share leaves with an
eager one whose graph is still alive (its outputs kept): torch ties the leaves'
gradients to the stream of the older graph, and the capture fails.

Run it: python -m fp8_precision_linear_amd.block [--layers N] [--sequences N]
[--length N] [--steps N] trains on random tokens with a Llama-2-7B layer's shape
and prints the time of a step.
"""
import torch

from .decoder import need_positions, rope_tables
from .embedding import Embedding
from .linear import FP8Linear
from .mlp import FP8SwiGLUMLP
from .norm import FP8NormLinear, RMSNormFunction
from .qk_norm import qk_norm_rope
from .self_attention import Sequences, attention


class FP8Block(torch.nn.Module):
    """One layer.  qk_norm: norms of queries and keys, with a weight [head_dim]
    each.  window > 0: a token sees the last `window` positions of its sequence,
    its own among them."""

    def __init__(self, d, f, q_heads, kv_heads, head_dim, eps=1e-5, qk_norm=True, window=0, device=None):
        super().__init__()
        self.q_heads, self.kv_heads, self.head_dim, self.eps, self.window = q_heads, kv_heads, head_dim, eps, window
        self.attn_in = FP8NormLinear(d, (q_heads + 2 * kv_heads) * head_dim, eps=eps, device=device)
        one = lambda n: torch.nn.Parameter(torch.ones(n, device=device))  # noqa: E731
        self.q_norm, self.k_norm = (one(head_dim), one(head_dim)) if qk_norm else (None, None)
        self.attn_out = FP8Linear(q_heads * head_dim, d, device=device)
        self.norm_mlp = one(d)
        self.mlp = FP8SwiGLUMLP(d, f, device=device)

    def forward(self, x, residual, seqs, rope, positions=None):
        """(x, h) for the next layer; x [tokens, d], residual [tokens, d] or None
        (the first layer: x is the residual stream).  rope: (cos, sin) of
        decoder.rope_tables; positions: seqs.positions(), made here if None."""
        T, Hq, H, D = seqs.tokens, self.q_heads, self.kv_heads, self.head_dim
        need_positions(rope, min(seqs.max_len, T))   # (the bound may be a loose one)
        positions = seqs.positions() if positions is None else positions
        qkv, h = (self.attn_in(x), x) if residual is None else self.attn_in(x, residual)
        q, k, v = qk_norm_rope(qkv.view(T, Hq + 2 * H, D), Hq, H, self.q_norm, self.k_norm, self.eps, rope, positions)
        o = attention(q, k, v, seqs, window=self.window)
        n, h = RMSNormFunction.apply(self.attn_out(o.view(T, Hq * D)), h, self.norm_mlp, self.eps)
        return self.mlp(n), h


class FP8Model(torch.nn.Module):
    """Embedding, layers (their qk_norm and window: FP8Block), and the product that
    gives logits behind the last norm."""

    def __init__(self, vocab, layers, d, f, q_heads, kv_heads, head_dim, positions, eps=1e-5, qk_norm=True, embed_scale=1.0,
                 device=None, window=0):
        super().__init__()
        self.embedding = Embedding(vocab, d, scale=embed_scale, device=device)
        self.layers = torch.nn.ModuleList(FP8Block(d, f, q_heads, kv_heads, head_dim, eps, qk_norm, window, device)
                                          for _ in range(layers))
        self.head = FP8NormLinear(d, vocab, eps=eps, device=device)
        self.rope = rope_tables(positions, head_dim, device=device)

    def _apply(self, fn, *args, **kwargs):
        super()._apply(fn, *args, **kwargs)
        # the rotation's tables go where the weights go, and stay float32
        positions, half = self.rope[0].shape
        dev = fn(self.rope[0]).device
        if self.rope[0].is_meta:   # nothing to move
            self.rope = rope_tables(positions, 2 * half, device=dev)
        else:
            self.rope = tuple(t.to(dev) for t in self.rope)
        return self

    def forward(self, ids, seqs):
        """Logits float32 [tokens, vocab] of the packed sequences' tokens, whose
        ids are [tokens]."""
        if seqs.max_len > self.rope[0].shape[0]:
            raise ValueError(f"sequences up to {seqs.max_len} tokens, {self.rope[0].shape[0]} positions")
        positions = seqs.positions()
        x, h = self.embedding(ids), None
        for layer in self.layers:
            x, h = layer(x, h, seqs, self.rope, positions)
        return self.head(x) if h is None else self.head(x, h)[0]


def main(argv=None):
    import argparse
    import time

    ap = argparse.ArgumentParser(description="train on random tokens with a Llama-2-7B layer's shape")
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--length", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    vocab, dev = 32000, "cuda"
    model = FP8Model(vocab, a.layers, 4096, 11008, 32, 32, 128, a.length, device=dev)
    opt = torch.optim.SGD(model.parameters(), lr=0.1)
    seqs = Sequences.from_lists([max(1, a.length - 100 * i) for i in range(a.sequences)], device=dev)
    ids = torch.randint(0, vocab, (seqs.tokens,), device=dev)
    for step in range(a.steps + 1):
        if step == 1:     # the first one also loads and allocates
            torch.cuda.synchronize()
            start = time.perf_counter()
        loss = torch.nn.functional.cross_entropy(model(ids, seqs)[:-1], ids[1:])
        opt.zero_grad()
        loss.backward()
        opt.step()
    torch.cuda.synchronize()
    ms = (time.perf_counter() - start) / max(a.steps, 1) * 1e3
    assert bool(loss.isfinite())
    print(f"{a.layers} layers, {seqs.tokens} tokens in {a.sequences} sequences: {ms:.1f} ms a step")


if __name__ == "__main__":
    main()
