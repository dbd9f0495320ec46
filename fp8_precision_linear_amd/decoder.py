"""A decoder layer of the Llama 2 kind served with FP8-AMAX products: the norms,
the cache, the attention and the gated MLP of this package run together.

    h  = x + residual                       rmsnorm_quantize -> codes
    q, k, v = h8 . wqkv^T                   scaled_gemm, float32
    q, k <- norms of the heads, rotated     qk_norm_rope_fwd, where the layer has them
    q  <- rotated; k, v -> the FP8 cache    kv_append
    o  = attention(q, cache)                kv_attention, bf16
    a  = o8 . wo^T                          quantize, scaled_gemm
    h  = h + a                              rmsnorm_quantize -> codes
    g  = h8 . w_gate_up^T, silu(g) u        scaled_gemm, swiglu_fwd
    m  = a8 . w_down^T                      scale_cast, scaled_gemm

The layer returns (m, h): the next layer's x and residual, so that every
addition happens in the norm that follows it, and a product's fp32 output is
read once.  Prompts, chunks of prompts and single tokens are one call: the
batch says which tokens are new.  Weights are quantised once, at construction
(post-training quantisation); activations with current scaling.

Run it: python -m fp8_precision_linear_amd.decoder [--layers N] [--tokens N]
decodes with random weights of a Llama-2-7B layer's shape and prints the time
of a step.
"""
import torch

from . import E4M3, OP_FWD, compute_bias, quantize, scale_cast, scaled_gemm_auto, swiglu_fwd
from .attention import KVBatch, KVCache, kv_append, kv_attention
from .embedding import embedding_fwd
from .norm import rmsnorm_fwd, rmsnorm_quantize
from .qk_norm import qk_norm_rope_fwd


def rope_tables(positions, head_dim, base=10000.0, device="cuda"):
    """(cos, sin) float32 [positions, head_dim / 2] of rotary positions."""
    inv = base ** (-torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def need_positions(rope, most):
    """Refuses tables with fewer than `most` positions (the rotation alone would
    turn every later token as the last)."""
    if rope is not None and rope[0].shape[0] < most:
        raise ValueError(f"the rotation's tables hold {rope[0].shape[0]} positions, the sequences up to {most}")


class FP8DecoderLayer:
    """Weights: wqkv [(q_heads + 2 kv_heads) head_dim, d], wo [d, q_heads
    head_dim], w_gate_up [2f, d], w_down [d, f]; norm weights [d].  q_norm, k_norm
    [head_dim], both or neither: the norms of queries and keys.  window > 0: a
    token sees the last `window` positions, its own among them."""

    def __init__(self, norm_attn, wqkv, wo, norm_mlp, w_gate_up, w_down, q_heads, kv_heads, head_dim, eps=1e-5,
                 q_norm=None, k_norm=None, window=0):
        d = norm_attn.shape[0]
        if wqkv.shape != ((q_heads + 2 * kv_heads) * head_dim, d) or wo.shape != (d, q_heads * head_dim):
            raise ValueError(f"wqkv {tuple(wqkv.shape)} and wo {tuple(wo.shape)} do not fit {q_heads} + 2 * {kv_heads} "
                             f"heads of {head_dim} and d = {d}")
        if w_gate_up.dim() != 2 or w_gate_up.shape[1] != d or w_down.shape != (d, w_gate_up.shape[0] // 2):
            raise ValueError(f"w_gate_up {tuple(w_gate_up.shape)} and w_down {tuple(w_down.shape)} do not chain")
        self.q_heads, self.kv_heads, self.head_dim, self.eps, self.window = q_heads, kv_heads, head_dim, eps, window
        self.norm_attn, self.norm_mlp = norm_attn, norm_mlp
        if (q_norm is None) != (k_norm is None):
            raise ValueError("norm weights for both queries and keys, or for neither")
        self.q_norm, self.k_norm = q_norm, k_norm
        # codes and biases, made once
        self.wqkv, self.wo, self.w_gate_up, self.w_down = (
            quantize(w.contiguous(), E4M3)[:2] for w in (wqkv, wo, w_gate_up, w_down))

    @classmethod
    def random(cls, d, f, q_heads, kv_heads, head_dim, device="cuda", std=0.02):
        w = lambda *shape: torch.randn(*shape, device=device, dtype=torch.bfloat16) * std  # noqa: E731
        one = torch.ones(d, device=device)
        return cls(one, w((q_heads + 2 * kv_heads) * head_dim, d), w(d, q_heads * head_dim), one.clone(), w(2 * f, d),
                   w(d, f), q_heads, kv_heads, head_dim)

    def cache(self, num_blocks, block_size=64, fmt=E4M3, device="cuda"):
        return KVCache(num_blocks, self.kv_heads, self.head_dim, block_size, fmt, device)

    @classmethod
    def from_block(cls, block):
        """The layer that serves what block.FP8Block trained."""
        w = lambda t: None if t is None else t.detach()  # noqa: E731
        return cls(w(block.attn_in.norm_weight), w(block.attn_in.weight), w(block.attn_out.weight), w(block.norm_mlp),
                   w(block.mlp.w1), w(block.mlp.w2), block.q_heads, block.kv_heads, block.head_dim, block.eps,
                   w(block.q_norm), w(block.k_norm), block.window)

    @torch.no_grad()
    def forward(self, x, residual, cache, batch, rope, window=None, positions=None):
        """(x, h) for the next layer; x [tokens, d] float32 or bf16, residual
        [tokens, d] bf16 or None (the first layer: x is the residual stream).
        window: in place of the layer's own (0: none).  positions:
        batch.positions(), made here if None; a layer with norms of queries and
        keys asks for it."""
        T, Hq, H, D = batch.tokens, self.q_heads, self.kv_heads, self.head_dim
        need_positions(rope, batch.max_len)
        n8, bn, _, h, _ = rmsnorm_quantize(x, self.norm_attn, E4M3, residual=residual, eps=self.eps)
        qkv = scaled_gemm_auto(OP_FWD, n8, E4M3, bn, self.wqkv[0], E4M3, self.wqkv[1]).view(T, Hq + 2 * H, D)
        if self.q_norm is None:
            q = kv_append(cache, batch, qkv[:, Hq:Hq + H], qkv[:, Hq + H:], q=qkv[:, :Hq], rope=rope)
        else:
            positions = batch.positions() if positions is None else positions
            # (keys and values reach the cache in bf16: 2^-8 beside the 2^-4 of their codes)
            q, k, v = qk_norm_rope_fwd(qkv, Hq, H, self.q_norm, self.k_norm, self.eps, rope, positions)
            kv_append(cache, batch, k, v)
        o = kv_attention(cache, batch, q, window=self.window if window is None else window).view(T, Hq * D)
        o8, bo, _ = quantize(o, E4M3)
        a = scaled_gemm_auto(OP_FWD, o8, E4M3, bo, self.wo[0], E4M3, self.wo[1])
        n8, bn, _, h, _ = rmsnorm_quantize(a, self.norm_mlp, E4M3, residual=h, eps=self.eps)
        g = scaled_gemm_auto(OP_FWD, n8, E4M3, bn, self.w_gate_up[0], E4M3, self.w_gate_up[1])
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
        s = swiglu_fwd(g, amax=amax)
        bs = compute_bias(amax, E4M3)
        s8 = scale_cast(s, bs, E4M3)
        return scaled_gemm_auto(OP_FWD, s8, E4M3, bs, self.w_down[0], E4M3, self.w_down[1]), h

    __call__ = forward


class FP8Decoder:
    """Layers and their caches over one block table, with a final norm.
    embedding: optional [vocab, d] table; forward then also takes token ids."""

    def __init__(self, layers, norm_weight, num_blocks, positions, block_size=64, fmt=E4M3, eps=1e-5, embedding=None,
                 embed_scale=1.0):
        self.layers, self.norm_weight, self.eps = list(layers), norm_weight, eps
        dev = norm_weight.device
        self.caches = [l.cache(num_blocks, block_size, fmt, dev) for l in self.layers]
        self.block_size = block_size
        self.rope = rope_tables(positions, self.layers[0].head_dim, device=dev)
        self.embedding, self.embed_scale = embedding, embed_scale

    @torch.no_grad()
    def forward(self, x, batch):
        """Final hidden states [tokens, d] bf16 of the batch's new tokens, whose
        embeddings are x [tokens, d] bf16, or whose ids are x [tokens] int32 or
        int64; the caches receive their keys and values."""
        if x.dim() == 1:
            if self.embedding is None:
                raise ValueError("token ids for a decoder without an embedding")
            x = embedding_fwd(x, self.embedding, self.embed_scale)
        h = None
        normed = any(getattr(l, "q_norm", None) is not None for l in self.layers)
        more = {"positions": batch.positions()} if normed else {}   # made once for all of them
        for layer, cache in zip(self.layers, self.caches):
            x, h = layer(x, h, cache, batch, self.rope, **more)
        return rmsnorm_fwd(x, self.norm_weight, residual=h, eps=self.eps)[0]

    __call__ = forward


def main(argv=None):
    import argparse
    import time

    ap = argparse.ArgumentParser(description="decode with random weights of a Llama-2-7B layer's shape")
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args(argv)
    d, f, heads, D = 4096, 11008, 32, 128
    torch.manual_seed(0)
    layers = [FP8DecoderLayer.random(d, f, heads, heads, D) for _ in range(a.layers)]
    per = -(-(a.prompt + a.tokens) // 64)
    model = FP8Decoder(layers, torch.ones(d, device="cuda"), per * a.sequences, a.prompt + a.tokens)
    tables = [list(range(i * per, (i + 1) * per)) for i in range(a.sequences)]
    embed = lambda n: torch.randn(n, d, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    lens = [a.prompt] * a.sequences
    out = model(embed(sum(lens)), KVBatch.from_lists(lens, lens, tables))
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.tokens):
        lens = [n + 1 for n in lens]
        out = model(embed(a.sequences), KVBatch.from_lists([1] * a.sequences, lens, tables))
    torch.cuda.synchronize()
    ms = (time.perf_counter() - start) / a.tokens * 1e3
    assert bool(out.isfinite().all())
    print(f"{a.layers} layers, {a.sequences} sequences of {lens[0]} tokens: {ms:.2f} ms a token")


if __name__ == "__main__":
    main()
