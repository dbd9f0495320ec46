"""Measured cases of the operators that a transformer on FP8 products trains
with: the embedding at its start, the norms of queries and keys with the
rotation, and attention over packed sequences, each with its gradient.

Operators (formulas: include/fp8lin_train.h)
  embed       out[t] = scale * table[id[t]]
  embed_grad  dtable[v] = scale * sum of dout[t] over the t with id[t] = v
  qk          queries and keys of the fused product's rows, normed for each head
              and rotated by their position, values beside them, in bf16
  qk_grad     gradients of the fused rows and of the two norm weights
  attn        softmax attention of packed sequences, grouped heads, causal or
              not, optionally in a window; out and lse
  attn_grad   dq, dk, dv from dout, out and lse

Shapes are those of GPT-111M (d 768, 12 heads of 64, 50257 tokens), Llama-2-7B
(4096, 32 heads of 128, 32000 tokens), 13B (5120, 40 heads) and 70B (8192, 64
query and 8 key heads).  With `own` false the operators are computed by
elementary torch operations in fp32; with `own` true by the framework's kernels.
"""
import math
import random

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ cases
def _embed(name, op, tokens, vocab, d, x="bf16", scale=1.0, pad=0):
    """x: the table's type (embed) or dout's (embed_grad); pad: rows of padding at the end (id -1)."""
    return {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "d": d, "x": x, "scale": scale, "pad": pad}


def _qk(name, op, tokens, q_heads, kv_heads, head_dim, x="fp32", rope="halves", norm=True, positions=4096):
    return {"name": name, "op": op, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "x": x, "rope": rope, "norm": norm, "positions": positions}


def _attn(name, op, batch, q_heads, kv_heads, head_dim, lo, hi, causal=True, window=0, pattern=1):
    """lo..hi tokens a sequence."""
    return {"name": name, "op": op, "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "lo": lo, "hi": hi, "causal": causal, "window": window, "pattern": pattern}


def listed():
    return [
        # one decoded token for each of four 7B conversations: latency
        _embed("embed 7B, 4 tokens", "embed", 4, 32000, 4096),
        # a prompt's 8192 tokens of the 70B model, an fp32 master table
        _embed("embed 70B, 8192 tokens", "embed", 8192, 32000, 8192, x="fp32"),
        # the GPT-111M training step's 2048 tokens, scaled embeddings
        _embed("embed gradient 111M", "embed_grad", 2048, 50257, 768, scale=768 ** 0.5),
        # the 13B backward workload's 4096 tokens, one short of even and 100 of them padding
        _embed("embed gradient 13B", "embed_grad", 4095, 32000, 5120, x="fp32", pad=100),
        # a served batch: one token for each of 8 70B conversations
        _qk("qk norm 70B, 8 tokens", "qk", 8, 64, 8, 128),
        # the 70B layer's 8192 tokens
        _qk("qk norm 70B, 8192 tokens", "qk", 8192, 64, 8, 128),
        # the GPT-111M training step
        _qk("qk norm gradient 111M", "qk_grad", 2048, 12, 12, 64, rope="pairs"),
        # the 13B backward workload
        _qk("qk norm gradient 13B", "qk_grad", 4095, 40, 40, 128),
        # the GPT-111M training step: two sequences of 1024
        _attn("attention 111M, 2 x 1024", "attn", 2, 12, 12, 64, 1024, 1024),
        # four packed documents of different length through the 7B layer
        _attn("attention 7B, 4 documents", "attn", 4, 32, 32, 128, 700, 4000),
        # the GPT-111M training step's gradient
        _attn("attention grad 111M", "attn_grad", 2, 12, 12, 64, 1024, 1024),
        # two long documents of the 70B layer, eight query heads on each key head
        _attn("attention grad 70B", "attn_grad", 2, 64, 8, 128, 3500, 4096),
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over lo..hi by its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "qk", "qk_grad", "attn", "attn", "attn_grad", "attn_grad"))
    if op in ("embed", "embed_grad"):
        d = rng.choice((768, 1024, 2048, 4096, 5120, 8 * rng.randint(90, 1024), rng.randint(700, 5119)))
        vocab = rng.choice((256, 32000, 50257, rng.randint(1000, 60000)))
        if op == "embed_grad":
            vocab = min(vocab, 32000 * 5120 // d)
        tokens = _log_int(rng, 1, 8000)
        c = _embed("", op, tokens, vocab, d, rng.choice(("fp32", "bf16")), rng.choice((1.0, d ** 0.5)),
                   rng.choice((0, 0, tokens // 10)))
    elif op in ("qk", "qk_grad"):
        heads = rng.choice(((12, 12, 64), (32, 32, 128), (40, 40, 128), (64, 8, 128), (32, 8, 64), (16, 1, 128),
                            (16, 4, 256)))
        most = 8192 * 80 * 128 if op == "qk" else 4095 * 120 * 128
        tokens = _log_int(rng, 1, min(12000, most // ((heads[0] + 2 * heads[1]) * heads[2]) // 2))
        c = _qk("", op, tokens, *heads, rng.choice(("fp32", "fp32", "bf16")), rng.choice(("none", "halves", "pairs")),
                rng.random() < 0.8, rng.choice((512, 4096, 20000)))
    else:
        heads = rng.choice(((12, 12, 64), (32, 32, 128), (40, 40, 128), (64, 8, 128), (32, 8, 64), (16, 1, 128),
                            (16, 4, 256)))
        # pairs of the largest listed case of the operator: a drawn one has at most a third of its work
        batch = _log_int(rng, 1, 24)
        hi = _log_int(rng, 1, min(4000, int(4000 * (32 / (heads[0] * heads[2] / 128) / batch) ** 0.5)))
        causal = rng.random() < 0.75
        c = _attn("", op, batch, *heads, rng.choice((0, hi // 4, hi)), hi, causal,
                  rng.choice((0, 0, rng.randint(1, 2000))) if causal else 0, rng.randint(1, 1 << 20))
    del c["name"]
    return c


def _lengths(case):
    """Tokens of each sequence: from the case alone; one at least in all."""
    r = random.Random(case["pattern"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    n[0] = max(n[0], 1)
    return n


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _tokens(case, g):
    """Token ids with the frequencies of a text: the n-th most frequent token
    about 1 / n as often as the first; the last `pad` of them padding."""
    u = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(case["vocab"] + 1)) - 1).long().clamp_(0, case["vocab"] - 1)
    ids = torch.randperm(case["vocab"], generator=g, device="cuda")[rank]
    if case["pad"]:
        ids[-case["pad"]:] = -1
    return ids


def _angles(positions, head_dim):
    inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("embed", "embed_grad"):
        s["ids"] = _tokens(case, g)
        if op == "embed":
            s["table"] = _normal(g, case["vocab"], case["d"], std=0.02).to(_dtype(case["x"]))
        else:
            s["dout"] = _normal(g, case["tokens"], case["d"], std=1e-2).to(_dtype(case["x"]))
        return s
    Hq, H, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op in ("qk", "qk_grad"):
        T = case["tokens"]
        # the fused query / key / value product's rows
        s["qkv"] = _normal(g, T, Hq + 2 * H, D).to(_dtype(case["x"]))
        s["wq"] = s["wk"] = s["rope"] = None
        if case["norm"]:
            s["wq"], s["wk"] = 1.0 + _normal(g, D, std=0.1), 1.0 + _normal(g, D, std=0.1)
        s["positions"] = torch.randint(0, case["positions"], (T,), generator=g, device="cuda", dtype=torch.int32)
        if case["rope"] != "none":
            s["rope"] = _angles(case["positions"], D)
        if op == "qk_grad":
            s["dq"], s["dk"], s["dv"] = (_normal(g, T, n, D, std=1e-2).to(torch.bfloat16) for n in (Hq, H, H))
        return s
    n = _lengths(case)
    T = sum(n)
    cu = [0]
    for a in n:
        cu.append(cu[-1] + a)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["tokens"], s["longest"] = T, max(n)
    # queries, keys and values side by side in a token's row
    s["qkv"] = _normal(g, T, Hq + 2 * H, D).to(torch.bfloat16)
    if op == "attn_grad":
        s["dout"] = _normal(g, T, Hq, D, std=1e-2).to(torch.bfloat16)
        made = _plain_attn(s)     # what the forward pass left
        s["out"], s["lse"] = made["out"], made["lse"]
    return s


def _split(case, x):
    Hq, H = case["q_heads"], case["kv_heads"]
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    case = s["case"]
    op = case["op"]
    if op == "embed":
        from fp8_precision_linear_amd.embedding import embedding_fwd
        return embedding_fwd(s["ids"], s["table"], scale=case["scale"])
    if op == "embed_grad":
        from fp8_precision_linear_amd.embedding import embedding_bwd
        return embedding_bwd(s["dout"], s["ids"], case["vocab"], scale=case["scale"])
    if op in ("qk", "qk_grad"):
        from fp8_precision_linear_amd import qk_norm
        more = {"wq": s["wq"], "wk": s["wk"], "eps": EPS, "rope": s["rope"], "positions": s["positions"],
                "rope_pairs": case["rope"] == "pairs"}
        if op == "qk":
            q, k, v = qk_norm.qk_norm_rope_fwd(s["qkv"], case["q_heads"], case["kv_heads"], **more)
            return {"q": q, "k": k, "v": v}
        dx, dwq, dwk = qk_norm.qk_norm_rope_bwd(s["dq"], s["dk"], s["dv"], s["qkv"], **more)
        return {"dx": dx, "dwq": dwq, "dwk": dwk} if case["norm"] else {"dx": dx}
    from fp8_precision_linear_amd import self_attention as sa
    seqs = sa.Sequences(s["cu"], max_len=s["longest"], tokens=s["tokens"])
    q, k, v = _split(case, s["qkv"])
    if op == "attn":
        out, lse = sa.attention_fwd(q, k, v, seqs, causal=case["causal"], window=case["window"])
        return {"out": out, "lse": lse}
    dq, dk, dv = sa.attention_bwd(s["dout"], q, k, v, s["out"], s["lse"], seqs, causal=case["causal"],
                                  window=case["window"])
    return {"dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------ plain forms, fp32
def _plain_embed(s):
    ids, f32 = s["ids"], torch.float32
    there = (ids >= 0) & (ids < s["case"]["vocab"])
    rows = s["table"][ids.clamp(0, s["case"]["vocab"] - 1)].to(f32) * s["case"]["scale"]
    return torch.where(there[:, None], rows, 0.0).to(torch.bfloat16)


def _plain_embed_grad(s):
    """Tokens sorted by id; the rows of an id added from the first to the last."""
    case, ids = s["case"], s["ids"]
    there = (ids >= 0) & (ids < case["vocab"])
    key, order = torch.sort(torch.where(there, ids, case["vocab"]), stable=True)
    out = torch.zeros(case["vocab"] + 1, case["d"], device="cuda")
    out.index_add_(0, key, s["dout"][order].to(torch.float32))
    return out[:case["vocab"]] * case["scale"]


def _turn(x, s, back=False):
    """x [T, heads, D] rotated by its tokens' positions, or back."""
    rope = s["case"]["rope"]
    if rope == "none":
        return x
    pos = s["positions"].long()
    c, n = s["rope"][0][pos][:, None], s["rope"][1][pos][:, None]
    n = -n if back else n
    if rope == "halves":
        a, b = x.chunk(2, -1)
        return torch.cat((a * c - b * n, b * c + a * n), -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)


def _plain_qk(s):
    q, k, v = _split(s["case"], s["qkv"].to(torch.float32))

    def one(x, w):
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * w
        return _turn(x, s).to(torch.bfloat16)
    return {"q": one(q, s["wq"]), "k": one(k, s["wk"]), "v": v.to(torch.bfloat16)}


def _plain_qk_grad(s):
    f32 = torch.float32
    q, k, _ = _split(s["case"], s["qkv"].to(f32))

    def one(dy, x, w):
        dn = _turn(dy.to(f32), s, back=True)
        if w is None:
            return dn, None
        r = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
        xhat = x * r
        g = dn * w
        return r * (g - xhat * (g * xhat).mean(2, keepdim=True)), (dn * xhat).sum(0).sum(0)
    dq, dwq = one(s["dq"], q, s["wq"])
    dk, dwk = one(s["dk"], k, s["wk"])
    dx = torch.cat((dq, dk, s["dv"].to(f32)), 1).to(s["qkv"].dtype)
    return {"dx": dx} if dwq is None else {"dx": dx, "dwq": dwq, "dwk": dwk}


def _padded(s):
    """Rows of the sequences padded to the longest [B, n], which of them are
    tokens, and who sees whom [B, n, n]."""
    case, cu, n = s["case"], s["cu"].long(), s["longest"]
    t = torch.arange(n, device="cuda")
    real = t[None] < (cu[1:] - cu[:-1])[:, None]
    row = (cu[:-1, None] + t[None]).clamp(max=s["tokens"] - 1)
    see = real[:, None, :] & real[:, :, None]
    if case["causal"]:
        see = see & (t[None, :] <= t[:, None])
    if case["window"]:
        see = see & (t[None, :] > t[:, None] - case["window"])
    return row, real, see[:, None]


def _heads(x, row, real, group):
    """[T, H, D] as [B, H * group, n, D] in fp32, zeros where there is no token."""
    x = torch.where(real[..., None, None], x[row].to(torch.float32), 0.0).transpose(1, 2)
    return x if group == 1 else x.repeat_interleave(group, 1)


def _plain_attn(s):
    case = s["case"]
    row, real, see = _padded(s)
    G = case["q_heads"] // case["kv_heads"]
    q, k, v = _split(case, s["qkv"])
    q, k, v = _heads(q, row, real, 1), _heads(k, row, real, G), _heads(v, row, real, G)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(case["head_dim"] ** -0.5)
    score = torch.where(see, score, -torch.inf)
    m = score.amax(3, keepdim=True).clamp(min=-3e38)
    p = score.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    return {"out": o.transpose(1, 2)[real].to(torch.bfloat16), "lse": lse.transpose(1, 2)[real]}


def _plain_attn_grad(s):
    case, bf16 = s["case"], torch.bfloat16
    row, real, see = _padded(s)
    H, D = case["kv_heads"], case["head_dim"]
    G, scale = case["q_heads"] // H, D ** -0.5
    q, k, v = _split(case, s["qkv"])
    q, k, v = _heads(q, row, real, 1), _heads(k, row, real, G), _heads(v, row, real, G)
    do, o = _heads(s["dout"], row, real, 1), _heads(s["out"], row, real, 1)
    lse = torch.where(real[..., None], s["lse"][row], 0.0).transpose(1, 2)[..., None]
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale).sub_(lse).exp_()
    p = torch.where(see, p, 0.0)
    delta = (do * o).sum(3, keepdim=True)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous()).sub_(delta).mul_(p)
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q) * scale
    shared = lambda x: x.unflatten(1, (H, G)).sum(2).transpose(1, 2)[real].to(bf16)  # noqa: E731
    return {"dq": dq.transpose(1, 2)[real].to(bf16), "dk": shared(dk), "dv": shared(dv)}


PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "qk": _plain_qk, "qk_grad": _plain_qk_grad,
         "attn": _plain_attn, "attn_grad": _plain_attn_grad}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    size = 4 if case.get("x") == "fp32" else 2
    if op in ("embed", "embed_grad"):
        T, V, d = case["tokens"] - case["pad"], case["vocab"], case["d"]
        if op == "embed_grad":
            return {"bytes": T * d * size + 4 * V * d + 8 * T, "flops": T * d}
        # rows read: the expected number of different tokens
        p = [math.log((v + 2) / (v + 1)) / math.log(V + 1) for v in range(V)]
        rows = sum(1 - (1 - a) ** T for a in p)
        return {"bytes": int(rows * d * size) + 2 * case["tokens"] * d + 8 * T, "flops": T * d}
    Hq, H, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op in ("qk", "qk_grad"):
        T = case["tokens"]
        n = T * (Hq + 2 * H) * D
        angles = 0 if case["rope"] == "none" else 4 * D * min(T, case["positions"])
        per = size + 2 if op == "qk" else 2 * size + 2
        return {"bytes": n * per + angles + 4 * T, "flops": (9 if op == "qk" else 16) * n}
    n = _lengths(case)
    T, window = sum(n), case["window"]
    pairs = 0
    for a in n:
        if not case["causal"]:
            pairs += a * a
        elif not window or window >= a:
            pairs += a * (a + 1) // 2
        else:
            pairs += window * (window + 1) // 2 + (a - window) * window
    if op == "attn":
        return {"bytes": T * (4 * Hq * D + 4 * H * D + 4 * Hq), "flops": 4 * pairs * Hq * D}
    return {"bytes": T * (8 * Hq * D + 8 * H * D + 4 * Hq), "flops": 10 * pairs * Hq * D}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_embed(case, s):
    f64 = torch.float64
    ids = s["ids"].cpu().tolist()
    if case["op"] == "embed":
        good = torch.tensor([0 <= i < case["vocab"] for i in ids], device="cuda")
        rows = torch.index_select(s["table"], 0, torch.tensor([max(i, 0) for i in ids], device="cuda")).to(f64)
        return rows * good.to(f64)[:, None] * case["scale"]
    where = {}
    for t, i in enumerate(ids):
        if 0 <= i < case["vocab"]:
            where.setdefault(i, []).append(t)
    out = torch.zeros(case["vocab"], case["d"], dtype=f64, device="cuda")
    dout = s["dout"].to(f64)
    for i, ts in where.items():
        out[i] = dout[ts].sum(0) * case["scale"]
    return out


def _exact_qk(case, s):
    """The rotation as a product with a unit complex number; the gradient by
    applying the norm's Jacobian, r (I - xhat xhat^T / D) diag(w)."""
    f64, D = torch.float64, case["head_dim"]
    halves = case["rope"] != "pairs"

    def turned(x, sign):
        if case["rope"] == "none":
            return x
        z = torch.complex(x[..., : D // 2], x[..., D // 2:]) if halves else torch.complex(x[..., 0::2], x[..., 1::2])
        angle = torch.complex(s["rope"][0].to(f64), sign * s["rope"][1].to(f64))
        z = z * angle[s["positions"].long()][:, None]
        return torch.cat((z.real, z.imag), -1) if halves else torch.view_as_real(z).flatten(-2)

    def root(x):
        return (x.pow(2).sum(-1, keepdim=True) / D + EPS).pow(-0.5)
    q, k, v = _split(case, s["qkv"].to(f64))
    if case["op"] == "qk":
        made = [turned(x if w is None else x * root(x) * w.to(f64), 1.0) for x, w in ((q, s["wq"]), (k, s["wk"]))]
        return {"q": made[0], "k": made[1], "v": v}
    dx, dw = [], []
    for dy, x, w in ((s["dq"], q, s["wq"]), (s["dk"], k, s["wk"])):
        dn = turned(dy.to(f64), -1.0)
        if w is None:
            dx.append(dn)
            continue
        r = root(x)
        u = dn * w.to(f64)
        dx.append(r * u - x * (r.pow(3) / D) * (x * u).sum(-1, keepdim=True))
        dw.append((dn * x * r).sum((0, 1)))
    dx = torch.cat((*dx, s["dv"].to(f64)), 1)
    return {"dx": dx, "dwq": dw[0], "dwk": dw[1]} if dw else {"dx": dx}


def _exact_attn(case, s):
    """Sequence by sequence, key head by key head, from the softmax itself."""
    f64 = torch.float64
    Hq, H, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    G = Hq // H
    grad = case["op"] == "attn_grad"
    names = ("dq", "dk", "dv") if grad else ("out", "lse")
    parts = {n: [] for n in names}
    at = 0
    for n in _lengths(case):
        x = s["qkv"][at:at + n].to(f64).transpose(0, 1)
        q, k, v = x[:Hq].reshape(H, G * n, D), x[Hq:Hq + H], x[Hq + H:]
        i = torch.arange(n, device="cuda").repeat(G)[:, None]
        j = torch.arange(n, device="cuda")[None]
        hide = torch.zeros(G * n, n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= j > i
        if case["window"]:
            hide |= i - j >= case["window"]
        rows = {m: [] for m in names}
        for h in range(H):
            score = (torch.mm(q[h], k[h].t().contiguous()) / D ** 0.5).masked_fill_(hide, -torch.inf)
            lse = torch.logsumexp(score, 1)
            p = torch.exp(score - lse[:, None])
            if not grad:
                rows["out"].append(torch.mm(p, v[h]).view(G, n, D))
                rows["lse"].append(lse.view(G, n))
                continue
            do = s["dout"][at:at + n, G * h:G * h + G].to(f64).transpose(0, 1).reshape(G * n, D)
            dp = torch.mm(do, v[h].t().contiguous())
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) / D ** 0.5
            rows["dq"].append(torch.mm(ds, k[h]).view(G, n, D))
            rows["dk"].append(torch.mm(ds.t().contiguous(), q[h])[None])
            rows["dv"].append(torch.mm(p.t().contiguous(), do)[None])
        for m in names:
            parts[m].append(torch.cat(rows[m]).transpose(0, 1))
        at += n
    return {m: torch.cat(p) for m, p in parts.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("embed", "embed_grad"):
        return _exact_embed(case, s)
    if case["op"] in ("qk", "qk_grad"):
        return _exact_qk(case, s)
    return _exact_attn(case, s)
