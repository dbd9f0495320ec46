"""64-bit forms of attention over packed sequences and its gradients, and the
error bounds of the kernels' arithmetic.

Bounds.  h = 2^-8 is half a step of bf16 relative to a value, u = 2^-18 covers
fp32: sums of up to 4096 products in fp32 stay below 2^-24 * 4096^(1/2) * (a few)
of the sum of magnitudes, and so do exp, its argument (2^-24 of lse and of the
logits, at most 64 in size here) and lse.
  out  h sum_j p_j |v_j|  (p rounded)  + h |out|  + u sum_j p_j |v_j|
  lse  u (1 + |lse|)
  dv   h sum p |dout| + h |dv| + u sum p |dout|
  ds   (before its rounding) e = u p (sum_d |dout v| + sum_d |dout out|)
  dq   scale (h sum |ds| |k| + sum e |k|) + h |dq|;  dk likewise with q
each enlarged by 1 + 2^-6 for second order terms, plus 2^-126 for results below
the normal numbers."""
import torch

H8, U = 2.0 ** -8, 2.0 ** -18
MORE, TINY = 1 + 2.0 ** -6, 2.0 ** -126


def visible(n, causal, window):
    i = torch.arange(n)[:, None]
    j = torch.arange(n)[None]
    see = torch.ones(n, n, dtype=torch.bool)
    if causal:
        see &= j <= i
    if window:
        see &= j > i - window
    return see.cuda()


def forward(q, k, v, lens, scale, causal=True, window=0):
    """{name: (value, bound)} for out and lse, float64, sequence by sequence."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    b_out = torch.zeros_like(out)
    at = 0
    for n in lens:
        see = visible(n, causal, window)
        for a in range(Hq):
            qa, ka, va = (x[at:at + n, b].double() for x, b in ((q, a), (k, a // G), (v, a // G)))
            s = (qa @ ka.t().contiguous() * scale).masked_fill(~see, -torch.inf)
            lse[at:at + n, a] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[at:at + n, a, None])
            p = torch.where(see, p, 0.0)
            out[at:at + n, a] = p @ va
            b_out[at:at + n, a] = (H8 + U) * (p @ va.abs())
        at += n
    return {"out": (out, MORE * (b_out + H8 * out.abs()) + TINY), "lse": (lse, U * (1 + lse.abs()))}


def backward(dout, q, k, v, out, lse, lens, scale, causal=True, window=0):
    """{name: (value, bound)} for dq, dk, dv from the forward's out and lse."""
    f64 = torch.float64
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    made = {n: torch.zeros(t.shape, dtype=f64, device="cuda") for n, t in (("dq", q), ("dk", k), ("dv", v))}
    err = {n: torch.zeros_like(t) for n, t in made.items()}
    at = 0
    for n in lens:
        see = visible(n, causal, window)
        r = slice(at, at + n)
        for a in range(Hq):
            b = a // G
            qa, ka, va, ga, oa = (x[r, c].double() for x, c in ((q, a), (k, b), (v, b), (dout, a), (out, a)))
            p = torch.exp(qa @ ka.t().contiguous() * scale - lse[r, a, None].double())
            p = torch.where(see, p, 0.0)
            dp = ga @ va.t().contiguous()
            ds = p * (dp - (ga * oa).sum(1, keepdim=True))
            e = U * p * (ga.abs() @ va.abs().t().contiguous() + (ga * oa).abs().sum(1, keepdim=True))
            made["dq"][r, a] += scale * (ds @ ka)
            err["dq"][r, a] += abs(scale) * ((H8 * ds.abs() + e) @ ka.abs())
            dst, et, pt = ds.t().contiguous(), e.t().contiguous(), p.t().contiguous()
            made["dk"][r, b] += scale * (dst @ qa)
            err["dk"][r, b] += abs(scale) * ((H8 * dst.abs() + et) @ qa.abs())
            made["dv"][r, b] += pt @ ga
            err["dv"][r, b] += (H8 + U) * (pt @ ga.abs())
        at += n
    return {n: (made[n], MORE * (err[n] + H8 * made[n].abs()) + TINY) for n in made}


def inside(got, want, what):
    """Every element of `got` within the bound of its value."""
    for name, t in got.items():
        value, bound = want[name]
        off = (t.double() - value).abs()
        ok = off <= bound
        assert bool(ok.all()), (f"{what}: {name}: {int((~ok).sum())} of {ok.numel()} outside; worst "
                                f"{(off / bound).max().item():.3g} of the bound")
