"""The gradients of attention over packed sequences where logits are large: p =
exp(s - lse) is as exact as its argument.

Bounds, beside those of seq_ref.backward (which takes the same out and lse): the
argument is formed in units of log2 as fma(t, c, -l), with t = q.k summed in fp32,
c = scale log2(e) and l = lse log2(e) rounded.  In natural units it is off by
  2^-24 D scale sum |q k|      t: D additions of at most the magnitudes' sum
  2 2^-24 |s|                  c: log2(e) as a float (2^-26) and the product
  2 2^-24 |lse|                l: likewise
so p is off by p (e^E - 1) for E their sum, dv by that times |dout|, and ds by that
times (|dp| + |delta|).

The exponential has no results below fp32's normal numbers, nor have the products
operands below bf16's: a p or ds of less than 2^-126 counts as zero and is off by as
much, which |dout|, |dp| + |delta|, |q| and |k| multiply as they do the rest.  (Logits
of some 256 reach this: e^-88 = 2^-127; dk of 3e-37 was 0, 2^-126 = 1.2e-38 of p times
|dp| + |delta| of about 10 and scale |q| of about 4.)"""
import pytest
import torch

import seq_ref
from gpu_util import need_gpu, say
from test_gpu_self_attention import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    need_gpu()
    from fp8_precision_linear_amd import self_attention
    return self_attention


@pytest.mark.parametrize("heads", [(2, 2, 64), (4, 2, 128), (2, 1, 256)])
@pytest.mark.parametrize("power", [2, 4, 6])
@pytest.mark.parametrize("causal", [True, False])
def test_gradients_of_large_logits(sa, heads, power, causal):
    Hq, H, D = heads
    lens = [150, 65, 1]
    say("large", heads, power, causal)
    q, k, v, dout = inputs(lens, Hq, H, D, 30 + power)
    q, k = q * 2.0 ** power, k * 2.0 ** power
    seqs = sa.Sequences.from_lists(lens)
    scale = D ** -0.5
    out, lse = sa.attention_fwd(q, k, v, seqs, causal=causal)
    got = dict(zip(("dq", "dk", "dv"), sa.attention_bwd(dout, q, k, v, out, lse, seqs, causal=causal)))
    want = seq_ref.backward(dout, q, k, v, out, lse, lens, scale, causal)
    more = {n: torch.zeros_like(b) for n, (_, b) in want.items()}
    at, G = 0, Hq // H
    for n in lens:
        see, r = seq_ref.visible(n, causal, 0), slice(at, at + n)
        for a in range(Hq):
            b = a // G
            qa, ka, va, ga, oa = (x[r, c].double() for x, c in ((q, a), (k, b), (v, b), (dout, a), (out, a)))
            s = qa @ ka.t().contiguous() * scale
            la = lse[r, a, None].double()
            p = torch.where(see, torch.exp(s - la), 0.0)
            e = 2.0 ** -24 * (D * scale * (qa.abs() @ ka.abs().t().contiguous()) + 2 * s.abs() + 2 * la.abs())
            dp = torch.where(see, p * torch.expm1(e) * (1 + seq_ref.H8) + seq_ref.TINY, 0.0)
            ds = dp * ((ga @ va.t().contiguous()).abs() + (ga * oa).sum(1, keepdim=True).abs()) + seq_ref.TINY * see
            more["dv"][r, b] += dp.t().contiguous() @ ga.abs()
            more["dq"][r, a] += scale * (ds @ ka.abs())
            more["dk"][r, b] += scale * (ds.t().contiguous() @ qa.abs())
        at += n
    seq_ref.inside(got, {n: (w, bound + more[n] * (1 + seq_ref.H8)) for n, (w, bound) in want.items()}, f"{heads} 2^{power}")
