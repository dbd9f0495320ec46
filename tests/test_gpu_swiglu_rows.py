"""SwiGLU of more short rows than one grid's lanes hold (2^24 workgroups of 256):
the same bits as the rows give in calls that fit one launch."""
import pytest
import torch

from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f", [4, 3])
def test_many_short_rows(f):
    fl = need_gpu()
    rows, cut = (1 << 24) + 77, 1 << 23
    say("swiglu", rows, f)
    g = torch.Generator(device="cuda").manual_seed(f)
    h = torch.randn(rows, 2 * f, generator=g, device="cuda")
    da = torch.randn(rows, f, generator=g, device="cuda")
    h[-1] = 30.0
    am, dam = (torch.empty(1, device="cuda") for _ in range(2))
    a, dh = fl.swiglu_fwd(h, amax=am), fl.swiglu_bwd(h, da, amax=dam)
    assert am.item() == a.float().abs().max().item() == 900.0
    assert dam.item() == dh.float().abs().max().item()
    for part in (slice(0, cut), slice(cut, rows)):
        assert torch.equal(a[part], fl.swiglu_fwd(h[part].clone()))
        assert torch.equal(dh[part], fl.swiglu_bwd(h[part].clone(), da[part].clone()))
