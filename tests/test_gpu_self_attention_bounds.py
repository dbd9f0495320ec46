"""Attention over packed sequences writes nothing outside of its outputs and its
workspace, whatever cu_tokens holds: every buffer lies between guards."""
import pytest
import torch

from gpu_util import need_gpu, say
from test_gpu_self_attention import inputs

pytestmark = pytest.mark.gpu
GUARD = 4096      # bytes on either side
FILL = 0xA5


@pytest.fixture(scope="module")
def sa():
    need_gpu()
    from fp8_precision_linear_amd import self_attention
    return self_attention


class Guarded:
    """Tensors between guards."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = torch.empty(shape, dtype=dtype, device="meta").numel() * torch.empty(0, dtype=dtype).element_size()
        flat = torch.full((n + 2 * GUARD,), FILL, dtype=torch.uint8, device="cuda")
        self.all.append((flat, n))
        return flat[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for flat, n in self.all:
            assert bool((flat[:GUARD] == FILL).all()) and bool((flat[GUARD + n:] == FILL).all())


# (tokens, cu_tokens, max_len): past the tensors and before them, falling, cut by the
# bound; sequences that overlap, with more tiles than rows and sequences may have; and
# such among many short ones, whose tiles are counted through
ARRAYS = [(200, [0, 300, 900], 1000), (200, [-50, 20, 1 << 30], 1 << 30), (200, [150, 10, 190, 5, 250], 100),
          (1024, [0, 1024] * 4, 1024), (1000, [0, 999, 3, 1000, 1, 1000, 0, 1000, 500], 1 << 30),
          (2048, [0, 2048] * 20 + list(range(0, 600, 10)), 2048),
          (2048, list(range(0, 900, 9)) + [2048, 0, 2048, 5, 2047], 2048),
          (2047, [2047, 0] * 60, 2000)]


@pytest.mark.parametrize("heads", [(2, 2, 64), (4, 1, 128), (2, 1, 256), (24, 24, 64), (24, 24, 128)])
@pytest.mark.parametrize("array", range(len(ARRAYS)))
@pytest.mark.parametrize("mask", [{}, {"causal": False}, {"window": 100}])
def test_any_arrays(sa, heads, array, mask):
    Hq, H, D = heads
    T, cu, most = ARRAYS[array]
    say("arrays", heads, array, mask)
    q, k, v, dout = (t.contiguous() for t in inputs([T], Hq, H, D, 7))
    seqs = sa.Sequences(torch.tensor(cu, dtype=torch.int32, device="cuda"), max_len=most, tokens=T)
    make = Guarded()
    out, lse = make((T, Hq, D), torch.bfloat16), make((T, Hq), torch.float32)
    grads = [make((T, n, D), torch.bfloat16) for n in (Hq, H, H)]
    ws = make((sa.attention_bwd_workspace_bytes(seqs, Hq, H, D),), torch.uint8)
    out.zero_()
    lse.zero_()
    sa.attention_fwd(q, k, v, seqs, out=out, lse=lse, **mask)
    make.check()
    sa.attention_bwd(dout, q, k, v, out, lse, seqs, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws, **mask)
    make.check()
