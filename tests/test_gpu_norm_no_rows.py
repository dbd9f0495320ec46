"""fp8_rmsnorm_quantize and fp8_rmsnorm_bwd of no rows through the C entry
points: only the words that they write are given, and nothing else is read."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [1, 64, 4099, 8192])
def test_no_rows(d):
    fl = need_gpu()
    amax = torch.full((1,), 7.0, device="cuda")
    bias = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert fl.lib.fp8_rmsnorm_quantize(None, fl.FP32, None, fl.FP32, None, fl.FP32, 0, d, 1e-5, None, None, fl.E4M3, 0,
                                       None, None, amax.data_ptr(), bias.data_ptr(), s) == 0
    dw = torch.full((d,), 7.0, device="cuda")
    assert fl.lib.fp8_rmsnorm_bwd(None, fl.FP32, None, fl.FP32, None, fl.FP32, None, None, 0, d, None, dw.data_ptr(),
                                  None, None, 0, s) == 0
    torch.cuda.synchronize()
    assert amax.item() == 0 and int(bias) == 0 and bool((dw == 0).all())
