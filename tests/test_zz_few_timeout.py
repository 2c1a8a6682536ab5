"""The waits of the layer for a few tokens, made to run out without a fault: gate/up products that are left out never
arrive, every warp that waits for them or behind them gives up after about a second, copies in flight land, the error word
reports it and is cleared by reading, and the next call on the same workspace is right."""
import pytest
import torch

import nvfp4_expert_gemms_gb300 as M
from test_few_ops import Layer

pytestmark = pytest.mark.gpu

MOE_ERR_DEVICE_TIMEOUT = 5


# every format; NVFP4's scales by TMA (H and I multiples of 256) and lane by lane; more teams than units, and fewer
@pytest.mark.parametrize("fmt,T,E,k,H,I", [("fp8", 16, 128, 8, 2048, 768), ("int4", 5, 8, 2, 512, 256), ("nvfp4_w4a16", 3, 16, 4, 1024, 512),
                                           ("nvfp4_w4a16", 32, 8, 8, 384, 640), ("bf16", 1, 2, 1, 128, 128)])
def test_few_waits_run_out(fmt, T, E, k, H, I):
    layer = Layer(fmt, T, E, k, H, I, seed=T)
    want = layer.run()
    layer.check(want)
    M.moe_debug_few_timeout()
    layer.run()
    assert M.moe_get_device_error(layer.ws) == MOE_ERR_DEVICE_TIMEOUT
    assert M.moe_get_device_error(layer.ws) == 0  # read and cleared
    assert torch.equal(layer.run(), want)
    assert M.moe_get_device_error(layer.ws) == 0
