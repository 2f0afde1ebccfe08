"""A wait of the 8-bit products that gave up is told to the caller: NaN in its results alone could be the data's."""
import time

import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from mixture_experts_layer_pack_gb300 import binding as B


@pytest.mark.gpu
def test_a_wait_that_gave_up_is_told_once():
    """A block waits with the products' own bounded wait on a barrier that nothing arrives at: it gives up after 2 s, the status says so once, and the
    same layer's results are the ones before."""
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *n: torch.randn(*n, generator=g, device="cuda").bfloat16()  # noqa: E731
    lin = M.MoEFp8Linear(300, 400)
    x, w = r(500, 300), M.fp8_quantize(r(400, 300), M.MOE_B_SQUARE)
    before = lin.forward(x, w)[0]
    assert M.moe_fp8_status() == 0
    t0 = time.monotonic()
    M.moe_fp8_selftest_timeout()
    assert M.moe_fp8_status() == B.MOE_ERR_TIMEOUT and time.monotonic() - t0 >= 1.5
    assert M.moe_fp8_status() == 0
    assert torch.equal(lin.forward(x, w)[0], before) and M.moe_fp8_status() == 0
    side = torch.cuda.Stream()                  # one word a device, whatever the stream
    M.moe_fp8_selftest_timeout(side)
    torch.cuda.synchronize()
    assert M.moe_fp8_status() == B.MOE_ERR_TIMEOUT and M.moe_fp8_status(side) == 0
