"""Every wait of the 4-bit products is bounded.

The test hook makes CTA 0's weight producer arm a ring stage without loading it.  The wait for it
has to run out, the device error word to record MOE_ERR_TIMEOUT, the launch to end, and the next
call, without the hook, to give the result of the call before it.  Rows per group choose the kernel:
streaming, then tcgen05 with tiles of 32, 128 and 192 tokens.
"""

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
from sparse_mixture_experts_warp_b200.workloads import Workload
import w4_check as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["up", "down"])
@pytest.mark.parametrize("rows", [1, 12, 60, 300])
def test_withheld_stage_times_out_and_context_stays_usable(op, rows):
    G, D, F = 2, 4096, 4096                         # several rounds of every ring, several tiles
    d = M.desc_of(Workload("wait", T=1, D=D, E=G, F=F, k=1))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    a = torch.randn(G * rows, D, generator=gen, device="cuda").to(torch.bfloat16)
    gate, w = (W.random_w4(G, F, D, 128, True, i) for i in (1, 2))
    offsets = torch.tensor([0, rows, G * rows], dtype=torch.int32, device="cuda")
    out = torch.zeros(G * rows, F, dtype=torch.bfloat16, device="cuda")

    def call():
        if op == "up":
            M.moe_expert_up_w4(d, G, F, a, offsets, gate, w, out)
        else:
            M.moe_expert_down_w4(d, G, F, a, offsets, w, out)

    call()
    assert M.get_device_error() == 0
    ref = out.clone()
    M.debug_inject(1)
    try:
        call()
        status, code = M.device_error_status()      # synchronises: a bounded wait of about 2 s
    finally:
        M.debug_inject(0)
    assert status == 5, (status, hex(code))         # MOE_ERR_TIMEOUT
    assert 0x100 <= code < 0x200
    assert M.get_device_error() == 0                # the word was cleared
    out.zero_()
    call()
    assert M.get_device_error() == 0
    assert torch.equal(out, ref)
