"""Calls of the 4-bit products, their conversions and the step gradients that have nothing to do: no
tokens, rows or matrices (no GPU)."""

import ctypes

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
from sparse_mixture_experts_warp_b200.build import build
from sparse_mixture_experts_warp_b200.workloads import WORKLOADS, Workload, scaled

OK, INVALID, WORKSPACE = 0, 1, 3
P = 0x10000


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def _w4():
    return M.MoeW4(codes=P, scales=P, zeros=None, row_scale=P, group=128, reserved=0)


def test_nothing_to_do_takes_empty_buffers():
    """No tokens, rows or matrices: tensors without elements have no address, and no kernel is
    enqueued.  The other arguments are checked all the same."""
    L, n0, b, w = M.lib(), M.kernel_launches(), ctypes.byref, ctypes.byref(_w4())
    d = M.desc_of(scaled(WORKLOADS["mixtral"], T=4, D=256, F=512))
    none = M.desc_of(scaled(WORKLOADS["mixtral"], T=0, D=256, F=512))
    # the step gradients
    assert L.moe_combine_backward(b(none), None, None, None, None, None, None, None) == OK
    assert L.moe_permute_backward(b(none), None, None, None, None, None) == OK
    bad = M.desc_of(scaled(WORKLOADS["mixtral"], T=0, D=256, F=512))
    bad.k = 9
    assert L.moe_combine_backward(b(bad), None, None, None, None, None, None, None) == INVALID
    assert L.moe_permute_backward(b(bad), None, None, None, None, None) == INVALID
    # the products
    assert L.moe_expert_up_w4(b(d), 8, 512, None, 0, P, w, w, None, None) == OK
    assert L.moe_expert_down_w4(b(d), 8, 512, None, 0, P, w, None, None) == OK
    assert L.moe_expert_up_w4(b(d), 8, 512, None, 0, None, w, w, None, None) == INVALID
    assert L.moe_expert_up_w4(b(d), 8, 512, None, 0, P, None, w, None, None) == INVALID
    assert L.moe_expert_up_w4(b(d), 8, 512, None, 0, P, w, None, None, None) == INVALID
    assert L.moe_expert_down_w4(b(d), 8, 512, None, 0, P, None, None, None) == INVALID
    assert L.moe_expert_up_w4(b(d), 8, 512, P, 0, P, w, w, P + 2, None) == INVALID
    assert L.moe_expert_up_w4(b(d), 8, 512, None, 1, P, w, w, P, None) == INVALID
    assert L.moe_expert_up_w4(b(d), 8, 512, P, 1, P, w, w, None, None) == INVALID
    assert L.moe_expert_down_w4(b(d), 8, 512, None, 1, P, w, P, None) == INVALID
    assert L.moe_expert_down_w4(b(d), 8, 512, P, 1, P, w, None, None) == INVALID
    # the conversions
    empty = ctypes.byref(M.MoeW4(None, None, None, None, 64, 0))
    assert L.moe_quantize_w4(0, 64, 64, M.BF16, None, empty, None) == OK
    assert L.moe_dequantize_w4(0, 64, 64, empty, M.F32, None, None) == OK
    assert L.moe_quantize_w4(1, 64, 64, M.BF16, None, w, None) == INVALID
    assert L.moe_quantize_w4(1, 64, 64, M.BF16, P, empty, None) == INVALID
    assert L.moe_quantize_w4(0, 64, 64, 7, None, empty, None) == INVALID
    assert L.moe_quantize_w4(0, 64, 64, M.BF16, None, None, None) == INVALID
    # the layer
    layer = lambda d, *a: L.moe_layer_forward_w4(b(d), *a, None)      # noqa: E731
    need = M.workspace_size(none)
    assert layer(none, None, P, None, w, w, w, None, None, None, None, P, need) == OK
    assert layer(none, None, None, None, w, w, w, None, None, None, None, P, need) == INVALID
    assert layer(none, None, P, None, w, w, w, None, None, None, None, P, need - 1) == WORKSPACE
    assert layer(d, None, P, None, w, w, w, None, None, None, P, P, 1 << 40) == INVALID
    assert layer(d, P, P, None, w, w, w, None, None, None, None, P, 1 << 40) == INVALID
    assert M.kernel_launches() == n0


def test_the_binding_takes_empty_tensors():
    """(on the CPU the binding's check of the device is left out)"""
    d = M.desc_of(Workload("none", T=0, D=256, E=8, F=512, k=2))
    x, inv = torch.empty(0, 256, dtype=torch.bfloat16), torch.empty(0, 2, dtype=torch.int32)
    gates = torch.empty(0, 2)
    here, stream, M._here, M._stream = M._here, M._stream, lambda *t: None, lambda s: None
    try:
        M.moe_combine_backward(d, x, x, inv, gates, x, gates)
        M.moe_combine_backward(d, x, None, inv, gates, x, None)
        M.moe_permute_backward(d, x, inv, x, x)
        M.moe_permute_backward(d, x, inv, None, x)
        off = torch.zeros(3, dtype=torch.int32)
        gate, down = (M.empty_w4(2, *s, device="cpu") for s in ((512, 256), (256, 512)))
        h = torch.empty(0, 512, dtype=torch.bfloat16)
        # (addresses of host memory: without rows nothing is launched)
        for t in (gate.codes, gate.scales, gate.row_scale, down.codes, down.scales, down.row_scale):
            assert t.data_ptr() % 16 == 0
        assert off.data_ptr()
        M.moe_expert_up_w4(d, 2, 512, x, off, gate, gate, h)
        M.moe_expert_down_w4(d, 2, 512, h, off, down, x)
        w = M.empty_w4(0, 64, 128, device="cpu")
        M.moe_quantize_w4(torch.empty(0, 64, 128), w)
        M.moe_dequantize_w4(w, torch.empty(0, 64, 128))
    finally:
        M._here, M._stream = here, stream
