"""The library as the first CUDA call of a host thread, on which no context is current yet: every
entry point of the 4-bit weights, the step gradients and the layer runs there, and gives what the
main thread got."""

import threading

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
import w4_check as W
from sparse_mixture_experts_warp_b200.workloads import Workload

pytestmark = pytest.mark.gpu


def _products(op, rows):
    d = M.desc_of(Workload("first", T=1, D=128, E=2, F=128, k=1, act="relu"))
    w = W.random_w4(2, 128, 128, 64, True, rows)
    a = torch.randn(2 * rows, 128, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(a)
    if op == "up":
        return lambda: M.moe_expert_up_w4(d, 2, 128, a, off, None, w, out), [out]
    return lambda: M.moe_expert_down_w4(d, 2, 128, a, off, w, out), [out]


def _quantize():
    X, w = torch.randn(2, 128, 192, device="cuda"), M.empty_w4(2, 128, 192, 64, True)
    outs = [w.codes, w.scales.view(torch.uint8), w.zeros, w.row_scale]
    for t in outs:
        t.zero_()
    return lambda: M.moe_quantize_w4(X, w), outs


def _dequantize():
    w, out = W.random_w4(2, 128, 192), torch.zeros(2, 128, 192, device="cuda")
    return lambda: M.moe_dequantize_w4(w, out), [out]


def _steps(which):
    d = M.desc_of(Workload("first", T=50, D=64, E=4, F=64, k=2))
    y = torch.randn(100, 64, device="cuda").to(torch.bfloat16)
    inv = torch.randperm(100, device="cuda").int().view(50, 2)
    gates = torch.rand(50, 2, device="cuda")
    dout = torch.randn(50, 64, device="cuda").to(torch.bfloat16)
    if which == "merge":
        dy, dg = torch.zeros_like(y), torch.zeros_like(gates)
        return lambda: M.moe_combine_backward(d, dout, y, inv, gates, dy, dg), [dy, dg]
    dx = torch.zeros_like(dout)
    return lambda: M.moe_permute_backward(d, y, inv, None, dx), [dx]


def _layer(T, E):
    w = Workload("first", T=T, D=256, E=E, F=256, k=2)
    d = M.desc_of(w)
    x = torch.randn(T, 256, device="cuda").to(torch.bfloat16)
    Wg = torch.randn(E, 256, device="cuda").to(torch.bfloat16)
    q = [W.random_w4(E, 256, 256, 128, False, s) for s in range(3)]
    ws, out = M.empty_workspace(d), torch.zeros_like(x)
    return lambda: M.moe_layer_forward_w4(d, x, Wg, None, *q, None, None, None, out, ws), [out]


CALLS = {
    **{f"{op}, {n} rows": (lambda op=op, n=n: _products(op, n))
       for op in ("up", "down") for n in (1, 12, 40, 130)},
    "quantize": _quantize, "dequantize": _dequantize,
    "merge gradient": lambda: _steps("merge"), "dispatch gradient": lambda: _steps("dispatch"),
    "layer, one token": lambda: _layer(1, 8), "layer, 64 experts": lambda: _layer(70, 64),
}


@pytest.mark.parametrize("name", CALLS)
def test_first_call_of_a_host_thread(name):
    call, outs = CALLS[name]()
    call()
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    errors = []

    def run():
        try:
            call()
        except Exception as e:                      # noqa: BLE001 (shown by the assert below)
            errors.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    assert M.get_device_error() == 0
    for o, ref in zip(outs, want):
        assert torch.equal(o, ref)
