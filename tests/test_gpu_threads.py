"""Host threads that launch the same kernels at different sizes at once, around the 4-bit products:
no launch may be refused for what another thread's needs, and the results are those of a call
alone."""

import ctypes
import threading

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
import w4_check as W
from sparse_mixture_experts_warp_b200.workloads import Workload

pytestmark = pytest.mark.gpu

i32 = dict(dtype=torch.int32, device="cuda")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _layer(w4, **kw):
    """make(): fresh outputs and (C function, arguments without the stream) of a layer call."""
    w = Workload("threads", D=64, F=64, **kw)
    d = M.desc_of(w)
    x = torch.randn(w.T, 64, device="cuda").to(torch.bfloat16)
    Wg = torch.randn(w.E, 64, device="cuda").to(torch.bfloat16)
    q = [W.random_w4(w.E, 64, 64, 64, False, s) for s in range(3)]
    b = [W.values64(m).to(torch.bfloat16) for m in q]

    def make():
        out, ws = torch.zeros_like(x), M.empty_workspace(d)
        f = M.lib().moe_layer_forward_w4 if w4 else M.lib().moe_layer_forward
        form = [m._ref() for m in q] if w4 else [_p(m) for m in b]
        return [out], (ws, q, b, x, Wg, d), f, (
            ctypes.byref(d), _p(x), _p(Wg), None, *form, None, None, None, _p(out), _p(ws),
            ws.numel())

    return make


def _product(G, rows, dtype, D=64, F=64):
    d = M.desc_of(Workload("threads", T=1, D=D, E=2, F=F, k=1, act="relu", dtype=dtype))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    a = torch.randn(G * rows, D, device="cuda").to(dt)
    up = (torch.randn(G, F, D, device="cuda") * D ** -0.5).to(dt)
    off = torch.arange(0, G * rows + 1, rows, **i32)

    def make():
        h = torch.zeros(G * rows, F, dtype=dt, device="cuda")
        return [h], (a, up, off, d), M.lib().moe_expert_up, (
            ctypes.byref(d), G, F, _p(a), G * rows, _p(off), None, _p(up), _p(h))

    return make


def _permute(T, k, E):
    d = M.desc_of(Workload("threads", T=T, D=64, E=E, F=64, k=k))
    ids = torch.randint(0, E, (T, k), **i32)
    x = torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda")

    def make():
        outs = [torch.zeros(n, **i32) for n in (E, E + 1, T * k, T * k)]
        scratch = M.empty_scratch(d)
        return outs, (ids, x, scratch, d), M.lib().moe_permute, (
            ctypes.byref(d), _p(ids), _p(x), None, *(_p(o) for o in outs), _p(scratch),
            scratch.numel())

    return make


def _route(**kw):
    w = Workload("threads", D=64, F=64, **kw)
    d = M.desc_of(w)
    dt = torch.bfloat16 if w.dtype == "bf16" else torch.float32
    x = torch.randn(w.T, 64, device="cuda").to(dt)
    Wg = torch.randn(w.E, 64, device="cuda").to(dt)
    choice = w.select == "expert"

    def make():
        ids = torch.zeros(*((w.E, w.c) if choice else (w.T, w.k)), **i32)
        gates = torch.zeros(w.T, w.E if choice else w.k, device="cuda")
        scratch = M.empty_scratch(d)
        return [ids, gates], (x, Wg, scratch, d), M.lib().moe_route, (
            ctypes.byref(d), _p(x), _p(Wg), None, _p(ids), _p(gates), None, None, None, _p(scratch),
            scratch.numel())

    return make


PAIRS = {
    "layer on 4-bit weights": lambda: (_layer(True, T=300, E=8, k=2), _layer(True, T=3000, E=64, k=6)),
    "layer": lambda: (_layer(False, T=300, E=8, k=2), _layer(False, T=3000, E=64, k=6)),
    "bf16 product": lambda: (_product(1, 40, "bf16"), _product(200, 3, "bf16")),
    "fp32 product": lambda: (_product(1, 1, "f32", D=16384), _product(1, 1, "f32", D=30000)),
    "permutation": lambda: (_permute(5000, 2, 8), _permute(10000, 6, 256)),
    "expert choice": lambda: (_route(T=16384, E=8, c=100, select="expert"),
                              _route(T=32768, E=8, c=100, select="expert")),
    "router, fp32": lambda: (_route(T=100, E=240, c=9, select="expert", dtype="f32"),
                             _route(T=100, E=256, c=9, select="expert", dtype="f32")),
    "router, tensor cores": lambda: (_route(T=100, E=16, k=2), _route(T=600, E=24, k=2)),
}


@pytest.mark.parametrize("pair", PAIRS)
def test_threads_of_unlike_sizes(pair):
    jobs = []
    for make in PAIRS[pair]():
        want, keep, f, args = make()
        assert f(*args, None) == 0
        for _ in range(2):
            outs, own, f, args = make()
            stream = torch.cuda.Stream()
            jobs.append((outs, want, stream, f, (*args, ctypes.c_void_p(stream.cuda_stream)),
                         keep, own))
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(jobs)), []

    def run(outs, want, stream, f, args, *_):
        status = f(*args)                           # (binds the thread's context)
        start.wait()
        for i in range(1500):
            status = status or f(*args)
            if i % 16 == 15:
                stream.synchronize()                # the launch queue never fills up
        if status:
            errors.append(status)

    threads = [threading.Thread(target=run, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, [M.status_string(e) for e in errors]
    assert M.get_device_error() == 0
    for outs, want, *_ in jobs:
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
