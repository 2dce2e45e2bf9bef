"""Calls that overlap: several host threads that launch the same kernels at different sizes, and
products that run on two streams at once.  The steps need no scratch, so nothing asks a caller to
put them one after the other."""

import ctypes
import threading

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
import w4_check as W
from sparse_mixture_experts_warp_b200.workloads import Workload

pytestmark = pytest.mark.gpu


class Product:
    """A down product [G * rows, K] x [G, N, K] on weights of its own, and its output."""

    def __init__(self, G, rows, N, K, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.size = G, K
        self.d = M.desc_of(Workload("threads", T=1, D=N, E=max(2, min(G, 256)), F=K, k=1))
        self.a = torch.randn(G * rows, K, generator=gen, device="cuda").to(torch.bfloat16)
        self.w = W.random_w4(G, N, K, 128, False, seed)
        self.offsets = torch.arange(0, G * rows + 1, rows, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(G * rows, N, dtype=torch.bfloat16, device="cuda")

    def call(self, out, stream):
        M.moe_expert_down_w4(self.d, *self.size, self.a, self.offsets, self.w, out, stream)

    def c_call(self, out, stream):
        """The C function and its arguments."""
        G, K = self.size
        p = [ctypes.c_void_p(t.data_ptr()) for t in (self.a, self.offsets, out)]
        return M.lib().moe_expert_down_w4, (
            ctypes.byref(self.d), G, K, p[0], self.a.shape[0], p[1], self.w._ref(), p[2],
            ctypes.c_void_p(stream.cuda_stream))


class Quantizer:
    """Rows of K elements to codes; the scales' side tables need more than 48 KB."""

    def __init__(self, K, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.X = torch.randn(1, 64, K, generator=gen, device="cuda").to(torch.bfloat16)
        self.out = torch.zeros(1, 64, K // 2, dtype=torch.uint8, device="cuda")
        self.forms = []

    def _form(self, out):
        w = M.empty_w4(1, 64, 2 * out.shape[-1], 32, True)
        self.forms.append(M.W4(out, w.scales, w.zeros, w.row_scale, 32))
        return self.forms[-1]

    def call(self, out, stream):
        M.moe_quantize_w4(self.X, self._form(out), stream)

    def c_call(self, out, stream):
        return M.lib().moe_quantize_w4, (
            1, 64, self.X.shape[-1], M.BF16, ctypes.c_void_p(self.X.data_ptr()),
            self._form(out)._ref(), ctypes.c_void_p(stream.cuda_stream))


# Pairs whose launches of one kernel need different amounts of shared memory: the streaming product
# by K and rows, the tcgen05 one by G (tiles of 32, 128 and 192 tokens), the quantiser by its side
# tables of very long rows.
PAIRS = {
    "streaming": lambda: (Product(1, 1, 64, 128, 1), Product(1, 6, 64, 8192, 2)),
    "tcgen05, 32 tokens": lambda: (Product(1, 12, 64, 128, 3), Product(200, 8, 64, 128, 4)),
    "tcgen05, 128 tokens": lambda: (Product(1, 40, 64, 128, 5), Product(200, 20, 64, 128, 6)),
    "tcgen05, 192 tokens": lambda: (Product(1, 130, 64, 128, 7), Product(100, 130, 64, 128, 8)),
    "quantiser": lambda: (Quantizer(196608, 9), Quantizer(262144, 10)),
}


@pytest.mark.parametrize("pair", PAIRS)
def test_threads_of_unlike_sizes(pair):
    """Two threads of either size launch at once, without a step of Python between a thread's
    calls; no launch may be refused for what another thread's needs."""
    jobs = []
    for job in PAIRS[pair]():
        job.call(job.out, None)
        for _ in range(2):
            out, stream = torch.zeros_like(job.out), torch.cuda.Stream()
            jobs.append((out, job.out, stream, *job.c_call(out, stream)))
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(jobs)), []

    def run(out, want, stream, f, args):
        status = f(*args)                           # (binds the thread's context)
        start.wait()
        for i in range(4000):
            status = status or f(*args)
            if i % 32 == 31:
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
    for out, want, *_ in jobs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("one,two", [((2, 3, 512, 4096), (3, 5, 512, 2048)),
                                     ((2, 90, 512, 1024), (4, 2, 512, 4096)),
                                     ((2, 60, 512, 1024), (2, 300, 512, 1024)),
                                     ((4, 8, 512, 4096), (2, 10, 512, 4096))])
def test_products_on_two_streams_at_once(one, two):
    """Products of each kernel in flight together, with no wait between the streams: the bits are
    those of the same calls one after the other."""
    work = [Product(*shape, seed) for seed, shape in enumerate((one, two))]
    for job in work:
        job.call(job.out, None)
    outs = [[torch.zeros_like(job.out) for _ in range(8)] for job in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for i in range(8):
        for job, mine, stream in zip(work, outs, streams):
            job.call(mine[i], stream)
    torch.cuda.synchronize()
    assert M.get_device_error() == 0
    for job, mine in zip(work, outs):
        assert all(torch.equal(o, job.out) for o in mine)
