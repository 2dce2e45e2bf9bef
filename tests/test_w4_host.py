"""4-bit expert weights and the dispatch / merge gradients on the host (no GPU): the layout rule,
the binding's shape checks, and the arguments that are refused before anything is launched."""

import ctypes

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
import w4_check as W
from sparse_mixture_experts_warp_b200.build import build
from sparse_mixture_experts_warp_b200.workloads import WORKLOADS, scaled

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 0x10000


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def _w4(**kw):
    f = dict(codes=P, scales=P, zeros=None, row_scale=P, group=128, reserved=0)
    f.update(kw)
    return ctypes.byref(M.MoeW4(**f))


def _desc(**kw):
    return M.desc_of(scaled(WORKLOADS["mixtral"], T=4, D=256, F=512, **kw))


def test_layout_rule():
    # byte 4 w + b of a 64-weight block holds nibbles 2 b (low) and 2 b + 1 (high) of word w
    codes = torch.zeros(1, 64, 32, dtype=torch.uint8)
    codes[0, 0, 0] = 0x21            # word 0: nibble 0 -> k 0, nibble 1 -> k 2
    codes[0, 0, 2] = 0x03            # word 0: nibble 4 -> k 1
    codes[0, 0, 4 * 1] = 0x05        # word 1 (c 0, j 1): k 32
    codes[0, 0, 4 * 2] = 0x07        # word 2 (c 1, j 0): k 8
    codes[0, 0, 31] = 0xf0           # word 7 (c 3, j 1): nibble 7 -> k 32 + 24 + 7 = 63
    q = W.codes64(codes)[0, 0]
    want = torch.zeros(64, dtype=torch.float64)
    for k, v in ((0, 1), (2, 2), (1, 3), (32, 5), (8, 7), (63, 15)):
        want[k] = v
    assert torch.equal(q, want)


def test_scale_times_code_is_a_bf16():
    s = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    q = torch.arange(-15, 16).double()
    v = s[:, None] * q
    assert torch.equal(v.to(torch.bfloat16).double(), v)


def test_plain_quantizer_error():
    g = torch.Generator().manual_seed(0)
    X = torch.randn(2, 64, 192, generator=g) * torch.exp(torch.randn(2, 64, 1, generator=g))
    for zeros in (False, True):
        q, s, z, row = W.quantize_plain(X, 32, zeros)
        at = torch.arange(192) // 32
        step = (s.float()[:, at].transpose(1, 2) * row[..., None]).double()
        zz = 8 if z is None else z[:, at].transpose(1, 2).double()
        err = ((q.double() - zz) * step - X.double()).abs()
        # half a step; with zero points their rounding and the scale's add one
        assert (err <= (1.6 if zeros else 0.51) * step).all()


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(row_scale=None), INVALID),
    (dict(codes=P + 8), INVALID), (dict(scales=P + 1), INVALID), (dict(zeros=P + 4), INVALID),
    (dict(row_scale=P + 4), INVALID), (dict(reserved=1), INVALID),
    (dict(group=0), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=256), UNSUPPORTED),
    (dict(group=-64), UNSUPPORTED),
])
def test_bad_weights_are_refused(kw, status):
    L, d, n0 = M.lib(), _desc(), M.kernel_launches()
    bad, good = _w4(**kw), _w4()
    assert L.moe_quantize_w4(2, 64, 128, M.BF16, P, bad, None) == status
    assert L.moe_dequantize_w4(2, 64, 128, bad, M.F32, P, None) == status
    assert L.moe_expert_up_w4(ctypes.byref(d), 8, 512, P, 8, P, good, bad, P, None) == status
    assert L.moe_expert_up_w4(ctypes.byref(d), 8, 512, P, 8, P, bad, good, P, None) == status
    assert L.moe_expert_down_w4(ctypes.byref(d), 8, 512, P, 8, P, bad, P, None) == status
    for i in range(3):
        w = [good] * 3
        w[i] = bad
        assert L.moe_layer_forward_w4(ctypes.byref(d), P, P, None, *w, None, None, None, P, P,
                                      1 << 40, None) == status
    assert M.kernel_launches() == n0


def test_bad_product_arguments_are_refused():
    L, n0, w = M.lib(), M.kernel_launches(), _w4()
    d = _desc()
    b = ctypes.byref
    up = lambda d, *a: L.moe_expert_up_w4(b(d), *a, None)            # noqa: E731
    down = lambda d, *a: L.moe_expert_down_w4(b(d), *a, None)        # noqa: E731
    assert up(d, 8, 512, P, 8, P, None, w, P) == INVALID            # SwiGLU without gate
    assert up(d, 8, 512, P, 8, P, w, None, P) == INVALID
    assert up(d, 8, 512, None, 8, P, w, w, P) == INVALID
    assert up(d, 8, 512, P, 8, None, w, w, P) == INVALID
    assert up(d, 8, 512, P, 8, P, w, w, None) == INVALID
    assert up(d, 8, 512, P + 2, 8, P, w, w, P) == INVALID
    assert up(d, 8, 512, P, 8, P, w, w, P + 2) == INVALID
    assert up(d, 0, 512, P, 8, P, w, w, P) == INVALID
    assert up(d, 8, 500, P, 8, P, w, w, P) == UNSUPPORTED
    assert up(d, 8, 512, P, 1 << 31, P, w, w, P) == UNSUPPORTED
    assert up(d, 8, 512, P, 8, P, w, _w4(group=64), P) == UNSUPPORTED   # unlike groups
    assert up(d, 8, 512, P, 8, P, _w4(zeros=P), w, P) == UNSUPPORTED
    assert down(d, 8, 512, None, 8, P, w, P) == INVALID
    assert down(d, 8, 512, P, -1, P, w, P) == INVALID
    assert down(d, 8, 512, P, 8, P, w, None) == INVALID
    f32 = _desc(dtype="f32")
    assert up(f32, 8, 512, P, 8, P, w, w, P) == UNSUPPORTED
    assert down(f32, 8, 512, P, 8, P, w, P) == UNSUPPORTED
    layer = lambda d, *a: L.moe_layer_forward_w4(b(d), *a, None)     # noqa: E731
    assert layer(f32, P, P, None, w, w, w, None, None, None, P, P, 1 << 40) == UNSUPPORTED
    assert layer(d, P, P, None, None, w, w, None, None, None, P, P, 1 << 40) == INVALID
    assert layer(d, P, P, None, w, w, w, None, None, None, P, P, 16) == WORKSPACE
    assert layer(d, None, P, None, w, w, w, None, None, None, P, P, 1 << 40) == INVALID
    sh = M.desc_of(scaled(WORKLOADS["v3"], T=4, D=256, F=512, F_shared=64))
    assert layer(sh, P, P, None, w, w, w, None, None, None, P, P, 1 << 40) == INVALID
    # nothing to do is fine: no rows, no tokens
    assert up(d, 8, 512, P, 0, P, w, w, P) == OK
    assert down(d, 8, 512, P, 0, P, w, P) == OK
    empty = M.desc_of(scaled(WORKLOADS["mixtral"], T=0, D=256, F=512))
    assert layer(empty, P, P, None, w, w, w, None, None, None, P, P, 1 << 40) == OK
    assert M.kernel_launches() == n0


def test_bad_conversions_are_refused():
    L, n0, w = M.lib(), M.kernel_launches(), _w4()
    for n, N, K, dt, W_, want in (
            (-1, 64, 64, M.BF16, P, INVALID), (1, 0, 64, M.BF16, P, INVALID),
            (1, 64, 0, M.F32, P, INVALID), (1, 64, 64, 2, P, INVALID),
            (1, 64, 64, M.F32, None, INVALID), (1, 64, 64, M.F32, P + 4, INVALID),
            (1, 96, 64, M.F32, P, UNSUPPORTED), (1, 64, 96, M.F32, P, UNSUPPORTED),
            (1 << 24, 128, 64, M.F32, P, UNSUPPORTED), (0, 64, 64, M.F32, P, OK)):
        assert L.moe_quantize_w4(n, N, K, dt, W_, w, None) == want, (n, N, K)
        assert L.moe_dequantize_w4(n, N, K, w, dt, W_, None) == want, (n, N, K)
    assert L.moe_quantize_w4(1, 64, 64, M.F32, P, None, None) == INVALID
    assert M.kernel_launches() == n0


def test_binding_checks_shapes():
    w = M.empty_w4(2, 64, 192, 128, True, device="cpu")
    assert (w.G, w.N, w.K, tuple(w.scales.shape)) == (2, 64, 192, (2, 2, 64))
    parts = (w.codes, w.scales, w.zeros, w.row_scale)
    one = M.W4(*[t[0] for t in parts], 128)
    assert (one.G, one.N, one.K) == (1, 64, 192)
    with pytest.raises(ValueError):
        M.W4(*parts, 100)
    with pytest.raises(ValueError):
        M.W4(*parts, 32)                                              # scales of another group
    with pytest.raises(ValueError):
        M.W4(w.codes.int(), *parts[1:], 128)
    with pytest.raises(ValueError):
        M.W4(w.codes, w.scales.view(torch.uint8), w.zeros, w.row_scale, 128)
    with pytest.raises(ValueError):
        M.W4(w.codes, w.scales, w.zeros.float(), w.row_scale, 128)
    with pytest.raises(ValueError):
        M.W4(w.codes, w.scales, w.zeros, w.row_scale.double(), 128)
    with pytest.raises(ValueError):
        M.W4(w.codes.transpose(0, 1).contiguous().transpose(0, 1), *parts[1:], 128)
    x = torch.zeros(2, 64, 128)
    with pytest.raises(ValueError):
        M.moe_quantize_w4(x, w)                                       # K differs
    with pytest.raises(ValueError):
        M.moe_dequantize_w4(w, torch.zeros(2, 64, 192, dtype=torch.float16))
    with pytest.raises(ValueError):
        M.moe_quantize_w4(torch.zeros(2, 64, 192), w)                 # not on a CUDA device
    d = _desc()
    rows, off = torch.zeros(4, 256), torch.zeros(9, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.moe_expert_up_w4(d, 8, 512, rows, off, w, w, rows)
    with pytest.raises(ValueError):
        M.moe_expert_down_w4(d, 8, 512, rows, off, w, rows)


def test_a_w4_keeps_to_its_tensors():
    """Other tensors need another W4, and the addresses handed on are the tensors' present ones."""
    w = M.empty_w4(2, 64, 192, 64, True, device="cpu")
    for name in ("codes", "scales", "zeros", "row_scale", "group", "N"):
        with pytest.raises(AttributeError):
            setattr(w, name, getattr(w, name))
    moved = [torch.zeros_like(t) for t in (w.codes, w.scales, w.zeros, w.row_scale)]
    for t, m in zip((w.codes, w.scales, w.zeros, w.row_scale), moved):
        t.data = m
    c = w._ref()._obj
    assert [c.codes, c.scales, c.zeros, c.row_scale] == [m.data_ptr() for m in moved]


def test_bad_gradient_arguments_are_refused():
    L, n0 = M.lib(), M.kernel_launches()
    d = _desc()
    merge = lambda *a: L.moe_combine_backward(ctypes.byref(d), *a, None)      # noqa: E731
    disp = lambda *a: L.moe_permute_backward(ctypes.byref(d), *a, None)       # noqa: E731
    assert merge(None, P, P, P, P, P) == INVALID
    assert merge(P, P, None, P, P, P) == INVALID
    assert merge(P, P, P, None, P, P) == INVALID
    assert merge(P, P, P, P, None, None) == INVALID                  # nothing asked for
    assert merge(P, None, P, P, P, P) == INVALID                     # dgates needs y
    for i in range(6):
        a = [P] * 6
        a[i] = P + 4
        assert merge(*a) == INVALID
    assert disp(None, P, P, P) == INVALID
    assert disp(P, None, None, P) == INVALID
    assert disp(P, P, None, None) == INVALID
    for i in range(4):
        a = [P] * 4
        a[i] = P + 4
        assert disp(*a) == INVALID
    host = torch.zeros(4, 256)
    with pytest.raises(ValueError):
        M.moe_combine_backward(d, host, host, host, host, host, host)
    with pytest.raises(ValueError):
        M.moe_permute_backward(d, host, host, None, host)
    bad = _desc()
    bad.k = 9
    assert L.moe_combine_backward(ctypes.byref(bad), P, P, P, P, P, P, None) == INVALID
    assert L.moe_permute_backward(ctypes.byref(bad), P, P, None, P, None) == INVALID
    empty = M.desc_of(scaled(WORKLOADS["mixtral"], T=0, D=256, F=512))
    assert L.moe_combine_backward(ctypes.byref(empty), P, P, P, P, P, P, None) == OK
    assert L.moe_permute_backward(ctypes.byref(empty), P, P, None, P, None) == OK
    assert M.kernel_launches() == n0


def test_header_declares_the_entry_points():
    names = M.header_functions()
    for n in ("moe_combine_backward", "moe_permute_backward", "moe_quantize_w4",
              "moe_dequantize_w4", "moe_expert_up_w4", "moe_expert_down_w4",
              "moe_layer_forward_w4"):
        assert n in names and hasattr(M.lib(), n)
