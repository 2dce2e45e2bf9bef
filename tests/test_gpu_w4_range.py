"""4-bit products at the ends of their ranges: token rows and row factors far from one, rows whose
elements differ by many powers of two, and the most groups a call takes on every kernel and tile.

The streaming product takes a token row as fp16 times a power of two, exact down to 2^-32 of the
row's largest element; an element below enters with an error of at most 2^-39 of the largest one,
so the sum with an error of at most 2^-39 max |a| sum |w|.  Everything else as in w4_check.py: the
inverse power and the row factor, applied one after the other, add one rounding of 2^-24 (sums are
normal numbers here; where a result is not, 2^-133 of w4_check.py covers it)."""

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
import w4_check as W
from sparse_mixture_experts_warp_b200.workloads import Workload

pytestmark = pytest.mark.gpu

# streaming, then tcgen05 with tiles of 32, 128 and 192 tokens, for two groups and K = 1024
ROWS = [3, 12, 40, 130]


def _offsets(n):
    return torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")


def _rows(n, K, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(2 * n, K, generator=gen, device="cuda"), gen


def _weights(zeros, seed, factor=1.0):
    """2 x 192 x 1024 with scales up to 256, so that sums are some 2^15 of a row."""
    w = W.random_w4(2, 192, 1024, 64, zeros, seed)
    w.scales.copy_((w.scales.float() * 32).to(torch.float8_e4m3fn))
    w.row_scale.mul_(factor)
    return w


def _check_up(act, n, a, gate, up):
    F, D = up.N, up.K
    d = M.desc_of(Workload("range", T=1, D=D, E=2, F=F, k=1, act=act))
    off, out = _offsets(n), torch.empty(2 * n, F, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_up_w4(d, 2, F, a, off, gate, up, out)
    u, um = W.product64(a, off, up, 2 * n)
    g = gm = None
    if gate is not None:
        g, gm = W.product64(a, off, gate, 2 * n)
    W.check(out, *W.expected(act, D, u, um, g, gm))


def _check_down(n, a, w):
    d = M.desc_of(Workload("range", T=1, D=w.N, E=2, F=w.K, k=1))
    off, out = _offsets(n), torch.empty(2 * n, w.N, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_down_w4(d, 2, w.K, a, off, w, out)
    y, ym = W.product64(a, off, w, 2 * n)
    v, e = W.expected(None, w.K, y, ym)
    most, total = a.double().abs().amax(-1), W.values64(w).abs().sum(-1)
    small = 2.0 ** -39 * most[:, None] * total.repeat_interleave(n, 0)
    W.check(out, v, e + small)
    return out, v, ym


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("rows,factors", [(-100, -30), (-100, 0), (-100, 60), (-60, -80), (0, -110),
                                          (0, 60), (100, -90), (90, 0), (100, -115)])
def test_magnitudes_of_rows_and_factors(n, rows, factors):
    """Rows around 2^rows and row factors around 2^(factors - 9)."""
    a, _ = _rows(n, 1024, n)
    _check_down(n, (a * 2.0 ** rows).to(torch.bfloat16), _weights(True, n + 1, 2.0 ** factors))


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_small_rows_through_an_activation(n, act):
    a, _ = _rows(n, 1024, n)
    _check_up(act, n, (a * 2.0 ** -100).to(torch.bfloat16), None,
              _weights(False, n + 1, 2.0 ** -30))


@pytest.mark.parametrize("n", ROWS)
def test_small_gate_times_large_up(n):
    a, _ = _rows(n, 1024, n)
    _check_up("swiglu", n, (a * 2.0 ** -100).to(torch.bfloat16), _weights(True, 1, 2.0 ** -30),
              _weights(True, 2, 2.0 ** 100))


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("spread", [20, 30, 36])
def test_elements_of_unlike_size_in_a_row(n, spread):
    """One outlier of 2^spread in every row.  Even outputs have no weight outside k = 192 .. 319,
    so most of them do not see it; while no element is below 2^-32 of it (2^-8 / 2^20), they come
    out as if it were not there."""
    a, gen = _rows(n, 1024, n + spread)
    a = torch.where(a.abs() < 2.0 ** -8, 2.0 ** -8, a)
    at = torch.randint(0, 1024, (2 * n,), generator=gen, device="cuda")
    a[torch.arange(2 * n, device="cuda"), at] = 2.0 ** spread
    w = _weights(False, n)
    w.codes[:, ::2] = 0x88                          # code 8 is zero
    w.codes[:, ::2, 96:160] = 0x91                  # k 192 .. 319
    out, v, mag = _check_down(n, a.to(torch.bfloat16), w)
    if spread == 20:
        quiet = (at < 192) | (at >= 320)
        assert quiet.any()
        out, v, mag = (t[quiet, ::2] for t in (out, v, mag))
        e = W.sum_error(1024, mag, v)
        W.check(out, v, e + 2.0 ** -8 * (v.abs() + e))


def test_a_row_of_subnormal_numbers():
    """In the streaming product, which brings them to the middle of fp16's range."""
    n = ROWS[0]
    a, _ = _rows(n, 1024, n)
    a[0] *= 2.0 ** -130
    a[1] = 0
    a = a.to(torch.bfloat16)
    assert 0 < a[0].float().abs().amax() < 2.0 ** -126
    _check_down(n, a, _weights(False, n, 2.0 ** 40))


@pytest.mark.parametrize("n", ROWS)
def test_a_row_of_largest_numbers(n):
    """2^122 around, on weights of code - zero 0 or 1 and scales below 2^-4, so that the magnitudes
    add up to some 2^125."""
    a, _ = _rows(n, 1024, n)
    a[0] = (a[0] * 2.0 ** 122).clamp(-2.0 ** 123, 2.0 ** 123)
    w = _weights(False, n, 2.0 ** -12)
    w.scales.copy_((w.scales.float() * 2.0 ** -13).to(torch.float8_e4m3fn))
    w.codes.bitwise_and_(0x11).bitwise_or_(0x88)
    _check_down(n, a.to(torch.bfloat16), w)


@pytest.mark.parametrize("op", ["up", "down"])
@pytest.mark.parametrize("rows", [1, 8, 20, 130])
def test_most_groups_on_every_kernel(op, rows):
    """1024 groups on the streaming kernel and on tiles of 32, 128 and 192 tokens: the largest
    group tables beside the largest rings."""
    G, N, K = 1024, 64, 64
    counts = torch.tensor([rows] * (G - 2) + [0, rows + 3], device="cuda")
    off = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
    n = int(off[-1])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    a = torch.randn(n, K, generator=gen, device="cuda").to(torch.bfloat16)
    gate, w = (W.random_w4(G, N, K, 64, True, s) for s in (1, 2))
    out = torch.zeros(n, N, dtype=torch.bfloat16, device="cuda")
    d = M.desc_of(Workload("groups", T=1, D=64, E=2, F=64, k=1))
    if op == "up":
        M.moe_expert_up_w4(d, G, N, a, off, gate, w, out)
    else:
        M.moe_expert_down_w4(d, G, K, a, off, w, out)
    assert M.get_device_error() == 0
    group = torch.repeat_interleave(torch.arange(G, device="cuda"), counts)
    v, g = W.values64(w), W.values64(gate)
    for lo in range(0, n, 8192):
        rows_ = slice(lo, lo + 8192)
        x = a[rows_].double()[:, None]
        sums = lambda m: (x * m[group[rows_]]).sum(-1)              # noqa: E731
        mags = lambda m: (x * m[group[rows_]]).abs().sum(-1)        # noqa: E731
        if op == "up":
            want = W.expected("swiglu", K, sums(v), mags(v), sums(g), mags(g))
        else:
            want = W.expected(None, K, sums(v), mags(v))
        W.check(out[rows_], *want)
