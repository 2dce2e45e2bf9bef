"""Helpers of the 4-bit weight tests: the form written out in 64 bits, one nibble rule at a time,
and the error that a product's arithmetic allows.

Tolerance of one output (derived, per element):
  * weights and rows enter the sums exactly; a sum of K products in fp32, 16 at a time, is off by
    at most (K / 16 + 16) 2^-23 S with S = sum |w x| (each of the K / 16 accumulations and the 16
    additions inside one loses at most 2^-23 of a partial sum, itself at most S);
  * row_scale adds 2^-24 of the result;
  * |d silu| <= 1.1, |d gelu| <= 1.13, |d relu| <= 1 carry the sums' errors to the output, and the
    activation's own exponential / erf / division add at most 2^-19 of its operands;
  * the bf16 rounding adds half a step, 2^-8 of the value.
"""

from __future__ import annotations

import math

import torch

import sparse_mixture_experts_warp_b200 as M


def codes64(codes):
    """[.., K / 2] bytes to [.., K] codes, float64: k = 32 j + 8 c + e is nibble e / 2 + 4 (e % 2)
    of little-endian word 2 c + j of its 64."""
    b = codes.long()
    word = sum(b[..., i::4] << (8 * i) for i in range(4))          # [.., K / 8]
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1] // 64, 64, dtype=torch.float64,
                      device=codes.device)
    for k in range(64):
        j, c, e = k // 32, (k % 32) // 8, k % 8
        out[..., k] = ((word[..., 2 * c + j::8] >> (4 * (e // 2 + 4 * (e % 2)))) & 15).double()
    return out.flatten(-2)


def values64(w, row_scale=True):
    """[G, N, K] values of a M.W4."""
    q = codes64(w.codes)
    at = torch.arange(w.K, device=q.device) // w.group
    zero = 8.0 if w.zeros is None else w.zeros.double()[..., at, :].transpose(-1, -2)
    v = (q - zero) * w.scales.double()[..., at, :].transpose(-1, -2)
    return v * w.row_scale.double()[..., None] if row_scale else v


def quantize_plain(W, group, zeros):
    """The rule of moe_quantize_w4 in fp32 torch steps: (codes [G, N, K], scales, zeros, row_scale)
    with scales and zeros [G, groups, N]."""
    W = W.float()
    K = W.shape[-1]
    # a tensor as divisor: torch turns a division by a number into a product with 1 / number
    n15, n7, n448 = torch.tensor([15.0, 7.0, 448.0], device=W.device).unbind()
    n = -(-K // group)
    g = torch.nn.functional.pad(W, (0, n * group - K)).unflatten(-1, (n, group))
    lo = g.amin(-1).clamp(max=0)
    t = (g.amax(-1).clamp(min=0) - lo) / n15 if zeros else g.abs().amax(-1) / n7
    row = t.amax(-1)
    row = torch.where(row < 2.0 ** -100, 0.0, row / n448)
    scale = torch.where(row[..., None] > 0, t / row[..., None], 0.0).to(torch.float8_e4m3fn)
    step = scale.float() * row[..., None]
    inv = torch.where(step > 0, 1 / step, 0.0)
    wide = lambda s: s.repeat_interleave(group, -1)[..., :K]          # noqa: E731
    q = torch.round(W * wide(inv))
    zero = None
    if zeros:
        zero = torch.round(-lo * inv).clamp(0, 15)
        q = (q + wide(zero)).clamp(0, 15)
        zero = zero.to(torch.uint8).transpose(-1, -2).contiguous()
    else:
        q = q.clamp(-8, 7) + 8
    return q, scale.transpose(-1, -2).contiguous(), zero, row


def random_w4(G, N, K, group=128, zeros=False, seed=0, std=0.05, device="cuda"):
    """Random codes, scales over the whole e4m3 range in use, row factors of both signs' size."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    w = M.empty_w4(G, N, K, group, zeros, device)
    w.codes.copy_(torch.randint(0, 256, w.codes.shape, generator=gen, device=device))
    w.scales.copy_((torch.rand(w.scales.shape, generator=gen, device=device) * 8 + 0.01)
                   .to(torch.float8_e4m3fn))
    if zeros:
        w.zeros.copy_(torch.randint(0, 16, w.zeros.shape, generator=gen, device=device))
    w.row_scale.copy_(torch.exp(torch.randn(w.row_scale.shape, generator=gen, device=device))
                      * std / 20)
    return w


def groups_of(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def product64(a, offsets, w, rows):
    """(sums, sums of magnitudes), [rows, N] float64, rows outside the groups zero."""
    out = torch.zeros(rows, w.N, dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(out)
    for e, lo, hi in groups_of(offsets):
        v = values64(M.W4(w.codes[e], w.scales[e], None if w.zeros is None else w.zeros[e],
                          w.row_scale[e], w.group))
        x = a[lo:hi].double()
        out[lo:hi] = x @ v.t()
        mag[lo:hi] = x.abs() @ v.abs().t()
    return out, mag


def sum_error(K, mag, value):
    return (K / 16 + 16) * 2.0 ** -23 * mag + 2.0 ** -24 * value.abs()


def expected(act, K, u, um, g=None, gm=None):
    """(value, allowed error) of the up product's output from its sums and magnitudes."""
    du = sum_error(K, um, u)
    if act == "swiglu":
        dg = sum_error(K, gm, g)
        s = g * torch.sigmoid(g)
        v = s * u
        e = 1.1 * u.abs() * dg + s.abs() * du + 1.1 * dg * du + 2.0 ** -19 * v.abs()
    elif act == "relu":
        v, e = u.clamp(min=0), du
    elif act == "gelu":
        v = 0.5 * u * torch.special.erfc(-u / math.sqrt(2.0))
        e = 1.13 * du + 2.0 ** -19 * u.abs()
    else:
        v, e = u, du
    # bf16 half step; 2^-133 is half the smallest bf16 step
    return v, e + 2.0 ** -8 * (v.abs() + e) + 2.0 ** -133


def check(got, value, error):
    off = (got.double() - value).abs()
    bad = ~(off <= error)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off, the worst "
                           f"{float((off / error).nan_to_num(1e30).max()):.3g} times what is allowed")
