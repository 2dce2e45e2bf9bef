"""4-bit expert weights on the GPU: conversions bit for bit against the rule in fp32 torch steps,
products against 64 bits within what their arithmetic allows (w4_check.py), the rows they may
write, and the layer that runs on them."""

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
import moe_check as C
import w4_check as W
from oracle import moe_oracle as O
from sparse_mixture_experts_warp_b200.workloads import WORKLOADS, Workload, scaled

pytestmark = pytest.mark.gpu


# ---- conversions -------------------------------------------------------------------------------

@pytest.mark.parametrize("G,N,K,group,zeros,dtype", [
    (1, 64, 64, 32, False, torch.float32),
    (1, 64, 64, 128, True, torch.bfloat16),         # one short group
    (3, 128, 192, 128, False, torch.bfloat16),      # the last group is short
    (2, 64, 1344, 64, True, torch.float32),
    (2, 192, 2048, 32, True, torch.bfloat16),
    (1, 64, 18496, 128, False, torch.bfloat16),     # rows longer than a block's registers
    (1, 64, 18496, 32, True, torch.float32),
    (5, 320, 960, 64, False, torch.float32),
])
def test_quantize_and_dequantize(G, N, K, group, zeros, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(G * N + K)
    X = torch.randn(G, N, K, generator=gen, device="cuda")
    X *= torch.exp(2 * torch.randn(G, N, 1, generator=gen, device="cuda"))
    X[0, 3] = 0                                     # a row of zeros
    X[0, 5, : K // 2] = 0                           # groups of zeros
    X[0, 7] = X[0, 7].abs()                         # one sign only
    X[0, 9] = -X[0, 9].abs()
    X[0, 11] = 1e-30                                # below what a row can hold
    X[0, 13, 0] = 1e30                              # other groups vanish beside it
    X = X.to(dtype)
    w = M.empty_w4(G, N, K, group, zeros)
    M.moe_quantize_w4(X, w)
    q, s, z, row = W.quantize_plain(X, group, zeros)
    assert torch.equal(w.row_scale, row)
    assert torch.equal(w.scales.float(), s.float())
    if zeros:
        assert torch.equal(w.zeros, z)
    assert torch.equal(W.codes64(w.codes), q.double())
    v = W.values64(w)
    f = torch.empty(G, N, K, device="cuda")
    M.moe_dequantize_w4(w, f)
    assert ((f.double() - v).abs() <= 2.0 ** -24 * v.abs() + 2.0 ** -149).all()
    b = torch.empty(G, N, K, dtype=torch.bfloat16, device="cuda")
    M.moe_dequantize_w4(w, b)
    assert torch.equal(b, f.to(torch.bfloat16))


@pytest.mark.parametrize("G,N,K,group,zeros,dtype", [
    (3, 6400, 192, 64, True, torch.bfloat16),       # blocks of 8 rows, one after the other
    (3, 6400, 2048, 128, False, torch.bfloat16),
    (10, 7616, 128, 32, False, torch.float32),      # of 32 rows
    (10, 7616, 192, 128, True, torch.float32),      # (and a short group)
    (10, 7616, 576, 32, True, torch.bfloat16),
    (1, 64, 4096, 64, False, torch.bfloat16),       # of 4 rows, 4 at a time, 2 or one
    (1, 64, 6464, 64, True, torch.float32),
    (1, 64, 9152, 128, True, torch.bfloat16),
])
def test_rows_per_block(G, N, K, group, zeros, dtype):
    test_quantize_and_dequantize(G, N, K, group, zeros, dtype)


@pytest.mark.parametrize("dtype,skip", [(torch.float32, 4), (torch.bfloat16, 8)])
def test_dequantize_to_16_byte_alignment(dtype, skip):
    w = W.random_w4(2, 64, 192, 64, True, 4)
    a = torch.empty(2, 64, 192, dtype=dtype, device="cuda")
    M.moe_dequantize_w4(w, a)
    room = torch.full((skip + a.numel() + skip,), 7.0, dtype=dtype, device="cuda")
    b = room[skip:-skip].view(a.shape)
    M.moe_dequantize_w4(w, b)
    assert torch.equal(a, b)
    assert (room[:skip] == 7).all() and (room[-skip:] == 7).all()


def test_nonfinite_rows_stand_for_nan():
    X = torch.randn(1, 64, 256, device="cuda")
    X[0, 1, 7] = float("nan")
    X[0, 2, 200] = float("inf")
    X[0, 3, 0] = -float("inf")
    for zeros in (False, True):
        w = M.empty_w4(1, 64, 256, 64, zeros)
        M.moe_quantize_w4(X, w)
        f = torch.empty_like(X)
        M.moe_dequantize_w4(w, f)
        bad = torch.isnan(f).all(-1)[0]
        assert bad[1:4].all()
        assert torch.isfinite(f[0, [0, *range(4, 64)]]).all()


# ---- products ------------------------------------------------------------------------------------

def _desc(D, F, act, E=8):
    return M.desc_of(Workload("w4", T=4, D=D, E=max(E, 2), F=F, k=1, act=act))


def _run(counts, D, F, act, group, zeros, spare=0, seed=0, op="up", first=0):
    G = len(counts)
    off = [first]
    for n in counts:
        off.append(off[-1] + n)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    rows = off[-1] + spare
    N, K = (F, D) if op == "up" else (D, F)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    a = torch.randn(rows, K, generator=gen, device="cuda").to(torch.bfloat16)
    if spare:
        a[off[-1]:] = float("nan")                  # rows behind the last group are not read
    w = W.random_w4(G, N, K, group, zeros, seed + 1)
    gate = W.random_w4(G, N, K, group, zeros, seed + 2) if op == "up" and act == "swiglu" else None
    out = torch.full((rows, N), -77.0, dtype=torch.bfloat16, device="cuda")
    d = _desc(D, F, act)
    if op == "up":
        M.moe_expert_up_w4(d, G, F, a, offsets, gate, w, out)
    else:
        M.moe_expert_down_w4(d, G, F, a, offsets, w, out)
    torch.cuda.synchronize()
    assert M.get_device_error() == 0
    u, um = W.product64(a, offsets, w, rows)
    g = gm = None
    if gate is not None:
        g, gm = W.product64(a, offsets, gate, rows)
    v, e = W.expected(act if op == "up" else None, K, u, um, g, gm)
    W.check(out[first:off[-1]], v[first:off[-1]], e[first:off[-1]])
    assert (out[off[-1]:] == -77).all() and (out[:first] == -77).all()
    return out


@pytest.mark.parametrize("act", ["swiglu", "relu", "gelu"])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0, 2], [3, 0, 5, 17, 0, 8]])
def test_up(act, group, zeros, counts):
    _run(counts, 320, 192, act, group, zeros)


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False)])
@pytest.mark.parametrize("counts", [[1], [2, 0, 0, 1], [9, 16, 7, 0, 33]])
def test_down(group, zeros, counts):
    _run(counts, 192, 448, "swiglu", group, zeros, op="down")


@pytest.mark.parametrize("op", ["up", "down"])
@pytest.mark.parametrize("counts,spare", [
    ([300], 0), ([129, 0, 255, 1, 64], 5), ([31, 32, 33, 257, 16, 15], 300), ([0, 0, 513, 0], 1),
    ([1] * 40 + [0] * 7 + [70, 2], 64),
])
def test_many_rows(op, counts, spare):
    _run(counts, 384, 320, "swiglu", 64, True, spare, op=op)


@pytest.mark.parametrize("op,D,F", [("up", 64, 64), ("down", 64, 64), ("up", 64, 4096),
                                    ("down", 64, 4096), ("up", 4096, 64), ("down", 4096, 64),
                                    ("up", 7168, 128), ("down", 128, 14336)])
@pytest.mark.parametrize("counts", [[1], [2, 1], [4, 11], [40, 100]])
def test_narrow_and_long(op, D, F, counts):
    _run(counts, D, F, "swiglu", 128, False, op=op)


@pytest.mark.parametrize("op", ["up", "down"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 100, 127,
                               128, 129, 200, 255, 256, 257])
def test_every_row_count(op, n):
    _run([n], 256, 192, "gelu", 32, True, spare=3, op=op, seed=n)


@pytest.mark.parametrize("op", ["up", "down"])
def test_many_groups(op):
    _run([(i * 7) % 4 for i in range(300)], 128, 128, "swiglu", 64, False, op=op)


@pytest.mark.parametrize("op", ["up", "down"])
@pytest.mark.parametrize("rows", [1, 20, 100])
def test_most_groups(op, rows):
    """1024 groups, the most a call takes, on each kernel and its largest tiles."""
    _run([rows] * 1023 + [0], 64, 64, "relu", 64, True, op=op)


@pytest.mark.parametrize("op", ["up", "down"])
@pytest.mark.parametrize("counts", [[2, 3], [70, 30]])
def test_groups_that_start_behind_row_zero(op, counts):
    _run(counts, 192, 256, "relu", 64, False, op=op, first=5)


def test_no_rows_at_all():
    out = _run([0, 0, 0], 128, 128, "swiglu", 64, False, spare=9)
    assert (out == -77).all()


def test_extreme_values_stay_in_their_rows():
    """Infinite, NaN and huge rows reach their own outputs only."""
    D, F, d = 256, 192, _desc(256, 192, "relu")
    for n in (5, 90):
        w = W.random_w4(2, F, D, 64, True, 3)
        off = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
        a = torch.randn(2 * n, D, device="cuda").to(torch.bfloat16)
        clean = torch.empty(2 * n, F, dtype=torch.bfloat16, device="cuda")
        M.moe_expert_up_w4(d, 2, F, a, off, None, w, clean)
        b = a.clone()
        b[1] = float("nan")
        b[n] = float("inf")
        b[n + 2] = 3e38
        out = torch.empty_like(clean)
        M.moe_expert_up_w4(d, 2, F, b, off, None, w, out)
        keep = torch.ones(2 * n, dtype=torch.bool, device="cuda")
        keep[[1, n, n + 2]] = False
        assert torch.equal(out[keep], clean[keep])
        assert not torch.isfinite(out[n].float()).all()


def test_zero_rows_and_weights():
    D, F = 128, 64
    d = _desc(D, F, "swiglu")
    w = M.empty_w4(1, F, D, 32, False)
    M.moe_quantize_w4(torch.zeros(1, F, D, device="cuda"), w)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    out = torch.full((4, F), 5.0, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_up_w4(d, 1, F, torch.ones(4, D, dtype=torch.bfloat16, device="cuda"), off, w, w,
                       out)
    assert (out == 0).all()


@pytest.mark.parametrize("counts", [[1, 1], [6, 0, 12], [150, 3, 90]])
def test_results_repeat_and_streams(counts):
    """The same bits every time, on another stream, and next to a call on a third one."""
    ref = _run(counts, 512, 640, "swiglu", 128, False, seed=5)
    again = _run(counts, 512, 640, "swiglu", 128, False, seed=5)
    assert torch.equal(ref, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _run(counts, 512, 640, "swiglu", 128, False, seed=5)
    torch.cuda.synchronize()
    assert torch.equal(ref, other)


def test_large_offsets():
    """Weights of more than 2^32 codes and outputs behind 2^31 elements."""
    G, D, F, T = 40, 8192, 14336, 4                 # 4.7e9 weights a matrix
    d = _desc(D, F, "relu")
    w = M.empty_w4(G, F, D, 128, False)
    w.codes.random_(0, 256)
    w.scales.copy_(torch.ones(1, device="cuda").to(torch.float8_e4m3fn).expand(w.scales.shape))
    w.row_scale.fill_(0.01)
    rows = 160000                                   # 160000 x 14336 outputs
    off = torch.full((G + 1,), rows - T, dtype=torch.int32)
    off[G] = rows
    off = off.cuda()                                # the last group has the last rows
    a = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    a[-T:] = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    out = torch.zeros(rows, F, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_up_w4(d, G, F, a, off, None, w, out)
    last = M.W4(w.codes[-1], w.scales[-1], None, w.row_scale[-1], 128)
    v64 = W.values64(last)
    x = a[-T:].double()
    u, um = x @ v64.t(), x.abs() @ v64.abs().t()
    v, e = W.expected("relu", D, u, um)
    W.check(out[-T:], v, e)
    assert not out[-T - 8:-T].any()


def test_captured_products_replay():
    """Two captured graphs and eager calls between their replays, with inputs that change."""
    D, F = 256, 512
    d = _desc(D, F, "swiglu")
    g, u, dn = (W.random_w4(4, *s, 64, True, 9 + i) for i, s in
                enumerate(((F, D), (F, D), (D, F))))
    runs = []
    for n in (3, 80):
        off = torch.tensor([0, n, n, 2 * n, 3 * n], dtype=torch.int32, device="cuda")
        a = torch.randn(3 * n, D, device="cuda").to(torch.bfloat16)
        h = torch.empty(3 * n, F, dtype=torch.bfloat16, device="cuda")
        y = torch.empty(3 * n, D, dtype=torch.bfloat16, device="cuda")

        def step(stream=None, a=a, h=h, y=y, off=off):
            M.moe_expert_up_w4(d, 4, F, a, off, g, u, h, stream)
            M.moe_expert_down_w4(d, 4, F, h, off, dn, y, stream)

        step()
        torch.cuda.synchronize()
        cap, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=cap):
            step(cap)
        runs.append((step, graph, a, h, y))
    for _ in range(2):
        for step, graph, a, h, y in runs:
            a.copy_(torch.randn(a.shape, device="cuda"))
            h.zero_(), y.zero_()
            graph.replay()
        got = [(h.clone(), y.clone()) for _, _, _, h, y in runs]
        for (step, _, _, h, y), (gh, gy) in zip(runs, got):
            step()
            assert torch.equal(h, gh) and torch.equal(y, gy)
    assert M.get_device_error() == 0


# ---- the layer -----------------------------------------------------------------------------------

@pytest.mark.parametrize("w,group,zeros", [
    (scaled(WORKLOADS["mixtral"], T=1, D=512, F=1024), 128, False),
    (scaled(WORKLOADS["mixtral"], T=37, D=512, F=768), 64, True),
    (scaled(WORKLOADS["mixtral"], T=700, D=256, F=512), 32, False),
    (scaled(WORKLOADS["v3"], T=96, D=512, E=64, F=256, F_shared=256), 128, True),
    (scaled(WORKLOADS["switch"], T=500, D=256, E=16, F=448), 64, False),
    (scaled(WORKLOADS["ec"], T=256, D=256, E=8, F=320, c=48, clusters=4), 64, False),
])
def test_layer(w, group, zeros):
    """The layer on 4-bit weights: its routing and output against the oracle on the values the
    weights stand for, and its h, y equal, bit for bit, to the step entry points'."""
    inp = C.inputs_for(w)
    d = M.desc_of(w)
    swiglu = w.act == "swiglu"
    form = {}
    for name in ("W_gate", "W_up", "W_down"):
        X = getattr(inp, name)
        if X is None:
            continue
        form[name] = q = M.empty_w4(*X.shape, group, zeros)
        M.moe_quantize_w4(X, q)
        wide = torch.empty(X.shape, device="cuda")
        M.moe_dequantize_w4(q, wide)
        setattr(inp, name, wide)                    # fp32 values for the oracle
    ws, out = M.empty_workspace(d), torch.empty_like(inp.x)

    def layer(stream=None):
        M.moe_layer_forward_w4(d, inp.x, inp.Wg, inp.bias, form.get("W_gate"), form["W_up"],
                               form["W_down"], inp.Ws_gate, inp.Ws_up, inp.Ws_down, out, ws,
                               stream)

    layer()
    torch.cuda.synchronize()
    assert M.get_device_error() == 0
    v = M.layer_views(d, ws)
    ref = C.check_routing(w, inp, v)
    C.check_full_output(w, inp, out, ref)
    n = int(v["offsets"][-1])
    h, y = torch.zeros_like(v["h"]), torch.zeros_like(v["y"])
    M.moe_expert_up_w4(d, w.E, w.F, v["x_perm"], v["offsets"], form["W_gate"] if swiglu else None,
                       form["W_up"], h)
    M.moe_expert_down_w4(d, w.E, w.F, h, v["offsets"], form["W_down"], y)
    assert torch.equal(h[:n], v["h"][:n]) and torch.equal(y[:n], v["y"][:n])
    eager = out.clone()
    cap, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=cap):
        layer(cap)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
