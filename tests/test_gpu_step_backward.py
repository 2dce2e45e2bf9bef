"""Gradients of the dispatch and of the merge as steps of their own (moe_permute_backward,
moe_combine_backward): against 64 bits, against differences of moe_combine, and in a training
step around experts written in torch.

Tolerances.  bf16 outputs are rounded once: half a step, 2^-8 of the value (fp32: 2^-24).  dy is
one product.  A dot of D products in fp32, four vectors a lane and a tree over lanes: at most
(D / 32 + 16) additions in a row, each 2^-24 of sum |dout y|.  dx is a sum of n terms: n 2^-24 of
the sum of magnitudes."""

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M
from sparse_mixture_experts_warp_b200.workloads import Workload

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _case(T, K, D, dtype, live, seed=0, ec=False, spare=0):
    """Random one-to-one inv with a share `live` of assignments kept, rows shuffled."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")         # noqa: E731
    keep = torch.rand(T * K, generator=gen, device="cuda") < live
    n = int(keep.sum())
    inv = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    inv[keep] = torch.randperm(n, generator=gen, device="cuda").int()
    w = Workload("s", T=T, D=D, E=K if ec else max(K, 2), F=64, k=0 if ec else K, c=1 if ec else 0,
                 select="expert" if ec else "token", dtype=dtype)
    dt = DT[dtype]
    return dict(d=M.desc_of(w), T=T, K=K, D=D, n=n, inv=inv.view(T, K), dt=dt,
                gates=torch.rand(T, K, generator=gen, device="cuda"),
                dout=rnd(T, D).to(dt), rows=rnd(n + spare, D).to(dt), add=rnd(T, D).to(dt))


def _pairs(c):
    src = torch.nonzero(c["inv"].reshape(-1) >= 0).reshape(-1)
    return src // c["K"], src, c["inv"].reshape(-1)[src].long()


CASES = [
    # T, K, D, dtype, live share, expert choice
    (1, 1, 64, "bf16", 1.0, False), (1, 8, 7168, "bf16", 1.0, False), (5, 2, 4, "f32", 0.8, False),
    (64, 2, 32, "f32", 1.0, False), (333, 3, 192, "bf16", 0.7, False), (17, 32, 640, "bf16", 0.5, False),
    (100, 6, 2048, "bf16", 0.9, False), (40, 2, 4096, "bf16", 1.0, False),
    (9, 4, 20004, "f32", 0.9, False),               # rows in several passes
    (7, 2, 16448, "bf16", 1.0, False), (3, 2, 1028, "f32", 0.0, False),    # nothing kept
    (130, 256, 128, "bf16", 0.02, True), (6, 256, 64, "bf16", 1.0, True),  # every expert
    (50, 33, 516, "f32", 0.3, True), (1, 7, 8, "f32", 1.0, True),
]


@pytest.mark.parametrize("T,K,D,dtype,live,ec", CASES)
def test_merge_gradient(T, K, D, dtype, live, ec):
    c = _case(T, K, D, dtype, live, ec=ec, spare=3)
    t, src, row = _pairs(c)
    dy = torch.full_like(c["rows"], -7)
    dg = torch.full((T, K), float("nan"), device="cuda")
    M.moe_combine_backward(c["d"], c["dout"], c["rows"], c["inv"], c["gates"], dy, dg)
    g = c["gates"].reshape(-1)[src].double()
    want = g[:, None] * c["dout"][t].double()
    assert ((dy[row].double() - want).abs() <= HALF[dtype] * want.abs() * 1.001).all()
    assert (dy[c["n"]:] == -7).all()                # rows that no assignment names
    term = c["dout"][t].double() * c["rows"][row].double()
    off = (dg.reshape(-1)[src].double() - term.sum(-1)).abs()
    assert (off <= (D / 32 + 16) * 2.0 ** -24 * term.abs().sum(-1)).all()
    assert (dg[c["inv"] < 0] == 0).all()
    # each alone, and dy over y
    only = torch.full_like(dg, 3.0)
    M.moe_combine_backward(c["d"], c["dout"], c["rows"], c["inv"], c["gates"], None, only)
    assert torch.equal(only, dg)
    other = torch.full_like(dy, -7)
    M.moe_combine_backward(c["d"], c["dout"], None, c["inv"], c["gates"], other, None)
    assert torch.equal(other, dy)
    y = c["rows"].clone()
    M.moe_combine_backward(c["d"], c["dout"], y, c["inv"], c["gates"], y, only)
    assert torch.equal(only, dg) and torch.equal(y[row], dy[row])
    assert torch.equal(y[c["n"]:], c["rows"][c["n"]:])


@pytest.mark.parametrize("T,K,D,dtype,live,ec", CASES)
@pytest.mark.parametrize("add", [False, True])
def test_dispatch_gradient(T, K, D, dtype, live, ec, add):
    c = _case(T, K, D, dtype, live, seed=1, ec=ec, spare=2)
    c["rows"][c["n"]:] = float("nan")
    t, _, row = _pairs(c)
    dx = torch.full((T, D), float("nan"), dtype=c["dt"], device="cuda")
    M.moe_permute_backward(c["d"], c["rows"], c["inv"], c["add"] if add else None, dx)
    want = c["add"].double() if add else torch.zeros(T, D, dtype=torch.float64, device="cuda")
    mag = want.abs()
    want = want.index_add(0, t, c["rows"][row].double())
    mag = mag.index_add(0, t, c["rows"][row].double().abs())
    off = (dx.double() - want).abs()
    assert (off <= HALF[dtype] * want.abs() + (K + 1) * 2.0 ** -23 * mag).all()
    if add:
        over = c["add"].clone()
        M.moe_permute_backward(c["d"], c["rows"], c["inv"], over, over)
        assert torch.equal(over, dx)


def test_nan_and_inf_stay_where_they_are():
    c = _case(20, 2, 256, "bf16", 0.8, seed=4)
    t, src, row = _pairs(c)
    c["dout"][3] = float("nan")
    c["rows"][int(row[-1]), 0] = float("inf")
    dy, dg = torch.zeros_like(c["rows"]), torch.zeros_like(c["gates"])
    M.moe_combine_backward(c["d"], c["dout"], c["rows"], c["inv"], c["gates"], dy, dg)
    assert torch.equal(torch.isnan(dy).all(-1), torch.zeros_like(dy[:, 0]).bool()
                       .index_fill(0, row[t == 3], True))
    bad = ~torch.isfinite(dg)
    want = torch.zeros_like(bad)
    want.view(-1)[src[(t == 3)]] = True
    want.view(-1)[src[-1]] = True
    assert torch.equal(bad, want)
    dx = torch.zeros(20, 256, dtype=torch.bfloat16, device="cuda")
    M.moe_permute_backward(c["d"], c["rows"], c["inv"], None, dx)
    assert torch.isfinite(dx).logical_not().sum() == 1


def test_offsets_behind_2_31():
    T, K, D = 170000, 2, 7168                       # 340000 x 7168 rows
    w = Workload("s", T=T, D=D, E=2, F=64, k=K)
    d = M.desc_of(w)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    inv = torch.arange(T * K, dtype=torch.int32, device="cuda").flip(0).view(T, K).contiguous()
    gates = torch.rand(T, K, generator=gen, device="cuda")
    dout = torch.randn(T, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    y = torch.randn(T * K, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    dg = torch.empty(T, K, device="cuda")
    dx = torch.empty_like(dout)
    M.moe_permute_backward(d, y, inv, dout, dx)
    s = torch.tensor([0, 1, 77777, 149796, 149797, T - 1], device="cuda")
    rows = y[inv[s].long()].double()
    want = dout[s].double() + rows.sum(1)
    mag = dout[s].double().abs() + rows.abs().sum(1)
    assert ((dx[s].double() - want).abs() <= 2.0 ** -8 * want.abs() + 3 * 2.0 ** -23 * mag).all()
    term = dout[s].double()[:, None] * rows
    M.moe_combine_backward(d, dout, y, inv, gates, y, dg)
    off = (dg[s].double() - term.sum(-1)).abs()
    assert (off <= (D / 32 + 16) * 2.0 ** -24 * term.abs().sum(-1)).all()
    want = gates[s].double()[..., None] * dout[s].double()[:, None]
    got = y[inv[s].long()].double()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() * 1.001).all()


def _routed(w, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    d = M.desc_of(w)
    x = torch.randn(w.T, w.D, generator=gen, device="cuda").to(DT[w.dtype])
    Wg = (torch.randn(w.E, w.D, generator=gen, device="cuda") / w.D ** 0.5).to(DT[w.dtype])
    ec = w.select == "expert"
    K, A = w.E if ec else w.k, M.rows_max(d)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = torch.empty(w.E, w.c, **i32) if ec else torch.empty(w.T, K, **i32)
    gates = torch.empty(w.T, K, device="cuda")
    M.moe_route(d, x, Wg, None, ids, gates)
    xp = torch.zeros(A, w.D, dtype=x.dtype, device="cuda")
    counts, offsets = torch.zeros(w.E, **i32), torch.zeros(w.E + 1, **i32)
    row_src, inv = torch.zeros(A, **i32), torch.zeros(w.T, K, **i32)
    M.moe_permute(d, ids, x, xp, counts, offsets, row_src, inv)
    return d, x, xp, gates, inv, offsets, gen


ROUTED = [
    Workload("r", T=60, D=32, E=4, F=48, k=2, dtype="f32"),
    Workload("r", T=90, D=64, E=8, F=64, k=1, dtype="f32", gate="raw", overflow="drop",
             capacity_factor=0.7),
    Workload("r", T=48, D=36, E=6, F=64, c=13, select="expert", dtype="f32"),
]


@pytest.mark.parametrize("w", ROUTED)
def test_against_differences_of_the_merge(w):
    """The merge is linear in y and in the gates, so differences of moe_combine along a direction
    are the gradient's products with it, up to the rounding of the fp32 merges."""
    d, x, xp, gates, inv, offsets, gen = _routed(w)
    n = int(offsets[-1])
    y = torch.zeros_like(xp)
    y[:n] = torch.randn(n, w.D, generator=gen, device="cuda")
    dout = torch.randn(w.T, w.D, generator=gen, device="cuda")
    dy, dg = torch.zeros_like(y), torch.empty_like(gates)
    M.moe_combine_backward(d, dout, y, inv, gates, dy, dg)

    def loss(y, gates):
        out = torch.empty_like(x)
        M.moe_combine(d, y, inv, gates, None, out)
        return (out.double() * dout.double()).sum(), (out.double() * dout.double()).abs().sum()

    vy = torch.zeros_like(y)
    vy[:n] = torch.randn(n, w.D, generator=gen, device="cuda")
    vg = torch.randn(gates.shape, generator=gen, device="cuda")
    base, m0 = loss(y, gates)
    # each loss is off by at most (slots + 1) 2^-24 of its terms' magnitudes a few times over, the
    # sums y + vy and gates + vg by 2^-24 of theirs
    for (a, b), g, v in (((y + vy, gates), dy, vy), ((y, gates + vg), dg, vg)):
        moved, m1 = loss(a, b)
        want = (g.double() * v.double()).sum()
        mag = (g.double() * v.double()).abs().sum()
        assert (moved - base - want).abs() <= 40 * 2.0 ** -24 * (m0 + m1 + mag)
    # and the dispatch: <dx, v> against <dx_perm, permute(x + v) - permute(x)>
    dxp = torch.zeros_like(xp)
    dxp[:n] = torch.randn(n, w.D, generator=gen, device="cuda")
    dx = torch.empty_like(x)
    M.moe_permute_backward(d, dxp, inv, None, dx)
    K = inv.shape[1]
    src = torch.nonzero(inv.reshape(-1) >= 0).reshape(-1)
    order = torch.empty(n, dtype=torch.long, device="cuda")
    order[inv.reshape(-1)[src].long()] = src // K
    assert torch.equal(xp[:n], x[order])
    v = torch.randn(w.T, w.D, generator=gen, device="cuda")
    left, right = (dx.double() * v.double()), dxp[:n].double() * v[order].double()
    assert (left.sum() - right.sum()).abs() <= (K + 1) * 2.0 ** -23 * right.abs().sum()


@pytest.mark.parametrize("w", ROUTED)
@pytest.mark.parametrize("captured", [False, True])
def test_training_step_around_other_experts(w, captured):
    """moe_route, moe_permute, experts of the caller's (tanh between two matrices), moe_combine,
    and back through both gradients: dx, dgates and the expert weights' gradients against
    autograd in 64 bits with the selection fixed.  Also captured into a graph and replayed."""
    d, x, xp, gates, inv, offsets, gen = _routed(w, seed=2)
    n, K, H = int(offsets[-1]), inv.shape[1], 24
    off = offsets.tolist()
    A1 = torch.randn(w.E, w.D, H, generator=gen, device="cuda") / w.D ** 0.5
    A2 = torch.randn(w.E, H, w.D, generator=gen, device="cuda") / H ** 0.5
    dout = torch.randn(w.T, w.D, generator=gen, device="cuda")
    group = torch.zeros(xp.shape[0], dtype=torch.long, device="cuda")
    for e in range(w.E):
        group[off[e]:off[e + 1]] = e
    live = (torch.arange(xp.shape[0], device="cuda") < n)[:, None]
    one = torch.nn.functional.one_hot(group, w.E).float() * live

    def experts(rows, one, A1, A2):                 # every expert on its own rows
        t = torch.tanh(torch.einsum("re,rd,edh->rh", one, rows, A1))
        return torch.einsum("re,rh,ehd->rd", one, t, A2)

    bufs = dict(out=torch.empty_like(x), dy=torch.zeros_like(xp), dg=torch.empty_like(gates),
                dx=torch.empty_like(x))

    def step():
        stream = torch.cuda.current_stream()
        rows = xp.clone().requires_grad_(True)
        p1, p2 = A1.clone().requires_grad_(True), A2.clone().requires_grad_(True)
        y = experts(rows, one, p1, p2)
        M.moe_combine(d, y.detach(), inv, gates, None, bufs["out"], stream)
        M.moe_combine_backward(d, dout, y.detach(), inv, gates, bufs["dy"], bufs["dg"], stream)
        dxp, d1, d2 = torch.autograd.grad(y, (rows, p1, p2), bufs["dy"])
        M.moe_permute_backward(d, dxp.contiguous(), inv, None, bufs["dx"], stream)
        return d1, d2

    d1, d2 = step()
    if captured:
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d1, d2 = step()
        for b in bufs.values():
            b.fill_(5)
        bufs["dy"].zero_()
        graph.replay()
        torch.cuda.synchronize()
    X = x.double().requires_grad_(True)
    Gt = gates.double().requires_grad_(True)
    P1, P2 = A1.double().requires_grad_(True), A2.double().requires_grad_(True)
    src = torch.nonzero(inv.reshape(-1) >= 0).reshape(-1)
    row = inv.reshape(-1)[src].long()
    token = torch.empty(n, dtype=torch.long, device="cuda")
    slot = torch.empty(n, dtype=torch.long, device="cuda")
    token[row], slot[row] = src // K, src
    y = experts(X[token], one[:n].double(), P1, P2)
    out = torch.zeros_like(X).index_add(0, token, Gt.reshape(-1)[slot][:, None] * y)
    out.backward(dout.double())
    # fp32 sums of up to 500 products through four layers of them: 1e-5 of the largest
    for got, want in ((bufs["out"], out), (bufs["dx"], X.grad), (bufs["dg"], Gt.grad),
                      (d1, P1.grad), (d2, P2.grad)):
        assert (got.double() - want).abs().max() <= 1e-5 * want.abs().max()
