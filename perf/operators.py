"""Workloads of the operators around a routed layer whose experts' products are not the built-in
bf16 ones: products with 4-bit weights, their quantisation, and the gradients of the dispatch and
of the weighted merge.

listed() names the measured cases, draw(rng) makes more of the same ranges, prepare(case, seed)
builds what a program has in hand before the call, run(state) is one pass, work(case) counts the
bytes and operations it cannot do without, and exact(case, seed) gives the outputs in 64 bits.
With own = False run() computes the operators in elementary torch operations, with own = True it
calls the framework.

4-bit matrices are [G, N, K] (one [N, K] nn.Linear weight per expert), with

    W[n, k] = row_scale[n] * scale[k // g, n] * (code[n, k] - zero[k // g, n])

code 0..15, scale e4m3, zero 0..15 (8 everywhere when it is not given) and row_scale fp32.  64
consecutive k of a row are 32 bytes, eight little-endian words; nibble i of word 2 c + j holds
k = 32 j + 8 c + (2 i if i < 4 else 2 i - 7).
"""

import math

import numpy as np
import torch

own = False

_LARGEST = 2.0 * 2 * 4096 * 4096 * 14336         # operations of the largest listed product


def listed():
    return [
        # one token of a Mixtral-wide layer (8 experts, top-2) being decoded: two experts' weights
        dict(name="up, one token", op="up", T=1, k=2, E=8, local=8, D=4096, F=14336, group=128,
             zeros=False, act="swiglu", zipf=0.0, spare=0, routing=1),
        dict(name="down, one token", op="down", T=1, k=2, E=8, local=8, D=4096, F=14336, group=128,
             zeros=False, act="swiglu", zipf=0.0, spare=0, routing=1),
        # sixteen sequences decoded at the DeepSeekMoE-16B width, zero points, small groups
        dict(name="up, 16 tokens, 64 experts", op="up", T=16, k=6, E=64, local=64, D=2048, F=1408,
             group=64, zeros=True, act="gelu", zipf=0.5, spare=3, routing=2),
        # one of eight expert-parallel ranks of the DeepSeek-V3 layer: 32 of 256 experts, 128 tokens
        dict(name="down, 128 tokens, 32 of 256", op="down", T=128, k=8, E=256, local=32, D=7168,
             F=2048, group=32, zeros=False, act="swiglu", zipf=0.3, spare=0, routing=3),
        # a prompt at the Mixtral width: the products are bound by the tensor cores
        dict(name="up, 2048 tokens", op="up", T=2048, k=2, E=8, local=8, D=4096, F=14336,
             group=128, zeros=False, act="swiglu", zipf=0.0, spare=0, routing=4),
        dict(name="down, 2048 tokens", op="down", T=2048, k=2, E=8, local=8, D=4096, F=14336,
             group=64, zeros=True, act="swiglu", zipf=0.5, spare=17, routing=5),
        # one projection of all Mixtral experts converted when a checkpoint is loaded
        dict(name="quantize, 8 x 14336 x 4096", op="quantize", E=8, N=14336, K=4096, group=128,
             zeros=False, dtype="bf16"),
        # an fp32 training copy of a narrow layer, zero points, groups that do not divide K
        dict(name="quantize, 4 x 1408 x 1984, fp32", op="quantize", E=4, N=1408, K=1984, group=128,
             zeros=True, dtype="f32"),
        # the merge of a Mixtral training batch
        dict(name="merge gradient, 4096 tokens", op="merge", T=4096, k=2, E=8, c=0, D=4096,
             dtype="bf16", capacity=0, zipf=0.0, spare=0),
        # expert choice at the DeepSeekMoE-16B width: a token has 0 to 64 experts
        dict(name="merge gradient, expert choice", op="merge", T=8190, k=0, E=64, c=256, D=2048,
             dtype="bf16", capacity=0, zipf=0.0, spare=0),
        # the dispatch of a DeepSeek-V3 training batch, top-8 of 256, a capacity that drops some
        dict(name="dispatch gradient, top-8", op="dispatch", T=4096, k=8, E=256, c=0, D=7168,
             dtype="bf16", capacity=150, zipf=0.3, spare=40, add=True),
        # the fp32 tiny layer: launch latency
        dict(name="dispatch gradient, tiny", op="dispatch", T=61, k=2, E=4, c=0, D=36,
             dtype="f32", capacity=0, zipf=0.0, spare=0, add=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["up", "up", "down", "down", "quantize", "merge", "dispatch"])
    if op in ("up", "down"):
        while True:
            E = _log_int(rng, 2, 256)
            c = dict(op=op, T=_log_int(rng, 1, 2048), k=rng.randint(1, min(8, E)), E=E,
                     local=E if rng.random() < 0.6 else rng.randint(1, E),
                     D=64 * _log_int(rng, 4, 112), F=64 * _log_int(rng, 2, 224),
                     group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                     act=rng.choice(["swiglu", "swiglu", "relu", "gelu"]),
                     zipf=rng.choice([0.0, 0.5, 1.0]), spare=rng.choice([0, 0, rng.randint(1, 200)]),
                     routing=rng.randrange(1 << 30))
            n = _counts(c)
            padded = c["local"] * max(1, int(n.max()))       # the plain form's rows
            if (c["local"] * c["D"] * c["F"] <= 8 * 4096 * 14336
                    and 4.0 * padded * c["D"] * c["F"] <= _LARGEST and n.sum() > 0):
                return c
    if op == "quantize":
        while True:
            c = dict(op=op, E=_log_int(rng, 1, 64), N=64 * _log_int(rng, 1, 224),
                     K=64 * _log_int(rng, 1, 224), group=rng.choice([32, 64, 128]),
                     zeros=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))
            if c["E"] * c["N"] * c["K"] <= 8 * 4096 * 14336:
                return c
    while True:
        f32 = rng.random() < 0.3
        E = _log_int(rng, 2, 256)
        T = _log_int(rng, 1, 16384)
        choice = rng.random() < 0.3
        c = dict(op=op, T=T, k=0 if choice else rng.randint(1, min(8, E)), E=E,
                 c=rng.randint(1, max(1, T // 4)) if choice else 0,
                 D=4 * _log_int(rng, 2, 1024) if f32 else 64 * _log_int(rng, 1, 112),
                 dtype="f32" if f32 else "bf16", capacity=0, zipf=rng.choice([0.0, 0.5, 1.0]),
                 spare=rng.choice([0, rng.randint(1, 100)]))
        rows = E * c["c"] if choice else T * c["k"]
        if not choice and rng.random() < 0.4:
            c["capacity"] = max(1, T * c["k"] // E)
        if op == "dispatch":
            c["add"] = rng.random() < 0.5
        if rows * c["D"] <= 32768 * 7168 and T * E <= 1 << 20:
            return c


# ---- routing of the products' cases: rows per expert, the same for every seed -----------------

def _counts(case):
    """Rows of each of the `local` first experts when T tokens take k of E experts each."""
    r = np.random.default_rng(case["routing"])
    T, k, E = case["T"], case["k"], case["E"]
    bias = -case["zipf"] * np.log(r.permutation(E) + 1.0)
    key = bias + r.gumbel(size=(T, E))
    top = np.argpartition(-key, k - 1, axis=1)[:, :k]
    n = np.bincount(top.ravel(), minlength=E)[:case["local"]]
    return n if n.sum() else np.eye(1, case["local"], dtype=n.dtype)[0]


# ---- 4-bit matrices ----------------------------------------------------------------------------

def _groups(W, g, fn, fill):
    """fn over the groups of g consecutive k of W [.., K] (a short last group is filled up)."""
    K = W.shape[-1]
    n = -(-K // g)
    if n * g != K:
        W = torch.nn.functional.pad(W, (0, n * g - K), value=fill)
    return fn(W.unflatten(-1, (n, g)), -1)


def _spread(s, g, K):
    """[.., groups] to [.., K]."""
    return s.repeat_interleave(g, -1)[..., :K]


def _over(x, n):
    """x / n, divided: a Python number as divisor would become a product with 1 / n."""
    return x / torch.full((), n, dtype=x.dtype, device=x.device)


def _quantize(W, g, with_zeros):
    """codes [E, N, K] (whole numbers as floats), scale and zero [E, N, groups], row_scale [E, N]"""
    K = W.shape[-1]
    if with_zeros:
        lo = _groups(W, g, torch.amin, 0.0).clamp(max=0)
        t = _over(_groups(W, g, torch.amax, 0.0).clamp(min=0) - lo, 15)
    else:
        t = _over(_groups(W.abs(), g, torch.amax, 0.0), 7)
    row = _over(t.amax(-1), 448)
    scale = torch.where(row[..., None] > 0, t / row[..., None], 0.0).float()
    scale = scale.to(torch.float8_e4m3fn).to(W.dtype)
    step = scale * row[..., None]
    inv = torch.where(step > 0, 1 / step, 0.0)
    q = (W * _spread(inv, g, K)).round_()
    if with_zeros:
        zero = (-lo * inv).round_().clamp_(0, 15)
        return q.add_(_spread(zero, g, K)).clamp_(0, 15), scale, zero, row
    return q.clamp_(-8, 7).add_(8), scale, None, row


def _pack(q):
    """[.., K] codes to [.., K / 2] bytes: k = 32 j + 8 c + 2 i + h is nibble 4 h + i of word
    2 c + j."""
    b = q.to(torch.uint8).unflatten(-1, (-1, 2, 4, 4, 2))          # .., block, j, c, i, h
    b = b.movedim(-4, -3).transpose(-1, -2).flatten(-5)              # .., block, c, j, h, i
    return b[..., 0::2] | (b[..., 1::2] << 4)


def _unpack(codes, dtype):
    b = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    b = b.unflatten(-1, (-1, 4, 2, 2, 4))                            # .., block, c, j, h, i
    return b.transpose(-1, -2).movedim(-3, -4).flatten(-5).to(dtype)


def _as_matrices(W, g, with_zeros):
    q, scale, zero, row = _quantize(W, g, with_zeros)
    return dict(codes=_pack(q),
                scales=scale.to(torch.float8_e4m3fn).transpose(-1, -2).contiguous(),
                zeros=None if zero is None else
                zero.to(torch.uint8).transpose(-1, -2).contiguous(),
                row_scale=row.contiguous(), group=g)


def _values(m, dtype, row_scale=True):
    """The [G, N, K] weights that a 4-bit matrix stands for."""
    g, K = m["group"], 2 * m["codes"].shape[-1]
    W = _unpack(m["codes"], dtype)
    if m["zeros"] is None:
        W -= 8
    else:
        W -= _spread(m["zeros"].transpose(-1, -2).to(dtype), g, K)
    W *= _spread(m["scales"].to(dtype).transpose(-1, -2), g, K)
    return W.mul_(m["row_scale"].to(dtype)[..., None]) if row_scale else W


def _random_matrices(gen, G, N, K, g, with_zeros):
    """Normal weights with a spread of row sizes, quantised (one expert at a time: memory)."""
    parts = []
    for _ in range(G):
        W = torch.randn(N, K, generator=gen, device="cuda").mul_(0.02)
        W *= torch.exp(0.3 * torch.randn(N, 1, generator=gen, device="cuda"))
        parts.append(_as_matrices(W, g, with_zeros))
    return dict(group=g, **{k: None if parts[0][k] is None else torch.stack([p[k] for p in parts])
                            for k in ("codes", "scales", "zeros", "row_scale")})


# ---- routed rows of the gradients' cases ------------------------------------------------------

def _dispatch(case, gen):
    """gates [T, K], inv [T, K] and row_src of the kept rows, as the router and the permutation
    leave them."""
    T, E, dev = case["T"], case["E"], "cuda"
    logits = torch.randn(T, E, generator=gen, device=dev)
    if case["c"]:
        gates = torch.softmax(logits, -1)
        picked = torch.topk(gates, case["c"], dim=0).indices.sort(dim=0).values.t()    # [E, c]
        row_src = (picked * E + torch.arange(E, device=dev)[:, None]).reshape(-1)
        inv = torch.full((T * E,), -1, dtype=torch.long, device=dev)
        inv[row_src] = torch.arange(row_src.numel(), device=dev)
        return gates, inv.view(T, E).int(), row_src
    k = case["k"]
    r = torch.randperm(E, generator=gen, device=dev)
    logits -= case["zipf"] * torch.log(r + 1.0)
    top, ids = torch.topk(logits, k)
    gates = torch.softmax(top, -1)
    order = torch.argsort(ids.reshape(-1), stable=True)                # rows by expert, token, slot
    n = torch.bincount(ids.reshape(-1), minlength=E)
    rank = torch.arange(T * k, device=dev) - torch.repeat_interleave(n.cumsum(0) - n, n)
    row_src = order[rank < case["capacity"]] if case["capacity"] else order
    inv = torch.full((T * k,), -1, dtype=torch.long, device=dev)
    inv[row_src] = torch.arange(row_src.numel(), device=dev)
    return gates, inv.view(T, k).int(), row_src


_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(dtype)

    op, s = case["op"], dict(case=dict(case))
    if op in ("up", "down"):
        n = _counts(case)
        rows = int(n.sum()) + case["spare"]
        G, D, F = case["local"], case["D"], case["F"]
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32,
                                    device="cuda")
        s["most"] = int(n.max())
        N, K = (F, D) if op == "up" else (D, F)
        s["a"] = normal(rows, K, std=1.0 if op == "up" else 0.3)
        s["out"] = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
        s["w"] = _random_matrices(gen, G, N, K, case["group"], case["zeros"])
        if op == "up" and case["act"] == "swiglu":
            s["w_gate"] = _random_matrices(gen, G, N, K, case["group"], case["zeros"])
    elif op == "quantize":
        E, N, K, g = case["E"], case["N"], case["K"], case["group"]
        dt = _TORCH[case["dtype"]]
        W = torch.empty(E, N, K, dtype=dt, device="cuda")
        for e in range(E):
            W[e] = (torch.randn(N, K, generator=gen, device="cuda").mul_(0.02)
                    * torch.exp(0.3 * torch.randn(N, 1, generator=gen, device="cuda")))
        u8 = dict(dtype=torch.uint8, device="cuda")
        n = -(-K // g)
        s.update(W=W, codes=torch.empty(E, N, K // 2, **u8),
                 scales=torch.empty(E, n, N, dtype=torch.float8_e4m3fn, device="cuda"),
                 zeros=torch.empty(E, n, N, **u8) if case["zeros"] else None,
                 row_scale=torch.empty(E, N, dtype=torch.float32, device="cuda"),
                 out=torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda"))
    else:
        dt = _TORCH[case["dtype"]]
        T, D = case["T"], case["D"]
        s["gates"], s["inv"], s["row_src"] = _dispatch(case, gen)
        rows = s["row_src"].numel() + case["spare"]
        if op == "merge":
            s["dout"] = normal(T, D, dtype=dt)
            s["y"] = normal(rows, D, dtype=dt)
            s["dy"] = torch.zeros(rows, D, dtype=dt, device="cuda")
            s["dgates"] = torch.zeros_like(s["gates"])
        else:
            s["dx_perm"] = normal(rows, D, dtype=dt)
            s["add"] = normal(T, D, dtype=dt) if case["add"] else None
            s["dx"] = torch.zeros(T, D, dtype=dt, device="cuda")
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _grouped(a, offsets, most, W):
    """a [rows, K] times its group's W [G, N, K], rows of a group padded to the largest's."""
    G, rows = W.shape[0], a.shape[0]
    at = offsets[:-1, None].long() + torch.arange(most, device=a.device)
    p = torch.bmm(a[at.clamp(max=rows - 1)], W.transpose(-1, -2))
    r = torch.arange(rows, device=a.device)
    g = (torch.searchsorted(offsets.long(), r, right=True) - 1).clamp(max=G - 1)
    pos = (r - offsets[g]).clamp(max=most - 1)
    return torch.where((r < offsets[-1])[:, None], p[g, pos], 0.0)


def _act(name, gate, up):
    if name == "swiglu":
        return gate * torch.sigmoid(gate) * up
    if name == "relu":
        return up.clamp(min=0)
    return 0.5 * up * (1 + torch.erf(up / math.sqrt(2.0)))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("up", "down"):
        a = s["a"].float()
        r = _grouped(a, s["offsets"], s["most"], _values(s["w"], torch.float32))
        if op == "up":
            gate = _grouped(a, s["offsets"], s["most"], _values(s["w_gate"], torch.float32)) \
                if c["act"] == "swiglu" else None
            r = _act(c["act"], gate, r)
        return {"out": r.to(torch.bfloat16)}
    if op == "quantize":
        W = s["W"].float()
        m = _as_matrices(W, c["group"], c["zeros"])
        return {"values": _values(m, torch.float32, False).mul_(m["row_scale"][..., None])
                .to(torch.bfloat16), "row_scale": m["row_scale"], "scales": m["scales"].float(),
                "zeros": m["zeros"]}
    dt, K = _TORCH[c["dtype"]], s["inv"].shape[1]
    token = s["row_src"] // K
    n = token.numel()
    if op == "merge":
        d = s["dout"].float()[token]
        dy = torch.zeros_like(s["y"])
        dy[:n] = (s["gates"].reshape(-1)[s["row_src"]][:, None] * d).to(dt)
        dg = torch.zeros_like(s["gates"])
        dg.view(-1)[s["row_src"]] = (d * s["y"][:n].float()).sum(-1)
        return {"dy": dy, "dgates": dg}
    dx = torch.zeros(c["T"], c["D"], dtype=torch.float32, device="cuda")
    if s["add"] is not None:
        dx += s["add"].float()
    dx.index_add_(0, token, s["dx_perm"][:n].float())
    return {"dx": dx.to(dt)}


# ---- the framework's calls ----------------------------------------------------------------------

def _handles(s):
    """The descriptor and the weights' handles that a program makes once."""
    import sparse_mixture_experts_warp_b200 as M
    from sparse_mixture_experts_warp_b200.workloads import Workload
    c = s["case"]
    E = min(256, c["E"])
    s["M"] = M
    if c["op"] in ("up", "down"):
        w = Workload("w4", T=c["T"], D=c["D"], E=E, F=c["F"], k=c["k"], act=c["act"])
        for key in ("w", "w_gate"):
            if key in s:
                s["own_" + key] = M.W4(**s[key])
    elif c["op"] == "quantize":
        w = None
    else:
        w = Workload("steps", T=c["T"], D=c["D"], E=E, F=64, k=c["k"], c=c["c"],
                     select="expert" if c["c"] else "token", dtype=c["dtype"])
    s["desc"] = M.desc_of(w) if w else None


def _framework(s):
    if "M" not in s:
        _handles(s)
    M, d, c = s["M"], s["desc"], s["case"]
    op = c["op"]
    if op == "up":
        M.moe_expert_up_w4(d, c["local"], c["F"], s["a"], s["offsets"], s.get("own_w_gate"),
                           s["own_w"], s["out"])
        return {"out": s["out"]}
    if op == "down":
        M.moe_expert_down_w4(d, c["local"], c["F"], s["a"], s["offsets"], s["own_w"], s["out"])
        return {"out": s["out"]}
    if op == "quantize":
        w = M.W4(s["codes"], s["scales"], s["zeros"], s["row_scale"], c["group"])
        M.moe_quantize_w4(s["W"], w)
        M.moe_dequantize_w4(w, s["out"])
        return {"values": s["out"], "row_scale": s["row_scale"], "scales": s["scales"].float(),
                "zeros": s["zeros"]}
    if op == "merge":
        M.moe_combine_backward(d, s["dout"], s["y"], s["inv"], s["gates"], s["dy"], s["dgates"])
        return {"dy": s["dy"], "dgates": s["dgates"]}
    M.moe_permute_backward(d, s["dx_perm"], s["inv"], s["add"], s["dx"])
    return {"dx": s["dx"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ---- bytes and operations -----------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("up", "down"):
        n = _counts(case)
        D, F = case["D"], case["F"]
        N, K = (F, D) if op == "up" else (D, F)
        mats = 2 if op == "up" and case["act"] == "swiglu" else 1
        groups = -(-K // case["group"]) * (2 if case["zeros"] else 1)
        rows = int(n.sum())
        return {"bytes": int((n > 0).sum()) * mats * N * (K // 2 + groups + 4)
                + 2 * rows * (K + N), "flops": 2.0 * mats * rows * N * K}
    if op == "quantize":
        w = case["E"] * case["N"] * case["K"]
        held = w // 2 + case["E"] * case["N"] * (
            4 + -(-case["K"] // case["group"]) * (2 if case["zeros"] else 1))
        # the weights in, the 4-bit form out and in again, the values out
        return {"bytes": w * (2 if case["dtype"] == "bf16" else 4) + 2 * held + 2 * w,
                "flops": 4.0 * w}
    e = 2 if case["dtype"] == "bf16" else 4
    T, D = case["T"], case["D"]
    K = case["E"] if case["c"] else case["k"]
    rows = case["E"] * case["c"] if case["c"] else T * K
    if case["capacity"]:
        rows = min(rows, case["E"] * case["capacity"])
    if op == "merge":
        return {"bytes": e * D * (T + 2 * rows) + 12 * T * K, "flops": 3.0 * rows * D}
    return {"bytes": e * D * (rows + T * (2 if case["add"] else 1)) + 4 * T * K,
            "flops": 1.0 * rows * D}


# ---- 64 bits ------------------------------------------------------------------------------------

def _nibble(m, e, dtype):
    """Codes of expert e by the layout's rule, one k of a block at a time."""
    words = m["codes"][e].view(torch.int32).long()
    out = torch.empty(words.shape[0], words.shape[1] // 8, 64, dtype=dtype, device=words.device)
    for k in range(64):
        j, c, i = k // 32, k % 32 // 8, k % 8
        at = i // 2 + 4 * (i % 2)
        out[..., k] = ((words[:, 2 * c + j::8] >> (4 * at)) & 15).to(dtype)
    return out.flatten(1)


def _weights64(m, e):
    q = _nibble(m, e, torch.float64)
    at = torch.arange(q.shape[1], device=q.device) // m["group"]
    zero = 8.0 if m["zeros"] is None else m["zeros"][e].double()[at].t()
    return (q - zero) * m["scales"][e].double()[at].t() * m["row_scale"][e].double()[:, None]


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("up", "down"):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lo = 0
        for e, n in enumerate(_counts(case).tolist()):
            if n:
                a = s["a"][lo:lo + n].double()
                z = a @ _weights64(s["w"], e).t()
                if op == "up" and case["act"] == "swiglu":
                    g = a @ _weights64(s["w_gate"], e).t()
                    z = z * g / (1 + torch.exp(-g))
                elif op == "up" and case["act"] == "relu":
                    z = torch.where(z > 0, z, 0.0)
                elif op == "up":
                    z = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
                out[lo:lo + n] = z
            lo += n
        return {"out": out}
    if op == "quantize":
        W, g = s["W"].double(), case["group"]
        K = W.shape[-1]
        most = torch.zeros(W.shape[:2], dtype=torch.float64, device="cuda")
        for k in range(0, K, g):
            part = W[..., k:k + g]
            if case["zeros"]:
                t = (part.amax(-1).clamp(min=0) - part.amin(-1).clamp(max=0)) / 15
            else:
                t = part.abs().amax(-1) / 7
            most = torch.maximum(most, t)
        # scales, zero points and codes are whole steps: values next to a border of one have no
        # 64-bit counterpart
        return {"values": None, "row_scale": most / 448, "scales": None, "zeros": None}
    T, K = s["inv"].shape
    token, slot = s["row_src"] // K, s["row_src"] % K
    if op == "merge":
        d = s["dout"].double()
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        dg = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        for r in range(0, token.numel(), 8192):
            t, j = token[r:r + 8192], slot[r:r + 8192]
            y = s["y"][r:r + t.numel()].double()
            dy[r:r + t.numel()] = s["gates"][t, j].double()[:, None] * d[t]
            dg[t, j] = torch.einsum("rd,rd->r", d[t], y)
        return {"dy": dy, "dgates": dg}
    dx = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
    if s["add"] is not None:
        dx += s["add"].double()
    for j in range(K):
        r = s["inv"][:, j].long()
        dx += torch.where((r >= 0)[:, None], s["dx_perm"][r.clamp(min=0)].double(), 0.0)
    return {"dx": dx}
