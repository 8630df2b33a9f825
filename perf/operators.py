"""Measured cases of the operators around a mixture-of-experts MLP: routing
(tokens sorted by expert, and back), the experts' products over ragged groups
of rows, and activation checkpoints in 8 bits with their use in the backward
pass.

`run` computes a pass either in plain torch operations (own = False) or
through the library's entry points (own = True).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLK = 32  # columns that share one scale of an 8-bit checkpoint


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoder that answers one request: one token to its experts and back
        dict(name="route_one", op="route", tokens=1, topk=8, groups=64, cols=4096, dtype="bf16",
             drop=0.0),
        # a prompt batch, or a training step's forward pass
        dict(name="route_batch", op="route", tokens=8192, topk=4, groups=64, cols=4096,
             dtype="bf16", drop=0.0),
        # odd sizes, with slots dropped by an expert's capacity
        dict(name="route_odd", op="route", tokens=1999, topk=3, groups=13, cols=1027, dtype="f16",
             drop=0.1),
        # the training step's gradients of the same two steps
        dict(name="route_grad", op="route_grad", tokens=8192, topk=4, groups=64, cols=4096,
             dtype="bf16", drop=0.02),
        # one token through its experts: four rows in four groups
        dict(name="rows_one", op="rows", rows=4, n=1024, k=2048, groups=32, dtype="bf16",
             b_layout="col"),
        # 32 requests that decode together, over 32 experts
        dict(name="rows_decode", op="rows", rows=128, n=4096, k=2048, groups=32, dtype="bf16",
             b_layout="col"),
        # the first product of a training step's experts
        dict(name="rows_batch", op="rows", rows=16384, n=4096, k=4096, groups=16, dtype="bf16",
             b_layout="col"),
        # the gradient of the rows, ragged sizes
        dict(name="rows_grad", op="rows", rows=5003, n=2056, k=1416, groups=24, dtype="f16",
             b_layout="row"),
        # the gradient of the experts' weights, added to fp32 gradients
        dict(name="weights_grad", op="weights", rows=16384, m=4096, n=2048, groups=16,
             dtype="bf16", eight=False, accumulate=True),
        # the same from inputs that were kept in 8 bits
        dict(name="weights_grad8", op="weights", rows=16384, m=4096, n=2048, groups=16,
             dtype="bf16", eight=True, accumulate=False),
        # the experts' activation, its inputs kept in 8 bits and brought back
        dict(name="swiglu_save", op="swiglu", rows=16384, cols=2048, dtype="bf16"),
        # its gradient, from the kept codes; ragged sizes
        dict(name="swiglu_grad", op="swiglu_grad", rows=9001, cols=1416, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _limits():
    b = f = 0
    for c in listed():
        w = work(c)
        b, f = max(b, w["bytes"]), max(f, w["flops"])
    return b, f


def draw(rng):
    lim = _limits()
    while True:
        op = rng.choice(["route", "route_grad", "rows", "rows", "weights", "weights", "swiglu",
                         "swiglu_grad"])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        # a model's widths come in multiples of 8; the routing and the
        # checkpoints also meet odd ones
        wide = lambda lo, hi: max(8, 8 * (_log(rng, lo, hi) // 8))
        some = lambda lo, hi: wide(lo, hi) if rng.random() < 0.6 else _log(rng, lo, hi)
        if op in ("route", "route_grad"):
            groups = _log(rng, 4, 256)
            c = dict(op=op, tokens=_log(rng, 1, 8192), topk=rng.randint(1, min(8, groups)),
                     groups=groups, cols=some(64, 8192), dtype=dtype,
                     drop=rng.choice([0.0, 0.0, 0.05, 0.3]))
        elif op == "rows":
            c = dict(op=op, rows=_log(rng, 1, 16384), n=wide(64, 8192), k=wide(64, 8192),
                     groups=_log(rng, 1, 64), dtype=dtype, b_layout=rng.choice(["col", "row"]))
        elif op == "weights":
            c = dict(op=op, rows=_log(rng, 1, 16384), m=wide(64, 8192), n=wide(64, 8192),
                     groups=_log(rng, 1, 64), dtype=dtype, eight=rng.random() < 0.5,
                     accumulate=rng.random() < 0.5)
        else:
            c = dict(op=op, rows=_log(rng, 1, 16384), cols=some(64, 8192), dtype=dtype)
        w = work(c)
        if w["bytes"] <= lim[0] and w["flops"] <= lim[1]:
            return c


def work(case):
    """Bytes and operations one pass cannot do without."""
    op = case["op"]
    if op in ("route", "route_grad"):
        t, s, h = case["tokens"], case["tokens"] * case["topk"], case["cols"]
        if op == "route":
            # ids, the three lists, X and Ys read, Xs and Y written, weights
            return {"bytes": 8 * s + 4 * (2 * s + case["groups"] + 1) + 2 * (2 * t * h + 2 * s * h)
                    + 4 * s, "flops": 2 * s * h}
        # dY, Ys, dXs read, dYs and dX written; places, weights, their gradient
        return {"bytes": 2 * (2 * t * h + 3 * s * h) + 12 * s, "flops": 4 * s * h}
    if op == "rows":
        r, n, k, g = case["rows"], case["n"], case["k"], min(case["groups"], case["rows"])
        return {"bytes": 2 * (r * k + r * n + g * n * k), "flops": 2 * r * n * k}
    if op == "weights":
        r, m, n, g = case["rows"], case["m"], case["n"], case["groups"]
        b = r * n + r * -(-n // BLK) if case["eight"] else 2 * r * n
        return {"bytes": 2 * r * m + b + 4 * g * m * n * (2 if case["accumulate"] else 1),
                "flops": 2 * r * m * n}
    r, c = case["rows"], case["cols"]
    q = 2 * r * c + r * -(-2 * c // BLK)
    if op == "swiglu":
        # [g|u] read, h, codes and scales written, then read and restored
        return {"bytes": 2 * 3 * r * c + 2 * q + 2 * 2 * r * c, "flops": 8 * r * c}
    # codes, scales and dh read, [dg|du] and h written
    return {"bytes": q + 2 * (r * c + 3 * r * c), "flops": 16 * r * c}


# ---------------------------------------------------------------- inputs

def _offsets(gen, rows, groups):
    """Group bounds of a skewed choice: some experts popular, some idle."""
    load = torch.randn(groups, generator=gen) * 0.7
    ids = torch.multinomial(torch.softmax(load, 0), rows, replacement=True, generator=gen)
    counts = torch.bincount(ids, minlength=groups)
    off = torch.zeros(groups + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return off


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(DT[dtype])


def _pow2(e):
    """2^e of an integer tensor, in 64 bits (the exponent's bits: exact)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _quantise(x):
    """Codes (uint8) and scales (uint8, 127 + e) of x in blocks of 32 columns:
    e the smallest integer with amax <= 448 * 2^e, 0 for a block of zeros."""
    rows, cols = x.shape
    nb = -(-cols // BLK)
    p = torch.zeros(rows, nb * BLK, dtype=torch.float32, device=x.device)
    p[:, :cols] = x.float()
    p = p.view(rows, nb, BLK)
    amax = p.abs().amax(2)
    m, ex = torch.frexp(amax)  # amax = m 2^ex, m in [0.5, 1)
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).to(torch.int32)
    q = (p.double() * _pow2(-e).unsqueeze(2)).float().to(torch.float8_e4m3fn)
    codes = q.view(torch.uint8).view(rows, nb * BLK)[:, :cols].contiguous()
    return codes, (e + 127).to(torch.uint8)


def _values(codes, scales, cols):
    """The values that codes and scales stand for, in 64 bits."""
    s = _pow2(scales.to(torch.int32) - 127).repeat_interleave(BLK, dim=1)[:, :cols]
    return codes.view(torch.float8_e4m3fn).float().double() * s


def _restore(codes, scales, cols, dtype):
    big = torch.finfo(DT[dtype]).max
    return _values(codes, scales, cols).clamp(-big, big).float().to(DT[dtype])


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    op, s = case["op"], {"case": case}
    dt = case["dtype"]
    empty = lambda shape, d: torch.empty(shape, dtype=d, device="cuda")
    if op in ("route", "route_grad"):
        t, k, g, h = case["tokens"], case["topk"], case["groups"], case["cols"]
        # a router's choice: the k best of g scores, popular experts among them
        score = torch.randn(t, g, generator=cpu) + 0.5 * torch.randn(g, generator=cpu)
        w, ids = torch.topk(score, k, dim=1)
        if case["drop"]:
            ids[torch.rand(t, k, generator=cpu) < case["drop"]] = -1
        s["weights"] = torch.softmax(w, 1).cuda()
        s["ids"] = ids.cuda()
        if op == "route":
            s["X"] = _normal(gen, (t, h), dt)
            s["Ys"] = _normal(gen, (t * k, h), dt)
            s["offsets"] = empty(g + 1, torch.int32)
            s["order"] = empty(t * k, torch.int32)
            s["pos"] = empty((t, k), torch.int32)
            # rows past the last group keep what they held
            s["Xs"] = torch.zeros((t * k, h), dtype=DT[dt], device="cuda")
            s["Y"] = empty((t, h), DT[dt])
        else:
            s["pos"] = _places(s["ids"], g)[2]
            s["dY"] = _normal(gen, (t, h), dt)
            s["Ys"] = _normal(gen, (t * k, h), dt)
            s["dXs"] = _normal(gen, (t * k, h), dt)
            s["dYs"] = torch.zeros((t * k, h), dtype=DT[dt], device="cuda")
            s["dw"] = empty((t, k), torch.float32)
            s["dX"] = empty((t, h), DT[dt])
        if own:
            from sparse_tiled_gemm_amd import gemm as G
            n = G.gemm_moe_sort_workspace(t, k, g)
            s["workspace"] = empty(max(n, 1), torch.uint8)
        return s
    if op in ("rows", "weights"):
        r, g, n = case["rows"], case["groups"], case["n"]
        off = _offsets(cpu, r, g)
        s["bounds"], s["offsets"] = off.tolist(), off.cuda()
        if op == "rows":
            k = case["k"]
            s["A"] = _normal(gen, (r, k), dt)
            shape = (g, n, k) if case["b_layout"] == "col" else (g, k, n)
            s["B"] = empty(shape, DT[dt])
            for i in range(g):
                s["B"][i] = _normal(gen, shape[1:], dt, k ** -0.5)
            s["D"] = empty((r, n), DT[dt])
        else:
            m = case["m"]
            s["A"] = _normal(gen, (r, m), dt)
            b = _normal(gen, (r, n), dt)
            s["B"], s["scales"] = _quantise(b) if case["eight"] else (b, None)
            s["D"] = empty((g, m, n), torch.float32)
            if case["accumulate"]:
                # the fp32 gradient so far
                s["D0"] = torch.randn((g, m, n), generator=gen, device="cuda")
        if own:
            from sparse_tiled_gemm_amd import gemm as G
            if op == "rows":
                d = G.make_grouped_desc("rows", r, n, case["k"], g, dt, dt, dt,
                                        b_layout=case["b_layout"])
            else:
                d = G.make_grouped_desc("weights", r, n, case["m"], g, dt,
                                        "e4m3" if case["eight"] else dt, "f32",
                                        has_c=case["accumulate"])
            s["plan"] = G.gemm_grouped_plan(d)
        return s
    r, c = case["rows"], case["cols"]
    gu = _normal(gen, (r, 2 * c), dt, 1.5)
    s["H"] = empty((r, c), DT[dt])
    nb = -(-2 * c // BLK)
    if op == "swiglu":
        s["GU"] = gu
        s["q"], s["scales"] = empty((r, 2 * c), torch.uint8), empty((r, nb), torch.uint8)
        s["back"] = empty((r, 2 * c), DT[dt])
    else:
        s["q"], s["scales"] = _quantise(gu)
        s["dH"] = _normal(gen, (r, c), dt)
        s["dGU"] = empty((r, 2 * c), DT[dt])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _places(ids, groups):
    """Bounds, order and places of slots sorted by group, first come first."""
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < groups)
    hot = flat.unsqueeze(1) == torch.arange(groups, device=flat.device)
    rank = torch.cumsum(hot.to(torch.int32), 0, dtype=torch.int32)
    counts = rank[-1] if len(flat) else torch.zeros(groups, dtype=torch.int32, device=flat.device)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.cumsum(counts, 0)
    at = flat.clamp(0, groups - 1).unsqueeze(1)
    pos = offsets[at.squeeze(1)] + rank.gather(1, at).squeeze(1) - 1
    pos = torch.where(ok, pos, torch.full_like(pos, -1)).to(torch.int32)
    # dropped slots land on one entry past the end, which is cut off
    order = torch.full((len(flat) + 1,), -1, dtype=torch.int32, device=flat.device)
    slots = torch.arange(len(flat), dtype=torch.int32, device=flat.device)
    order[torch.where(ok, pos, torch.full_like(pos, len(flat))).long()] = slots
    order[-1] = -1
    return offsets, order[:-1], pos.view(ids.shape)


def _scatter_rows(out, pos, rows):
    """out with row pos[s] = rows[s] for the slots that have a place."""
    full = torch.cat([out, torch.zeros_like(out[:1])])
    at = pos.reshape(-1).long()
    full[torch.where(at >= 0, at, torch.full_like(at, len(out)))] = rows
    return full[:-1]


def _gather_rows(rows, pos):
    """rows[pos] in fp32, zero where a slot has no place: tokens x topk x cols."""
    x = rows[pos.clamp(min=0).long()].float()
    return torch.where((pos >= 0).unsqueeze(2), x, torch.zeros_like(x))


def _plain_route(s):
    c = s["case"]
    offsets, order, pos = _places(s["ids"], c["groups"])
    x = s["X"].unsqueeze(1).expand(-1, c["topk"], -1).reshape(-1, c["cols"])
    Xs = _scatter_rows(s["Xs"], pos, x)
    Y = (_gather_rows(s["Ys"], pos) * s["weights"].unsqueeze(2)).sum(1)
    return [offsets, order, pos, Xs, Y.to(DT[c["dtype"]])]


def _plain_route_grad(s):
    c = s["case"]
    dy = s["dY"].float().unsqueeze(1)
    dYs = (dy * s["weights"].unsqueeze(2)).to(DT[c["dtype"]]).reshape(-1, c["cols"])
    dw = (_gather_rows(s["Ys"], s["pos"]) * dy).sum(2)
    dX = _gather_rows(s["dXs"], s["pos"]).sum(1).to(DT[c["dtype"]])
    return [_scatter_rows(s["dYs"], s["pos"], dYs), dw, dX]


def _plain_rows(s):
    c, out = s["case"], []
    for g, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if a < b:
            w = s["B"][g].float()
            w = w.t() if c["b_layout"] == "col" else w
            out.append((s["A"][a:b].float() @ w).to(DT[c["dtype"]]))
    return torch.cat(out)


def _plain_weights(s):
    c = s["case"]
    # an 8-bit value of a 16-bit tensor is a 16-bit value again
    B = _restore(s["B"], s["scales"], c["n"], c["dtype"]) if c["eight"] else s["B"]
    D = torch.empty_like(s["D"])
    for g, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        D[g] = s["A"][a:b].float().t() @ B[a:b].float()
        if c["accumulate"]:
            D[g] += s["D0"][g]
    return D


def _plain_swiglu(s):
    c = s["case"]
    g, u = s["GU"][:, :c["cols"]].float(), s["GU"][:, c["cols"]:].float()
    H = g / (1 + torch.exp(-g)) * u
    q, e = _quantise(s["GU"])
    return [H.to(DT[c["dtype"]]), e, _restore(q, e, 2 * c["cols"], c["dtype"])]


def _plain_swiglu_grad(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    v = _values(s["q"], s["scales"], 2 * c["cols"]).float()
    g, u, dh = v[:, :c["cols"]], v[:, c["cols"]:], s["dH"].float()
    sg = 1 / (1 + torch.exp(-g))
    dg = dh * u * sg * (1 + g * (1 - sg))
    return [torch.cat([dg, dh * g * sg], 1).to(dt), (g * sg * u).to(dt)]


_plain = {"route": _plain_route, "route_grad": _plain_route_grad, "rows": _plain_rows,
          "weights": _plain_weights, "swiglu": _plain_swiglu, "swiglu_grad": _plain_swiglu_grad}


def _own_route(s):
    from sparse_tiled_gemm_amd import gemm as G
    c = s["case"]
    t, k, h, rows = c["tokens"], c["topk"], c["cols"], c["tokens"] * c["topk"]
    G.gemm_moe_dispatch(t, k, c["groups"], h, c["dtype"], s["ids"], s["X"], h, s["offsets"],
                        s["order"], s["pos"], s["Xs"], h, s["workspace"], id_bytes=8)
    G.gemm_moe_combine(t, k, h, c["dtype"], s["pos"], s["weights"], s["Ys"], h, rows, s["Y"], h)
    return [s["offsets"], s["order"], s["pos"], s["Xs"], s["Y"]]


def _own_route_grad(s):
    from sparse_tiled_gemm_amd import gemm as G
    c = s["case"]
    t, k, h, rows = c["tokens"], c["topk"], c["cols"], c["tokens"] * c["topk"]
    G.gemm_moe_combine_backward(t, k, h, c["dtype"], s["pos"], s["weights"], s["dY"], h, s["Ys"], h,
                                rows, s["dYs"], h, s["dw"])
    G.gemm_moe_combine(t, k, h, c["dtype"], s["pos"], None, s["dXs"], h, rows, s["dX"], h)
    return [s["dYs"], s["dw"], s["dX"]]


def _own_rows(s):
    from sparse_tiled_gemm_amd import gemm as G
    G.gemm_grouped_run(s["plan"], s["A"], s["B"], None, s["offsets"], None, s["D"])
    return s["D"]


def _own_weights(s):
    from sparse_tiled_gemm_amd import gemm as G
    G.gemm_grouped_run(s["plan"], s["A"], s["B"], s["scales"], s["offsets"],
                       s["D0"] if s["case"]["accumulate"] else None, s["D"])
    return s["D"]


def _own_swiglu(s):
    from sparse_tiled_gemm_amd import gemm as G
    r, c, dt = s["case"]["rows"], s["case"]["cols"], s["case"]["dtype"]
    G.gemm_swiglu(r, c, dt, s["GU"], 2 * c, s["H"], c, s["q"], s["scales"])
    G.gemm_q8_load(r, 2 * c, dt, s["q"], s["scales"], s["back"], 2 * c)
    return [s["H"], s["scales"], s["back"]]


def _own_swiglu_grad(s):
    from sparse_tiled_gemm_amd import gemm as G
    r, c, dt = s["case"]["rows"], s["case"]["cols"], s["case"]["dtype"]
    G.gemm_swiglu_backward(r, c, dt, s["q"], s["scales"], s["dH"], c, s["dGU"], 2 * c, s["H"], c)
    return [s["dGU"], s["H"]]


_own = {"route": _own_route, "route_grad": _own_route_grad, "rows": _own_rows,
        "weights": _own_weights, "swiglu": _own_swiglu, "swiglu_grad": _own_swiglu_grad}


# ---------------------------------------------------------------- 64 bits

def _e4m3(x):
    """x rounded to the values of E4M3, ties to even (|x| <= 448)."""
    _, ex = torch.frexp(x)
    step = _pow2(torch.clamp(ex - 1, min=-6) - 3)  # spacing at |x|
    return torch.round(x / step) * step


def _checkpoint64(x):
    """Exponents and values of the 8-bit form of x (64 bits), by its definition."""
    rows, cols = x.shape
    vals, exps = torch.empty_like(x), []
    for b in range(0, cols, BLK):
        blk = x[:, b:b + BLK]
        amax = blk.abs().max(1).values
        e = torch.ceil(torch.log2(torch.where(amax > 0, amax / 448, torch.ones_like(amax))))
        # the logarithm may be off by one next to a power of two
        e = torch.where(amax > 448 * _pow2(e), e + 1, e)
        e = torch.where((amax > 0) & (amax <= 448 * _pow2(e - 1)), e - 1, e)
        sc = _pow2(e).unsqueeze(1)
        vals[:, b:b + BLK] = _e4m3(blk / sc) * sc
        exps.append((e + 127).to(torch.uint8))
    return torch.stack(exps, 1), vals


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = case["op"], case["dtype"]
    if op in ("route", "route_grad"):
        t, k, g, h = case["tokens"], case["topk"], case["groups"], case["cols"]
        slots = [(e, i) for i, e in enumerate(s["ids"].reshape(-1).tolist()) if 0 <= e < g]
        slots.sort()
        src = torch.tensor([i for _, i in slots], dtype=torch.long, device="cuda")
        w = s["weights"].double().reshape(-1)
        if op == "route":
            count = [0] * (g + 1)
            for e, _ in slots:
                count[e + 1] += 1
            for e in range(g):
                count[e + 1] += count[e]
            order = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
            order[:len(src)] = src.to(torch.int32)
            pos = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
            pos[src] = torch.arange(len(src), dtype=torch.int32, device="cuda")
            Xs = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
            Y = torch.zeros(t, h, dtype=torch.float64, device="cuda")
            if len(src):
                Xs[:len(src)] = s["X"].double()[src // k]
                Y.index_add_(0, src // k, s["Ys"][:len(src)].double() * w[src].unsqueeze(1))
            return [torch.tensor(count, dtype=torch.int32, device="cuda"), order, pos.view(t, k),
                    Xs, Y]
        dYs = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        dX = torch.zeros(t, h, dtype=torch.float64, device="cuda")
        if len(src):
            dy = s["dY"].double()[src // k]
            dw[src] = (dy * s["Ys"][:len(src)].double()).sum(1)
            dYs[:len(src)] = dy * w[src].unsqueeze(1)
            dX.index_add_(0, src // k, s["dXs"][:len(src)].double())
        return [dYs, dw.view(t, k), dX]
    if op in ("rows", "weights"):
        lens = [b - a for a, b in zip(s["bounds"], s["bounds"][1:])]
        A = torch.split(s["A"], lens)
        if op == "rows":
            W = s["B"].transpose(1, 2) if case["b_layout"] == "col" else s["B"]
            return torch.cat([torch.mm(a.double(), W[g].double()) for g, a in enumerate(A)
                              if len(a)])
        B = s["B"].double()
        if case["eight"]:
            big = torch.finfo(DT[dt]).max
            B = _values(s["B"], s["scales"], case["n"]).clamp(-big, big).to(DT[dt]).double()
        D = [torch.mm(a.double().t(), b) for a, b in zip(A, torch.split(B, lens))]
        if case["accumulate"]:
            D = [d + s["D0"][g].double() for g, d in enumerate(D)]
        return torch.stack(D)
    c = case["cols"]
    if op == "swiglu":
        x = s["GU"].double()
        e, v = _checkpoint64(x)
        big = torch.finfo(DT[dt]).max
        return [x[:, :c] * torch.sigmoid(x[:, :c]) * x[:, c:], e, v.clamp(-big, big)]
    x, dh = _values(s["q"], s["scales"], 2 * c), s["dH"].double()
    g, u = x[:, :c], x[:, c:]
    sg = torch.sigmoid(g)
    return [torch.cat([dh * u * (sg + g * sg * (1 - sg)), dh * g * sg], 1), g * sg * u]
