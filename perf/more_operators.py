"""Measured cases of the operators over a vocabulary: the rows of an embedding
table looked up by token, their gradient summed by token, and the softmax
cross entropy of a linear layer over the vocabulary, with its gradients.

`run` computes a pass either in plain torch operations (own = False) or
through the library's entry points (own = True).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EB = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoder's next token: one row of the table
        dict(name="embed_one", op="embed", tokens=1, vocab=32768, cols=4096, e_dtype="bf16",
             y_dtype="bf16", scaled=False, drop=0.0),
        # a training step's tokens, rows scaled by the root of the width
        dict(name="embed_batch", op="embed", tokens=16384, vocab=131072, cols=4096, e_dtype="bf16",
             y_dtype="bf16", scaled=True, drop=0.0),
        # odd sizes, padding among the tokens, an fp32 table
        dict(name="embed_odd", op="embed", tokens=2001, vocab=50021, cols=1027, e_dtype="f32",
             y_dtype="f16", scaled=True, drop=0.1),
        # a small batch, added to the fp32 gradient that the output layer left in the table
        dict(name="embed_grad_add", op="embed_grad", tokens=512, vocab=32768, cols=2048, dtype="bf16",
             d_dtype="f32", accumulate=True, hot=0.0, drop=0.0, scaled=False),
        # a training step's tokens, the whole gradient written
        dict(name="embed_grad", op="embed_grad", tokens=16384, vocab=131072, cols=2048, dtype="bf16",
             d_dtype="f32", accumulate=False, hot=0.0, drop=0.0, scaled=True),
        # long batches in which one token (padding that counts) is a third of all; ragged sizes
        dict(name="embed_grad_hot", op="embed_grad", tokens=50000, vocab=50021, cols=776, dtype="f16",
             d_dtype="f16", accumulate=False, hot=0.3, drop=0.05, scaled=False),
        # the probability of one token
        dict(name="xent_one", op="xent", tokens=1, vocab=32768, hidden=2048, dtype="bf16",
             ignore=0.0, scale=1.0),
        # the choices of a short question scored
        dict(name="xent_few", op="xent", tokens=48, vocab=131072, hidden=4096, dtype="bf16",
             ignore=0.0, scale=1.0),
        # a training step's forward pass
        dict(name="xent_batch", op="xent", tokens=8192, vocab=131072, hidden=4096, dtype="bf16",
             ignore=0.0, scale=1.0),
        # odd sizes: a width that is no multiple of 8, some tokens without a target
        dict(name="xent_odd", op="xent", tokens=1531, vocab=50021, hidden=1027, dtype="f16",
             ignore=0.1, scale=0.5),
        # a training step's gradients
        dict(name="xent_grad", op="xent_grad", tokens=4096, vocab=131072, hidden=2048, dtype="bf16",
             ignore=0.0, scale=1.0, dlse=False),
        # answers trained behind prompts that do not count, with a penalty on the normaliser
        dict(name="xent_grad_masked", op="xent_grad", tokens=3001, vocab=50021, hidden=1416,
             dtype="f16", ignore=0.6, scale=1.0, dlse=True),
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
        op = rng.choice(["embed", "embed_grad", "embed_grad", "xent", "xent", "xent_grad",
                         "xent_grad"])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        some = lambda lo, hi: (max(8, 8 * (_log(rng, lo, hi) // 8)) if rng.random() < 0.7
                               else _log(rng, lo, hi))
        vocab = _log(rng, 1000, 200000)
        if op == "embed":
            c = dict(op=op, tokens=_log(rng, 1, 65536), vocab=vocab, cols=some(64, 8192),
                     e_dtype=rng.choice([dtype, dtype, "f32"]), y_dtype=dtype,
                     scaled=rng.random() < 0.5, drop=rng.choice([0.0, 0.0, 0.1]))
        elif op == "embed_grad":
            c = dict(op=op, tokens=_log(rng, 1, 65536), vocab=vocab, cols=some(64, 8192),
                     dtype=dtype, d_dtype=rng.choice(["f32", "f32", dtype]),
                     accumulate=rng.random() < 0.4, hot=rng.choice([0.0, 0.0, 0.1, 0.5]),
                     drop=rng.choice([0.0, 0.0, 0.1]), scaled=rng.random() < 0.5)
        else:
            c = dict(op=op, tokens=_log(rng, 1, 8192), vocab=vocab, hidden=some(64, 8192),
                     dtype=dtype, ignore=rng.choice([0.0, 0.0, 0.1, 0.7]),
                     scale=rng.choice([1.0, 1.0, 0.5]))
            if op == "xent_grad":
                c["dlse"] = rng.random() < 0.3
        w = work(c)
        if w["bytes"] <= lim[0] and w["flops"] <= lim[1]:
            return c


def _share(vocab):
    """How often each token occurs: a power of its rank, as in text."""
    p = 1.0 / (torch.arange(vocab, dtype=torch.float64) + 2.7)
    return p / p.sum()


def _distinct(case):
    """Rows of the table that a case's tokens are expected to reach."""
    t = case["tokens"] * (1 - case.get("drop", 0.0)) * (1 - case.get("hot", 0.0))
    return float((1 - (1 - _share(case["vocab"])) ** t).sum()) + (case.get("hot", 0.0) > 0)


def work(case):
    """Bytes and operations one pass cannot do without."""
    op, t, v = case["op"], case["tokens"], case["vocab"]
    if op == "embed":
        # ids, the rows that occur, the rows written
        h = case["cols"]
        return {"bytes": 8 * t + h * (_distinct(case) * EB[case["e_dtype"]] + t * EB[case["y_dtype"]]),
                "flops": t * h}
    if op == "embed_grad":
        # ids and rows read; the table written, or the rows that occur read and written
        h, b = case["cols"], EB[case["d_dtype"]]
        rows = 2 * _distinct(case) if case["accumulate"] else v
        return {"bytes": 8 * t + h * (2 * t * (1 - case["drop"]) + rows * b), "flops": 2 * t * h}
    # tokens without a target need no product
    h, n = case["hidden"], max(1, round(t * (1 - case["ignore"])))
    if op == "xent":
        return {"bytes": 2 * h * (n + v) + 16 * t, "flops": 2 * n * h * v}
    # X, W, targets and three vectors read, dX and dW written; the logits are
    # not kept by the forward pass: three products
    return {"bytes": 2 * h * (n + v) + 2 * h * (t + v) + 20 * t, "flops": 6 * n * h * v}


# ---------------------------------------------------------------- inputs

def _tokens(gen, case):
    """Token ids (int64): Zipf's shares, a hot one, ids out of range where dropped."""
    t, v = case["tokens"], case["vocab"]
    cdf = torch.cumsum(_share(v), 0).cuda()
    r = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.searchsorted(cdf, r).clamp(max=v - 1)
    if case.get("hot"):
        ids[torch.rand(t, generator=gen, device="cuda") < case["hot"]] = v // 3
    drop = case.get("drop") or case.get("ignore")
    if drop:
        ids[torch.rand(t, generator=gen, device="cuda") < drop] = -100
    return ids


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(DT[dtype])


def _has_target(ids, vocab):
    return (ids >= 0) & (ids < vocab)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    t, v = case["tokens"], case["vocab"]
    empty = lambda shape, d: torch.empty(shape, dtype=d, device="cuda")
    s["ids"] = _tokens(gen, case)
    if op == "embed":
        h = case["cols"]
        s["E"] = _normal(gen, (v, h), case["e_dtype"], 0.02)
        s["scale"] = h ** 0.5 if case["scaled"] else 1.0
        s["Y"] = empty((t, h), DT[case["y_dtype"]])
        return s
    if op == "embed_grad":
        h = case["cols"]
        s["dY"] = _normal(gen, (t, h), case["dtype"])
        s["scale"] = h ** 0.5 if case["scaled"] else 1.0
        if case["accumulate"]:
            s["dE"] = _normal(gen, (v, h), case["d_dtype"])
        else:
            s["dE"] = empty((v, h), DT[case["d_dtype"]])
        if own:
            from sparse_tiled_gemm_amd import gemm as G
            s["workspace"] = empty(max(G.gemm_embed_workspace(t, v, h), 1), torch.uint8)
        return s
    h, dt = case["hidden"], case["dtype"]
    s["W"] = _normal(gen, (v, h), dt, h ** -0.5)
    # hidden states that point towards their targets, some more than others
    x = torch.randn((t, h), generator=gen, device="cuda")
    b = torch.rand((t, 1), generator=gen, device="cuda") * 10
    s["X"] = (x + b * s["W"][s["ids"].clamp(0, v - 1)].float()).to(DT[dt])
    if op == "xent":
        s["loss"], s["lse"] = empty(t, torch.float32), empty(t, torch.float32)
    else:
        lse = torch.full((t,), -math.inf, device="cuda")
        for v0 in range(0, v, 16384):
            z = (s["X"].float() @ s["W"][v0:v0 + 16384].float().t()) * case["scale"]
            lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        ok = _has_target(s["ids"], v)
        s["lse"] = torch.where(ok, lse, torch.zeros_like(lse))
        # the mean over the targets; 16-bit floats are trained with a larger loss
        g = (65536.0 if dt == "f16" else 1.0) / max(1, int(ok.sum()))
        s["dloss"] = torch.where(ok, torch.full_like(lse, g), torch.zeros_like(lse))
        s["dlse"] = 2e-3 * s["lse"] * s["dloss"] if case["dlse"] else None
        s["dX"], s["dW"] = empty((t, h), DT[dt]), empty((v, h), DT[dt])
    if own:
        from sparse_tiled_gemm_amd import gemm as G
        s["plan"] = G.gemm_xent_plan(G.make_xent_desc(t, v, h, dt, dt, dt, scale=case["scale"],
                                                      id_bytes=8))
        forward, backward = G.gemm_xent_workspace(s["plan"])
        s["workspace"] = empty(max(forward if op == "xent" else backward, 1), torch.uint8)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _plain_embed(s):
    ids = s["ids"]
    ok = _has_target(ids, s["case"]["vocab"])
    y = s["E"][torch.where(ok, ids, torch.zeros_like(ids))].float() * s["scale"]
    return torch.where(ok.unsqueeze(1), y, torch.zeros_like(y)).to(DT[s["case"]["y_dtype"]])


def _plain_embed_grad(s):
    c, ids = s["case"], s["ids"]
    ok = _has_target(ids, c["vocab"])
    dy = torch.where(ok.unsqueeze(1), s["dY"].float() * s["scale"], torch.zeros((), device="cuda"))
    at = torch.where(ok, ids, torch.zeros_like(ids))
    if c["accumulate"]:
        # the gradient so far, in place
        s["dE"].copy_(s["dE"].float().index_add_(0, at, dy))
        return s["dE"]
    g = torch.zeros((c["vocab"], c["cols"]), dtype=torch.float32, device="cuda")
    return g.index_add_(0, at, dy).to(DT[c["d_dtype"]])


def _plain_xent(s):
    c, ids = s["case"], s["ids"]
    ok = _has_target(ids, c["vocab"])
    at = torch.where(ok, ids, torch.zeros_like(ids)).unsqueeze(1)
    z = (s["X"].float() @ s["W"].float().t()) * c["scale"]
    m = z.max(1, keepdim=True).values
    lse = (m + torch.log(torch.exp(z - m).sum(1, keepdim=True))).squeeze(1)
    loss = lse - z.gather(1, at).squeeze(1)
    zero = torch.zeros_like(lse)
    return [torch.where(ok, loss, zero), torch.where(ok, lse, zero)]


def _plain_xent_grad(s):
    c, ids = s["case"], s["ids"]
    ok = _has_target(ids, c["vocab"])
    x, w = s["X"].float(), s["W"].float()
    zero = torch.zeros_like(s["lse"])
    g = torch.where(ok, s["dloss"], zero)
    gl = g if s["dlse"] is None else g + torch.where(ok, s["dlse"], zero)
    # d loss / d z = p - [v is the target], d lse / d z = p
    dz = torch.exp((x @ w.t()) * c["scale"] - s["lse"].unsqueeze(1)) * gl.unsqueeze(1)
    dz = torch.where(ok.unsqueeze(1), dz, torch.zeros((), device="cuda"))
    at = torch.where(ok, ids, torch.zeros_like(ids)).unsqueeze(1)
    dz.scatter_add_(1, at, -g.unsqueeze(1))
    dz = dz * c["scale"]
    return [(dz @ w).to(DT[c["dtype"]]), (dz.t() @ x).to(DT[c["dtype"]])]


_plain = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "xent": _plain_xent,
          "xent_grad": _plain_xent_grad}


def _own_embed(s):
    from sparse_tiled_gemm_amd import gemm as G
    c = s["case"]
    G.gemm_embed(c["tokens"], c["vocab"], c["cols"], c["e_dtype"], c["y_dtype"], s["ids"], s["E"], 0,
                 s["Y"], 0, scale=s["scale"], id_bytes=8)
    return s["Y"]


def _own_embed_grad(s):
    from sparse_tiled_gemm_amd import gemm as G
    c = s["case"]
    G.gemm_embed_backward(c["tokens"], c["vocab"], c["cols"], c["dtype"], c["d_dtype"], s["ids"],
                          s["dY"], 0, s["dE"], 0, s["workspace"], scale=s["scale"],
                          accumulate=c["accumulate"], id_bytes=8)
    return s["dE"]


def _own_xent(s):
    from sparse_tiled_gemm_amd import gemm as G
    G.gemm_xent_forward(s["plan"], s["X"], s["W"], s["ids"], s["loss"], s["lse"], s["workspace"])
    return [s["loss"], s["lse"]]


def _own_xent_grad(s):
    from sparse_tiled_gemm_amd import gemm as G
    G.gemm_xent_backward(s["plan"], s["X"], s["W"], s["ids"], s["lse"], s["dloss"], s["dlse"],
                         s["dX"], s["dW"], s["workspace"])
    return [s["dX"], s["dW"]]


_own = {"embed": _own_embed, "embed_grad": _own_embed_grad, "xent": _own_xent,
        "xent_grad": _own_xent_grad}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, v = case["op"], case["vocab"]
    rows = [i for i, e in enumerate(s["ids"].tolist()) if 0 <= e < v]
    rows = torch.tensor(rows, dtype=torch.long, device="cuda")
    ids = s["ids"][rows]
    if op == "embed":
        Y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        Y[rows] = s["E"][ids].double() * s["scale"]
        return Y
    if op == "embed_grad":
        if case["accumulate"]:
            dE = s["dE"].double()
        else:
            dE = torch.zeros(v, case["cols"], dtype=torch.float64, device="cuda")
        dE.index_put_((ids,), s["dY"][rows].double() * s["scale"], accumulate=True)
        return dE
    t, h, k = case["tokens"], case["hidden"], case["scale"]
    X = s["X"][rows].double()
    step = 8192
    if op == "xent":
        best = torch.full((len(rows),), -math.inf, dtype=torch.float64, device="cuda")
        total, picked = torch.zeros_like(best), torch.zeros_like(best)
        for v0 in range(0, v, step):
            z = torch.mm(X, s["W"][v0:v0 + step].double().t().contiguous()).mul_(k)
            new = torch.maximum(best, z.amax(1))
            total = total * torch.exp(best - new) + torch.exp(z - new.unsqueeze(1)).sum(1)
            best = new
            here = torch.nonzero((ids >= v0) & (ids < v0 + step)).squeeze(1)
            picked[here] = z[here, ids[here] - v0]
        loss = torch.zeros(t, dtype=torch.float64, device="cuda")
        lse = torch.zeros_like(loss)
        lse[rows] = best + torch.log(total)
        loss[rows] = lse[rows] - picked
        return [loss, lse]
    g = s["dloss"][rows].double()
    gl = g if s["dlse"] is None else g + s["dlse"][rows].double()
    lse = s["lse"][rows].double()
    dX = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    dW = torch.empty(v, h, dtype=torch.float64, device="cuda")
    acc = torch.zeros(len(rows), h, dtype=torch.float64, device="cuda")
    for v0 in range(0, v, step):
        W = s["W"][v0:v0 + step].double()
        dz = torch.exp(torch.mm(X, W.t().contiguous()) * k - lse.unsqueeze(1)) * gl.unsqueeze(1)
        here = torch.nonzero((ids >= v0) & (ids < v0 + step)).squeeze(1)
        dz[here, ids[here] - v0] -= g[here]
        acc += torch.mm(dz, W) * k
        dW[v0:v0 + step] = torch.mm(dz.t().contiguous(), X) * k
    dX[rows] = acc
    return [dX, dW]
