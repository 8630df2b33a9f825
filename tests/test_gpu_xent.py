"""The linear cross entropy (gemm_xent_forward, gemm_xent_backward) against
64-bit references with bounds that count roundings: types, tiles, odd sizes,
strides, tokens without a target, pieces of the vocabulary, and differences of
the loss."""
import pytest
import torch

from gpu_util import say
from moe_ref import DT
from sparse_tiled_gemm_amd import gemm as G
from vocab_ref import Xent, far

pytestmark = pytest.mark.gpu


def make(tokens, vocab, hidden, dtype, ignore=0.2, seed=0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    W = (torch.randn(vocab, hidden, generator=gen) * hidden ** -0.5).to(DT[dtype])
    y = torch.randint(0, vocab, (tokens,), generator=gen)
    x = torch.randn(tokens, hidden, generator=gen) * spread
    X = (x + 6 * torch.rand(tokens, 1, generator=gen) * W[y].float()).to(DT[dtype])
    y[torch.rand(tokens, generator=gen) < ignore] = -100
    y[torch.rand(tokens, generator=gen) < ignore / 8] = vocab
    return X, W, y


def padded(x, ld, off=0):
    """x on the device with rows ld apart, `off` elements into its buffer."""
    buf = torch.full((len(x) * ld + off + 8,), float("nan"), dtype=x.dtype, device="cuda")
    v = buf[off:].as_strided((len(x), x.shape[1]), (ld, 1), off)
    v.copy_(x)
    return v


def outputs(tokens, cols, dtype, ld):
    buf = torch.full((tokens * ld + 8,), 7.0, dtype=DT[dtype], device="cuda")
    return buf.as_strided((tokens, cols), (ld, 1)), buf


def run(tokens, vocab, hidden, dtype, dx="f32", dw="f32", scale=1.0, ignore=0.2, id_bytes=8, pad=0,
        off=0, piece=0, accumulate=False, dlse=True, data=None, gscale=1.0, spread=1.0,
        unaligned=False):
    say("xent", tokens, vocab, hidden, dtype, dx, dw, scale, ignore, pad, off, piece, accumulate)
    X, W, y = data or make(tokens, vocab, hidden, dtype, ignore, spread=spread)
    gen = torch.Generator().manual_seed(9)
    Xd, Wd = padded(X, hidden + pad, off), padded(W, hidden + pad, off)
    yd = y.cuda() if id_bytes == 8 else y.to(torch.int32).cuda()
    plan = G.gemm_xent_plan(G.make_xent_desc(
        tokens, vocab, hidden, dtype, dx, dw, scale=scale, accumulate=accumulate, id_bytes=id_bytes,
        unaligned=unaligned or off % 8 != 0, ldx=hidden + pad, ldw=hidden + pad, lddx=hidden + pad,
        lddw=hidden + 2 * pad, piece=piece))
    nf, nb = G.gemm_xent_workspace(plan)
    ws = [torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda") for n in (nf, nb)]
    loss, lse = (torch.full((tokens + 1,), 7.0, device="cuda") for _ in range(2))
    G.gemm_xent_forward(plan, Xd, Wd, yd, loss, lse, ws[0])
    torch.cuda.synchronize()
    ref = Xent(X, W, y, scale)
    rl, re, bl, be = ref.forward()
    assert far(loss[:-1], rl, bl, "f32") <= 0 and far(lse[:-1], re, be, "f32") <= 0
    assert loss[-1] == 7.0 and lse[-1] == 7.0
    # the gradient from the kernel's own lse
    dloss = (torch.rand(tokens, generator=gen) + 0.5) * gscale
    dl = (torch.rand(tokens, generator=gen) - 0.3) * gscale if dlse else None
    dloss[~ref.ok] = float("nan")  # enters nothing
    dX, bufX = outputs(tokens, hidden, dx, hidden + pad)
    dW, bufW = outputs(vocab, hidden, dw, hidden + 2 * pad)
    before = torch.randn(vocab, hidden, generator=gen).to(DT[dw])
    if accumulate:
        dW.copy_(before)
    keep = bufX.clone(), bufW.clone()
    args = (plan, Xd, Wd, yd, lse, dloss.cuda(), dl.cuda() if dlse else None)
    G.gemm_xent_backward(*args, dX, dW, ws[1])
    torch.cuda.synchronize()
    gX, gW, bX, bW = ref.grads(lse[:-1].cpu(), dloss, dl, dtype)
    if accumulate:
        gW = gW + before.double()
        bW = bW + 2.0 ** -24 * (gW.abs() + bW)
    assert far(dX, gX, bX, dx) <= 0, "dX"
    assert far(dW, gW, bW, dw) <= 0, "dW"
    assert not bool(dX[~ref.ok.cuda()].any())
    for w in ws:
        assert bool((w[-64:] == 0xFF).all())
    # nothing between or behind the rows; the same bits again, alone too
    first = dX.clone(), dW.clone()
    for buf, k, out, ld in ((bufX, keep[0], dX, hidden + pad), (bufW, keep[1], dW, hidden + 2 * pad)):
        k.as_strided(out.shape, (ld, 1)).copy_(out)
        assert torch.equal(k, buf)
    if accumulate:
        dW.copy_(before)
    dX.fill_(3.0)
    G.gemm_xent_backward(*args, dX, None, ws[1])
    G.gemm_xent_backward(*args, None, dW, ws[1])
    assert torch.equal(dX, first[0]) and torch.equal(dW, first[1])
    loss2, lse2 = loss.clone(), lse.clone()
    G.gemm_xent_forward(plan, Xd, Wd, yd, None, lse2, ws[0])
    assert torch.equal(lse, lse2) and torch.equal(loss, loss2)
    return ref, (X, W, y, dloss, dl, dX, dW)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,vocab,hidden", [
    (1, 1, 8), (1, 1000, 64), (1, 5000, 128), (5, 63, 72), (64, 513, 64), (65, 300, 136), (130, 1111, 264),
    (257, 777, 200), (300, 2048, 64), (513, 1025, 128), (2, 70001, 40), (16, 40000, 200),
    (17, 3000, 136)])
def test_sizes(dtype, tokens, vocab, hidden):
    run(tokens, vocab, hidden, dtype)


@pytest.mark.parametrize("tile", ["tiled64", "tiled128", "tiled256"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,vocab,hidden,piece", [
    (3, 400, 64, 0), (200, 900, 72, 256), (300, 1300, 520, 512), (520, 600, 328, 0)])
def test_every_tile(monkeypatch, tile, dtype, tokens, vocab, hidden, piece):
    monkeypatch.setenv("STGEMM_FORCE_KERNEL", tile)
    run(tokens, vocab, hidden, dtype, dx=dtype, dw=dtype, piece=piece)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,vocab,hidden,pad,off,piece", [
    (33, 501, 1, 0, 0, 0), (150, 700, 77, 0, 0, 256), (70, 300, 63, 2, 1, 0), (40, 300, 64, 0, 3, 256),
    (300, 600, 129, 7, 5, 256), (90, 400, 64, 8, 8, 0), (90, 400, 64, 3, 0, 0), (9, 1000, 130, 0, 0, 256),
    (16, 900, 264, 8, 8, 512)])
def test_odd_widths_and_strides(dtype, tokens, vocab, hidden, pad, off, piece):
    run(tokens, vocab, hidden, dtype, dx=dtype, dw="f32", pad=pad, off=off, piece=piece, id_bytes=4)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,vocab,hidden,pad,off", [
    (1, 1, 7, 0, 1), (1, 17, 8, 0, 1), (16, 5003, 9, 0, 0), (2, 40001, 15, 0, 3), (5, 700, 127, 1, 0),
    (7, 700, 128, 0, 1), (16, 3000, 129, 5, 7), (13, 20011, 1031, 0, 0), (3, 5003, 1096, 4, 0)])
def test_few_rows_of_any_alignment(dtype, tokens, vocab, hidden, pad, off):
    """W read where it lies, NaN between its rows."""
    run(tokens, vocab, hidden, dtype, pad=pad, off=off)


@pytest.mark.parametrize("tokens,vocab,hidden,pad,dtype,dw,accumulate", [
    (40, 33001, 1024, 0, "bf16", "bf16", False), (64, 20011, 1032, 8, "f16", "f16", True),
    (100, 33001, 1024, 0, "f16", "f32", False), (128, 20011, 1032, 8, "bf16", "f32", True),
    (3, 33001, 1048, 0, "bf16", "f16", True), (65, 20011, 1024, 0, "f16", "bf16", True)])
def test_few_rows_many_columns(tokens, vocab, hidden, pad, dtype, dw, accumulate):
    """Up to 128 rows dW's rows are written in turn, several steps a wave."""
    run(tokens, vocab, hidden, dtype, dx="f32", dw=dw, pad=pad, accumulate=accumulate)


@pytest.mark.parametrize("dx", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dw", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_types(dx, dw, accumulate):
    run(70, 600, 96, "bf16", dx=dx, dw=dw, accumulate=accumulate, piece=256)


@pytest.mark.parametrize("scale,spread", [(0.25, 1.0), (-1.0, 1.0), (8.0, 4.0), (0.0, 1.0)])
def test_scales(scale, spread):
    """Logits from all equal to some hundred apart."""
    run(100, 700, 128, "bf16", scale=scale, spread=spread)
    run(100, 700, 128, "f16", scale=scale, spread=spread)


@pytest.mark.parametrize("gscale", [1e-30, 1e-7, 1e7])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_of_any_size(dtype, gscale):
    """Gradients far outside fp16's range keep their bits in fp32 outputs."""
    run(80, 500, 64, dtype, gscale=gscale)


@pytest.mark.parametrize("ignore", [0.0, 0.9, 1.1])
@pytest.mark.parametrize("tokens", [1, 50, 400])
def test_tokens_without_target(tokens, ignore):
    run(tokens, 300, 64, "bf16", ignore=ignore)


@pytest.mark.parametrize("piece", [1, 256, 300, 512, 1024, 1 << 20])
def test_pieces(piece):
    run(140, 1500, 80, "f16", dx="f16", dw="f16", piece=piece)


@pytest.mark.parametrize("tokens", [3, 40, 100])
def test_copied_weights_beside_rows_that_are_read_where_they_lie(tokens):
    run(tokens, 700, 64, "bf16", unaligned=True, piece=256)


@pytest.mark.parametrize("tokens", [4, 100])
def test_an_infinite_coefficient_stays_in_its_row(tokens):
    """One token's dloss overflowed: its row of dX and dW say so, the other rows
    of dX keep their values."""
    vocab, hidden = 300, 64
    X, W, y = make(tokens, vocab, hidden, "f16", ignore=0.0)
    plan = G.gemm_xent_plan(G.make_xent_desc(tokens, vocab, hidden, "f16", "f32", "f32", id_bytes=8))
    ws = torch.empty(max(G.gemm_xent_workspace(plan)), dtype=torch.uint8, device="cuda")
    ref = Xent(X, W, y, 1.0)
    lse = ref.lse_rows.float()
    for bad in (float("inf"), float("nan")):
        g = torch.full((tokens,), 0.25)
        g[2] = bad
        dX, dW = torch.empty(tokens, hidden, device="cuda"), torch.empty(vocab, hidden, device="cuda")
        G.gemm_xent_backward(plan, X.cuda(), W.cuda(), y.cuda(), lse.cuda(), g.cuda(), None, dX, dW, ws)
        good = torch.arange(tokens) != 2
        g[2] = 0.25
        gX, _, bX, _ = ref.grads(lse, g, None, "f16")
        assert far(dX[good.cuda()], gX[good], bX[good], "f32") <= 0
        assert not bool(torch.isfinite(dX[2]).any()) and not bool(torch.isfinite(dW[y[2]]).any())


def test_no_dlse():
    run(60, 400, 64, "bf16", dlse=False)


def test_rows_of_masked_tokens_enter_nothing():
    X, W, y = make(100, 300, 64, "bf16", ignore=0.4)
    X[(y < 0) | (y >= 300)] = float("nan")
    run(100, 300, 64, "bf16", data=(X, W, y))


def test_no_tokens():
    plan = G.gemm_xent_plan(G.make_xent_desc(0, 300, 64, "bf16", dw_dtype="f32"))
    nf, nb = G.gemm_xent_workspace(plan)
    W = torch.zeros(300, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(nf, nb), dtype=torch.uint8, device="cuda")
    dW = torch.full((300, 64), 7.0, device="cuda")
    G.gemm_xent_forward(plan, None, W, None, None, None, ws)
    G.gemm_xent_backward(plan, None, W, None, None, None, None, None, dW, ws)
    assert not bool(dW.any())


def test_infinities_and_nan_stay_in_their_rows():
    """A row whose logits overflow gets what the formula gives; the others keep
    their values."""
    tokens, vocab, hidden = 70, 500, 64
    X, W, y = make(tokens, vocab, hidden, "bf16", ignore=0.0)
    bad = [3, 40]
    X[3, 0] = float("inf")
    X[40, 1] = float("nan")
    plan = G.gemm_xent_plan(G.make_xent_desc(tokens, vocab, hidden, "bf16", id_bytes=8))
    ws = torch.empty(max(G.gemm_xent_workspace(plan)), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    G.gemm_xent_forward(plan, X.cuda(), W.cuda(), y.cuda(), loss, lse, ws)
    assert not bool(torch.isfinite(lse[bad]).any()) and not bool(torch.isfinite(loss[bad]).any())
    good = torch.ones(tokens, dtype=torch.bool)
    good[bad] = False
    rl, re, bl, be = Xent(X[good], W, y[good], 1.0).forward()
    assert far(loss[good.cuda()], rl, bl, "f32") <= 0 and far(lse[good.cuda()], re, be, "f32") <= 0
    # a bad row's gradient with a zero weight of the loss is NaN, not hidden
    dX = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    G.gemm_xent_backward(plan, X.cuda(), W.cuda(), y.cuda(), lse, torch.ones(tokens, device="cuda"),
                         None, dX, None, ws)
    assert bool(torch.isfinite(dX[good.cuda()]).all()) and not bool(torch.isfinite(dX[bad]).any())


def test_against_differences():
    """Sums of dX d and dW e against differences of the 64-bit loss along d and
    e: within the gradients' own bounds and the difference's h^2 term, taken
    from two step widths."""
    tokens, vocab, hidden = 60, 400, 64
    ref, (X, W, y, dloss, dl, dX, dW) = run(tokens, vocab, hidden, "bf16")
    gen = torch.Generator().manual_seed(3)
    lse = ref.lse_rows.float()
    full = torch.zeros(tokens)
    full[ref.rows] = lse
    _, _, bX, bW = ref.grads(full, dloss, dl, "bf16")

    def value(x, w):
        z = x[ref.rows] @ w.t()
        l = torch.logsumexp(z, 1)
        zy = z.gather(1, ref.y.unsqueeze(1)).squeeze(1)
        return float((dloss[ref.rows].double() * (l - zy) + dl[ref.rows].double() * l).sum())

    for which, grad, bound in (("X", dX, bX), ("W", dW, bW)):
        d = torch.randn((tokens if which == "X" else vocab), hidden, generator=gen).double()
        at = lambda h: value(X.double() + h * d, W.double()) if which == "X" else \
            value(X.double(), W.double() + h * d)
        diff = lambda h: (at(h) - at(-h)) / (2 * h)
        d1, d2 = diff(1e-3), diff(2e-3)
        got = float((grad.double().cpu() * d).sum())
        assert abs(got - d1) <= float((bound * d.abs()).sum()) + abs(d2 - d1)


def test_replayed_and_shared_workspace():
    """Captured, replayed with new inputs between eager work; two plans' graphs
    on one workspace, one after the other."""
    shapes = [(70, 900, 64, "bf16"), (300, 700, 72, "f16")]
    work, graphs = [], []
    need = 0
    for t, v, h, dt in shapes:
        plan = G.gemm_xent_plan(G.make_xent_desc(t, v, h, dt, dw_dtype="f32", id_bytes=8, piece=512))
        need = max(need, *G.gemm_xent_workspace(plan))
        e = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device="cuda")
        work.append(dict(plan=plan, X=e(t, h, d=DT[dt]), W=e(v, h, d=DT[dt]), y=e(t, d=torch.int64),
                         loss=e(t), lse=e(t), g=e(t) + 0.5, dX=e(t, h, d=DT[dt]), dW=e(v, h)))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(w):
        G.gemm_xent_forward(w["plan"], w["X"], w["W"], w["y"], w["loss"], w["lse"], ws)
        G.gemm_xent_backward(w["plan"], w["X"], w["W"], w["y"], w["lse"], w["g"], None, w["dX"],
                             w["dW"], ws)

    for w in work:
        step(w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(w)
        graphs.append(g)
    names = ("loss", "lse", "dX", "dW")
    for seed in range(3):
        want = []
        for w, (t, v, h, dt) in zip(work, shapes):
            X, W, y = make(t, v, h, dt, seed=seed)
            w["X"].copy_(X), w["W"].copy_(W), w["y"].copy_(y)
            step(w)
            torch.cuda.synchronize()
            want.append([w[k].clone() for k in names])
            for k in names:
                w[k].zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for w, x in zip(work, want):
            assert all(torch.equal(w[k], y) for k, y in zip(names, x)), seed


def test_on_another_stream():
    X, W, y = make(80, 600, 64, "bf16")
    plan = G.gemm_xent_plan(G.make_xent_desc(80, 600, 64, "bf16", id_bytes=8))
    ws = [torch.empty(max(G.gemm_xent_workspace(plan)), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    Xd, Wd, yd = X.cuda(), W.cuda(), y.cuda()
    out = [(torch.zeros(80, device="cuda"), torch.zeros(80, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, w, (loss, lse) in zip(streams, ws, out):  # one plan, two calls at once
        with torch.cuda.stream(s):
            G.gemm_xent_forward(plan, Xd, Wd, yd, loss, lse, w)
    torch.cuda.synchronize()
    ref = Xent(X, W, y, 1.0).forward()
    for loss, lse in out:
        assert far(loss, ref[0], ref[2], "f32") <= 0 and far(lse, ref[1], ref[3], "f32") <= 0


def test_offsets_past_32_bits():
    """dW and W of more than 2^32 bytes: the probability is all on the last
    column."""
    vocab, hidden, tokens = 300000, 8192, 40
    W = torch.zeros(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    W[-1, :64], W[-2, :64] = 1.0, 0.5
    X = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    X[:, :64] = 1.0
    y = torch.full((tokens,), vocab - 2, device="cuda")
    plan = G.gemm_xent_plan(G.make_xent_desc(tokens, vocab, hidden, "bf16", id_bytes=8))
    ws = torch.empty(max(G.gemm_xent_workspace(plan)), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    G.gemm_xent_forward(plan, X, W, y, loss, lse, ws)
    # z = 64, 32 and zeros: lse = 64 and loss = 32, to e^-32 and V e^-64
    assert bool((lse == 64).all()) and bool((loss == 32).all())
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    G.gemm_xent_backward(plan, X, W, y, lse, torch.ones(tokens, device="cuda"), None, dX, dW, ws)
    # G = 1 at the last column, -1 at the target's, at most e^-32 elsewhere
    assert bool((dW[-1, :64] == tokens).all()) and bool((dW[-2, :64] == -tokens).all())
    assert bool((dX[:, :64] == 0.5).all())
    assert float(dW[:-2].float().abs().max()) < 1e-20 and not bool(dW[:, 64:].any())
