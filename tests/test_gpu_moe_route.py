"""Routing for a mixture-of-experts MLP on the GPU: sort, dispatch, combine
and its gradient against plain 64-bit references (tests/moe_ref.py)."""
import numpy as np
import pytest
import torch

import moe_ref as R
from gpu_util import say
from sparse_tiled_gemm_amd import gemm as G

pytestmark = pytest.mark.gpu


def _ids(tokens, topk, groups, seed, drop=0.0, id_bytes=8):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(max(groups, topk))[:topk] for _ in range(tokens)]) \
        if tokens else np.zeros((0, topk), np.int64)
    ids = ids.astype(np.int64)
    out = g.random(ids.shape) < drop
    ids[out] = g.choice([-1, groups, 2 ** 31 - 1, -2 ** 31] +
                        ([2 ** 40, -2 ** 40] if id_bytes == 8 else []), size=int(out.sum()))
    return ids if id_bytes == 8 else ids.astype(np.int32)


def _sort(ids, groups):
    t, k = ids.shape
    dev = torch.from_numpy(ids.copy()).cuda()
    out = [torch.full((n,), 77, dtype=torch.int32, device="cuda")
           for n in (groups + 1, max(t * k, 1), max(t * k, 1))]
    ws = torch.full((max(G.gemm_moe_sort_workspace(t, k, groups), 1),), 0x5A, dtype=torch.uint8,
                    device="cuda")
    G.gemm_moe_sort(t, k, groups, dev, *out, ws, id_bytes=ids.itemsize)
    torch.cuda.synchronize()
    return [out[0].cpu().numpy()] + [o.cpu().numpy()[:t * k] for o in out[1:]]


@pytest.mark.parametrize("tokens,topk,groups,drop,id_bytes", [
    (1, 1, 1, 0.0, 4), (1, 8, 64, 0.0, 8), (0, 2, 5, 0.0, 8), (63, 1, 3, 0.2, 4),
    (64, 4, 7, 0.0, 8), (257, 3, 13, 0.1, 4), (512, 2, 1024, 0.0, 8),    # one launch
    (513, 2, 1000, 0.3, 8), (1025, 1, 1, 0.5, 4), (4096, 1, 31, 0.1, 8),
    (4097, 1, 31, 0.1, 8), (4096, 8, 256, 0.05, 8), (5000, 2, 1024, 0.0, 4),  # chunked
    (1999, 3, 13, 1.0, 8), (40000, 8, 65, 0.01, 4),
])
def test_sort(tokens, topk, groups, drop, id_bytes):
    say("sort", tokens, topk, groups, drop, id_bytes)
    ids = _ids(tokens, topk, groups, tokens + groups, drop, id_bytes)
    for got, want in zip(_sort(ids, groups), R.sort_ref(ids, groups)):
        np.testing.assert_array_equal(got, want)


def test_sort_many_chunks():
    """More slots than 256 chunks of 1024: longer chunks."""
    ids = _ids(300001, 1, 37, 5, 0.1, 4)
    for got, want in zip(_sort(ids, 37), R.sort_ref(ids, 37)):
        np.testing.assert_array_equal(got, want)


def _rows(gen, n, cols, dtype, ld=0, off=0):
    """n x cols values in a buffer of leading dimension ld whose first element
    is `off` elements past an aligned address; (view, buffer)."""
    ld = ld or cols
    buf = torch.full((n * ld + 64,), 7.5, dtype=R.DT[dtype], device="cuda")
    v = buf[off:off + n * ld].view(n, ld)[:, :cols]
    v.copy_(torch.randn(n, cols, generator=gen).to(R.DT[dtype]))
    return v, buf


CASES = [  # tokens, topk, groups, cols, dtype, drop, ld extra, element offset
    (1, 8, 64, 4096, "bf16", 0.0, 0, 0), (1, 1, 1, 1, "f16", 0.0, 0, 1),
    (3, 2, 4, 7, "bf16", 0.0, 2, 1), (100, 2, 8, 128, "f16", 0.2, 8, 8),
    (129, 3, 5, 1027, "f16", 0.1, 0, 0), (700, 5, 9, 515, "bf16", 0.3, 3, 1),
    (2100, 1, 16, 72, "bf16", 0.0, 0, 0), (2049, 6, 30, 24, "f16", 0.5, 0, 3),
    (2800, 3, 20, 520, "f16", 0.1, 0, 0), (4200, 2, 11, 40, "bf16", 0.0, 0, 0),
    (500, 6, 21, 157, "f16", 0.05, 0, 0), (33, 2, 3, 256, "bf16", 0.0, 1, 1),
    (300, 9, 12, 2056, "bf16", 0.1, 0, 0), (50, 4, 6, 64, "f16", 1.0, 0, 0),
]


@pytest.mark.parametrize("case", CASES)
def test_dispatch_combine_and_gradient(case):
    tokens, topk, groups, cols, dtype, drop, ldx, off = case
    say(case)
    gen = torch.Generator().manual_seed(tokens * 7 + cols)
    ids = _ids(tokens, topk, groups, cols, drop)
    n, ld = tokens * topk, cols + ldx
    X, _ = _rows(gen, tokens, cols, dtype, ld, off)
    Xs, xs_buf = _rows(gen, n, cols, dtype, ld, off)
    before = xs_buf.clone()
    i32 = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")
    offsets, order, pos = i32(groups + 1), i32(n), i32(tokens, topk)
    ws = torch.empty(max(G.gemm_moe_sort_workspace(tokens, topk, groups), 1), dtype=torch.uint8,
                     device="cuda")
    G.gemm_moe_dispatch(tokens, topk, groups, cols, dtype, torch.from_numpy(ids).cuda(), X, ld,
                        offsets, order, pos, Xs, ld, ws, id_bytes=8)
    torch.cuda.synchronize()
    ro, rr, rp = R.sort_ref(ids, groups)
    np.testing.assert_array_equal(offsets.cpu().numpy(), ro)
    np.testing.assert_array_equal(order.cpu().numpy(), rr)
    np.testing.assert_array_equal(pos.cpu().numpy().reshape(-1), rp)
    # rows bit by bit; nothing outside them is touched
    have = int(ro[-1])
    want = before.clone()
    w2 = want[off:off + n * ld].view(n, ld)
    w2[:have, :cols] = X[torch.from_numpy(rr[:have] // topk).long().cuda()]
    assert torch.equal(xs_buf.view(torch.int16), want.view(torch.int16))

    # combine, with and without weights; the weight of a dropped slot is no number
    w = torch.rand(tokens, topk, generator=gen) - 0.3
    wd = w.clone()
    wd[torch.from_numpy(rp.reshape(tokens, topk)) < 0] = float("nan")
    Ys, _ = _rows(gen, n, cols, dtype, ld, off)
    p2 = torch.from_numpy(rp.reshape(tokens, topk))
    for weights, wr in [(wd.cuda(), w), (None, None)]:
        Y, y_buf = _rows(gen, tokens, cols, dtype, ld, off)
        yb = y_buf.clone()
        G.gemm_moe_combine(tokens, topk, cols, dtype, pos, weights, Ys, ld, n, Y, ld)
        torch.cuda.synchronize()
        ref, S = R.combine_ref(p2, wr, Ys.cpu())
        err = (Y.cpu().double() - ref).abs()
        assert (err <= R.half_step(dtype, ref) * 1.001 + (topk + 1) * R.U32 * S).all()
        yb[off:off + tokens * ld].view(tokens, ld)[:, :cols] = Y
        assert torch.equal(y_buf.view(torch.int16), yb.view(torch.int16))

    # gradient
    dY, _ = _rows(gen, tokens, cols, dtype, ld, off)
    dYs, d_buf = _rows(gen, n, cols, dtype, ld, off)
    db = d_buf.clone()
    dw = torch.full((tokens, topk), 9.0, device="cuda")
    G.gemm_moe_combine_backward(tokens, topk, cols, dtype, pos, wd.cuda(), dY, ld, Ys, ld, n, dYs,
                                ld, dw)
    torch.cuda.synchronize()
    yv, dv = Ys.cpu().double(), dY.cpu().double()
    tok = torch.arange(n) // topk
    slot = torch.from_numpy(rr[:have]).long()
    wantw = torch.zeros(n, dtype=torch.float64)
    wantw[slot] = (yv[:have] * dv[tok[slot]]).sum(1)
    S = torch.zeros(n, dtype=torch.float64)
    S[slot] = (yv[:have] * dv[tok[slot]]).abs().sum(1)
    err = (dw.cpu().double().reshape(-1) - wantw).abs()
    assert (err <= (cols + 2) * R.U32 * S).all()
    wantd = dv[tok[slot]] * w.reshape(-1)[slot].double().unsqueeze(1)
    err = (dYs.cpu().double()[:have] - wantd).abs()
    assert (err <= R.half_step(dtype, wantd) * 1.001 + R.U32 * wantd.abs()).all()
    db[off:off + n * ld].view(n, ld)[:have, :cols] = dYs[:have]
    assert torch.equal(d_buf.view(torch.int16), db.view(torch.int16))


def test_gradient_against_differences():
    """sum(Y * dY) changes with a weight by dw and with a row by dYs."""
    gen = torch.Generator().manual_seed(3)
    T, K, C = 5, 3, 40
    ids = _ids(T, K, 4, 1, 0.2)
    _, order, pos = R.sort_ref(ids, 4)
    p = torch.from_numpy(pos.reshape(T, K))
    w = torch.rand(T, K, generator=gen).double()
    Ys = torch.randn(T * K, C, generator=gen).half().double()
    dY = torch.randn(T, C, generator=gen).half().double()
    f = lambda w_, y_: float((R.combine_ref(p, w_, y_)[0] * dY).sum())
    dYs = torch.zeros(T * K, C, dtype=torch.float16, device="cuda")
    dw = torch.empty(T, K, device="cuda")
    G.gemm_moe_combine_backward(T, K, C, "f16", p.cuda(), w.float().cuda(), dY.half().cuda(), 0,
                                Ys.half().cuda(), 0, T * K, dYs, 0, dw)
    torch.cuda.synchronize()
    h = 2.0 ** -10  # the function is linear in each argument: differences are exact to rounding
    for t in range(T):
        for k in range(K):
            a, b = w.clone(), w.clone()
            a[t, k] += h
            b[t, k] -= h
            assert abs((f(a, Ys) - f(b, Ys)) / (2 * h) - float(dw[t, k])) < 1e-4
    for r, c in [(0, 0), (3, 17), (7, 39)]:
        a, b = Ys.clone(), Ys.clone()
        a[r, c] += h
        b[r, c] -= h
        want = (f(w, a) - f(w, b)) / (2 * h)
        assert abs(want - float(dYs[r, c])) <= abs(want) * 2.0 ** -11 + 1e-6


def test_places_out_of_range_add_nothing():
    """Places are device data: those outside 0 .. rows-1 count as dropped."""
    pos = torch.tensor([[0, 9, -5], [2 ** 31 - 1, 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    Ys = torch.arange(16, dtype=torch.float32).view(2, 8).half().cuda()
    Y = torch.empty(2, 8, dtype=torch.float16, device="cuda")
    w = torch.full((2, 3), 2.0, device="cuda")
    G.gemm_moe_combine(2, 3, 8, "f16", pos, w, Ys, 0, 2, Y, 0)
    torch.cuda.synchronize()
    assert torch.equal(Y, 2 * Ys)
    dYs, dw = torch.zeros_like(Ys), torch.full((2, 3), 5.0, device="cuda")
    G.gemm_moe_combine_backward(2, 3, 8, "f16", pos, w, Ys, 0, Ys, 0, 2, dYs, 0, dw)
    torch.cuda.synchronize()
    assert torch.equal(dYs, 2 * Ys)
    assert dw.cpu().tolist() == [[140.0, 0.0, 0.0], [0.0, 1100.0, 0.0]]


def test_infinities_and_nan_stay_in_their_rows():
    pos = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    Ys = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    Ys[0, 3], Ys[1, 5], Ys[3] = float("inf"), float("nan"), float("nan")  # row 3: no slot's
    Y = torch.empty(2, 16, dtype=torch.bfloat16, device="cuda")
    G.gemm_moe_combine(2, 2, 16, "bf16", pos, torch.ones(2, 2, device="cuda"), Ys, 0, 4, Y, 0)
    y = Y.cpu().float()
    assert y[0, 3] == float("inf") and torch.isnan(y[0, 5])
    keep = [c for c in range(16) if c not in (3, 5)]
    assert (y[0, keep] == 2).all() and (y[1] == 1).all()
