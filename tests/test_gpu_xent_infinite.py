"""Infinite logits of the linear cross entropy: lse and loss are what log sum exp
gives, infinities of either sign among finite logits and alone, in every kernel
of the forward pass."""
import pytest
import torch

from gpu_util import say
from moe_ref import DT
from sparse_tiled_gemm_amd import gemm as G
from test_gpu_xent import make
from vocab_ref import Xent, far

pytestmark = pytest.mark.gpu


def forward(X, W, y, dtype, **kw):
    tokens, hidden = X.shape
    plan = G.gemm_xent_plan(G.make_xent_desc(tokens, len(W), hidden, dtype, "f32", "f32", id_bytes=8, **kw))
    say("xent", tokens, len(W), hidden, dtype, plan.name)
    ws = torch.empty(max(G.gemm_xent_workspace(plan)), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    G.gemm_xent_forward(plan, X.cuda(), W.cuda(), y.cuda(), loss, lse, ws)
    return loss.cpu(), lse.cpu(), plan, ws


@pytest.mark.parametrize("tile", [None, "tiled64", "tiled128", "tiled256"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,vocab,hidden", [
    (1, 200, 64), (5, 700, 64), (12, 3001, 77), (40, 500, 64), (100, 1300, 72), (300, 900, 136)])
def test_one_infinite_row_of_the_weights(monkeypatch, tile, dtype, tokens, vocab, hidden):
    """Column v's logit is +inf for half of the tokens (lse +inf) and -inf for
    the others (nothing in their sums)."""
    if tile:
        monkeypatch.setenv("STGEMM_FORCE_KERNEL", tile)
    X, W, y = make(tokens, vocab, hidden, dtype, ignore=0.0)
    plus = torch.arange(tokens) % 2 == 0
    X[:, 0] = torch.where(plus, 1.0, -1.0)
    y %= vocab - 1  # (column v is the last one first, so that the rest stays whole)
    rest = Xent(X[~plus], W[:-1], y[~plus], 1.0).forward() if tokens > 1 else None
    for v in {vocab - 1, 0, vocab // 2}:
        Wi, yi = W.clone(), y.clone()
        Wi[[v, vocab - 1]] = Wi[[vocab - 1, v]]
        yi[y == v] = vocab - 1
        Wi[v] = 0.0
        Wi[v, 0] = float("inf")
        if tokens > 2:
            yi[2], yi[1] = v, v  # +inf - inf, and -(-inf)
        loss, lse, _, _ = forward(X, Wi, yi, dtype)
        assert bool((lse[plus] == float("inf")).all())
        own = torch.zeros(tokens, dtype=torch.bool)
        if tokens > 2:
            own[[1, 2]] = True
            assert bool(torch.isnan(loss[2])) and float(loss[1]) == float("inf")
        assert bool((loss[plus & ~own] == float("inf")).all())
        if rest:
            few = ~own[~plus]
            assert far(lse[~plus], rest[1], rest[3], "f32") <= 0
            assert far(loss[~plus][few], rest[0][few], rest[2][few], "f32") <= 0


@pytest.mark.parametrize("tile", [None, "tiled64", "tiled256"])
def test_only_infinite_logits(monkeypatch, tile):
    """All -inf: lse -inf.  All +inf: lse +inf.  A NaN among either: NaN."""
    if tile:
        monkeypatch.setenv("STGEMM_FORCE_KERNEL", tile)
    vocab, hidden = 300, 64
    W = torch.ones(vocab, hidden).bfloat16()
    W[:, 0] = float("inf")
    for tokens in (6, 70):
        X = torch.ones(tokens, hidden).bfloat16()
        X[1::3, 0] = -1.0
        X[2::3, 0] = float("nan")
        loss, lse, _, _ = forward(X, W, torch.zeros(tokens, dtype=torch.int64), "bf16")
        assert bool((lse[0::3] == float("inf")).all()) and bool((lse[1::3] == -float("inf")).all())
        assert bool(torch.isnan(lse[2::3]).all()) and bool(torch.isnan(loss).all())


@pytest.mark.parametrize("tokens", [5, 40, 300])
def test_gradient_of_an_infinite_logit(tokens):
    """Its token's row of dX and its column's row of dW are NaN, dW's others finite."""
    vocab, hidden = 700, 64
    X, W, y = make(tokens, vocab, hidden, "bf16", ignore=0.0)
    y %= vocab - 1
    X[:, 0] = -1.0
    X[3, 0] = 1.0
    W[-1] = 0.0
    W[-1, 0] = float("inf")
    loss, lse, plan, ws = forward(X, W, y, "bf16")
    assert float(lse[3]) == float("inf") and bool(torch.isfinite(lse[torch.arange(tokens) != 3]).all())
    dX, dW = torch.empty(tokens, hidden, device="cuda"), torch.empty(vocab, hidden, device="cuda")
    G.gemm_xent_backward(plan, X.cuda(), W.cuda(), y.cuda(), lse.cuda(), torch.ones(tokens, device="cuda"),
                         None, dX, dW, ws)
    assert bool(torch.isnan(dX[3]).all()) and bool(torch.isnan(dW[-1]).all())
    assert bool(torch.isfinite(dW[:-1]).all())
