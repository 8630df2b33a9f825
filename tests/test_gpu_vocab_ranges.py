"""The operators over a vocabulary at sizes that choose other kernels, or other
ways through them: the sort of the lookup's gradient at the smallest and
largest vocabularies and below eight columns, large lookups on both sides of
their borders, and the cross entropy of so many tokens that its preparation
takes several steps per workgroup."""
import pytest
import torch

import test_gpu_embed as embed
from gpu_util import say
from moe_ref import DT
from sparse_tiled_gemm_amd import gemm as G
from test_gpu_xent import make
from vocab_ref import Xent, embed_grad_ref, far

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the sort

@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,vocab,cols,kind", [
    (3000, 1, 8, "one"), (3000, 1, 7, "all"), (3000, 2, 513, "all"), (2100, 2, 1, "hot"),
    (2049, 3, 1, "all"), (3000, 3, 7, "hot"), (5000, 4, 5, "some"), (2500, 500, 1027, "hot"),
    (3000, 40, 3, "ends"), (2049, 1 << 20, 8, "some"), (40000, 1 << 20, 5, "hot"),
    (40000, (1 << 20) - 1, 16, "some"), (3000, 1 << 19, 7, "all")])
def test_sorted_gradient(tokens, vocab, cols, kind, accumulate):
    """From 2049 tokens on; 0 to 10 low and high bits of the ids."""
    embed.run_gradient(kind, tokens, vocab, cols, "f16", "f32", accumulate, 8, 0, 1.0)


@pytest.mark.parametrize("y,e", [("f32", "bf16"), ("bf16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("cols,pad", [(1, 2), (7, 0), (7, 5), (9, 1)])
def test_sorted_gradient_of_narrow_rows(y, e, cols, pad):
    embed.run_gradient("hot", 2500, 90, cols, y, e, False, 4, pad, 2.0)
    embed.run_gradient("hot", 2500, 90, cols, y, e, True, 4, pad, 2.0)


def test_sorted_gradients_at_once():
    """On two streams, a workspace each."""
    tokens, vocab, cols = 3000, 400, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    ids = [torch.randint(0, vocab, (tokens,), generator=gen, device="cuda") for _ in range(2)]
    dY = [torch.randint(-8, 9, (tokens, cols), generator=gen, device="cuda").half() for _ in range(2)]
    D = [torch.empty(vocab, cols, device="cuda") for _ in range(2)]
    n = G.gemm_embed_workspace(tokens, vocab, cols)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                G.gemm_embed_backward(tokens, vocab, cols, "f16", "f32", ids[i], dY[i], 0, D[i], 0, ws[i],
                                      id_bytes=8)
    torch.cuda.synchronize()
    for i in range(2):
        want = embed_grad_ref(ids[i].cpu(), dY[i].cpu(), vocab, 1.0)[0]
        assert torch.equal(D[i].cpu().double(), want)


# ---------------------------------------------------------------- large lookups

@pytest.mark.parametrize("e,y,tokens,cols,pad", [
    # 2^22 values and more: four tokens at a time, 16 or 64 lanes each
    ("bf16", "bf16", 32771, 128, 0), ("f32", "f16", 34953, 120, 8), ("f16", "bf16", 32767, 128, 0),
    ("bf16", "bf16", 600001, 7, 0), ("f16", "f32", 600003, 7, 3),
    ("bf16", "bf16", 4099, 1027, 0), ("f32", "bf16", 4086, 1027, 5), ("bf16", "f32", 4094, 1032, 8),
    # outputs of 32 MB and more: past the caches
    ("bf16", "bf16", 139811, 120, 0), ("f32", "f32", 69907, 120, 1), ("bf16", "f32", 1198373, 7, 0),
    ("bf16", "bf16", 16337, 1027, 0), ("f16", "f16", 16337, 1027, 3), ("f32", "f32", 8169, 1027, 0),
    ("bf16", "f32", 8131, 1032, 8), ("f32", "bf16", 16258, 1032, 0)])
def test_large_lookup(e, y, tokens, cols, pad):
    """Numbers of tokens that are no multiple of four, ids without a row among
    them, nothing written between the rows."""
    embed.test_lookup(e, y, tokens, 3001, cols, pad, 8)


# ---------------------------------------------------------------- many tokens

def loss_and_gradients(X, W, y, dtype, dloss, dlse):
    tokens, vocab, hidden = len(X), len(W), X.shape[1]
    say("xent", tokens, vocab, hidden, dtype)
    plan = G.gemm_xent_plan(G.make_xent_desc(tokens, vocab, hidden, dtype, "f32", "f32", id_bytes=8))
    ws = torch.empty(max(G.gemm_xent_workspace(plan)), dtype=torch.uint8, device="cuda")
    loss, lse = (torch.full((tokens,), 7.0, device="cuda") for _ in range(2))
    Xd, Wd, yd = X.cuda(), W.cuda(), y.cuda()
    G.gemm_xent_forward(plan, Xd, Wd, yd, loss, lse, ws)
    dX, dW = torch.empty(tokens, hidden, device="cuda"), torch.empty(vocab, hidden, device="cuda")
    G.gemm_xent_backward(plan, Xd, Wd, yd, lse, dloss.cuda(), dlse.cuda(), dX, dW, ws)
    return loss, lse, dX, dW


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,vocab,hidden", [
    (8193, 300, 24), (9001, 130, 40), (16385, 70, 16), (32768, 70, 16), (32769, 70, 16), (40001, 130, 9),
    (70001, 60, 8)])
def test_many_tokens(dtype, tokens, vocab, hidden):
    """Whole workgroups without a target, and the largest coefficient in the
    last one that has some, a thousand times the others."""
    X, W, y = make(tokens, vocab, hidden, dtype, ignore=0.3)
    y[100:700] = -1
    y[-1] = vocab - 1
    gen = torch.Generator().manual_seed(1)
    dloss, dlse = torch.rand(tokens, generator=gen) + 0.5, torch.rand(tokens, generator=gen) - 0.3
    dloss[-1] = 1000.0
    loss, lse, dX, dW = loss_and_gradients(X, W, y, dtype, dloss, dlse)
    ref = Xent(X, W, y, 1.0)
    rl, re, bl, be = ref.forward()
    assert far(loss, rl, bl, "f32") <= 0 and far(lse, re, be, "f32") <= 0
    gX, gW, bX, bW = ref.grads(lse.cpu(), dloss, dlse, dtype)
    assert far(dX, gX, bX, "f32") <= 0, "dX"
    assert far(dW, gW, bW, "f32") <= 0, "dW"
    assert not bool(dX[~ref.ok.cuda()].any())


@pytest.mark.parametrize("tokens", [4, 70])
def test_a_bad_row_of_no_weight_is_not_hidden(tokens):
    """X holds an infinity or NaN, and the token's dloss is zero: its row of dX
    is NaN, the others keep their values."""
    vocab, hidden = 500, 64
    X, W, y = make(tokens, vocab, hidden, "bf16", ignore=0.0)
    X[1, 0], X[3, 2] = float("inf"), float("nan")
    good = torch.ones(tokens, dtype=torch.bool)
    good[[1, 3]] = False
    dloss, dlse = good.float(), torch.zeros(tokens)
    loss, lse, dX, _ = loss_and_gradients(X, W, y, "bf16", dloss, dlse)
    assert not bool(torch.isfinite(dX[~good.cuda()]).any())
    n = int(good.sum())
    gX, _, bX, _ = Xent(X[good], W, y[good], 1.0).grads(lse.cpu()[good], torch.ones(n), torch.zeros(n),
                                                       "bf16")
    assert far(dX[good.cuda()], gX, bX, "f32") <= 0
