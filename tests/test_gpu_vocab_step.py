"""The operators over a vocabulary together, as a training step uses them:
tokens looked up, the loss at their targets, both gradients into one table
(sparse_tiled_gemm_amd.vocab), alone and around an ExpertMLP, eager and
replayed."""
import pytest
import torch

from gpu_util import say
from moe_ref import DT, half_step
from sparse_tiled_gemm_amd.moe import ExpertMLP
from sparse_tiled_gemm_amd.vocab import TiedVocab
from vocab_ref import Xent, embed_grad_ref, embed_ref, far

pytestmark = pytest.mark.gpu


def table(vocab, hidden, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(vocab, hidden, generator=gen) * hidden ** -0.5).to(DT[dtype])


def batch(tokens, vocab, seed):
    gen = torch.Generator().manual_seed(100 + seed)
    ids, y = (torch.randint(0, vocab, (tokens,), generator=gen) for _ in range(2))
    ids[::17], y[::5] = -1, vocab + 3
    ids[1::4] = 2  # a frequent token
    return ids, y


@pytest.mark.parametrize("dtype,tokens,vocab,hidden,id_type", [
    ("bf16", 300, 700, 96, torch.int64), ("f16", 1500, 901, 77, torch.int32),
    ("bf16", 12, 2000, 200, torch.int64), ("f16", 1, 50, 8, torch.int32)])
def test_step_against_64_bits(dtype, tokens, vocab, hidden, id_type):
    say("step", dtype, tokens, vocab, hidden)
    E = table(vocab, hidden, dtype)
    ids, y = batch(tokens, vocab, 0)
    se, sl = hidden ** 0.5, 0.7
    ends = TiedVocab(E.cuda(), tokens, embed_scale=se, logit_scale=sl)
    X0 = ends.embed(ids.to(id_type).cuda())
    ref0 = embed_ref(ids, E, se)
    assert far(X0, ref0, ref0.abs() * 2.0 ** -24, dtype) <= 0
    X = X0 * 0.5 + 0.25  # the layers
    loss, lse = ends.loss(X, y.to(id_type).cuda())
    ref = Xent(X.cpu(), E, y, sl)
    rl, re, bl, be = ref.forward()
    assert far(loss, rl, bl, "f32") <= 0 and far(lse, re, be, "f32") <= 0
    n = max(1, int(ref.ok.sum()))
    dloss = torch.full((tokens,), (64.0 if dtype == "f16" else 1.0) / n)
    dX = ends.loss_backward(dloss.cuda())
    gX, gE, bX, bE = ref.grads(lse.cpu(), dloss, None, dtype)
    assert far(dX, gX, bX, dtype) <= 0
    half = ends.dE.clone()
    assert far(half, gE, bE, "f32") <= 0
    dX0 = dX * 0.5  # exact
    dE = ends.embed_backward(dX0)
    want, bound, _ = embed_grad_ref(ids, dX0.cpu(), vocab, se, half.cpu())
    assert far(dE, want, bound, "f32") <= 0
    # alone, and the loss's gradient added to it: another order of the same sums
    alone = ends.embed_backward(dX0, accumulate=False).clone()
    want, bound, _ = embed_grad_ref(ids, dX0.cpu(), vocab, se)
    assert far(alone, want, bound, "f32") <= 0
    ends.loss_backward(dloss.cuda(), accumulate=True)
    both = want + gE
    assert far(ends.dE, both, bound + bE + 2.0 ** -23 * (both.abs() + bound + bE), "f32") <= 0


def test_training_step_around_experts_replayed():
    """Lookup, ExpertMLP, loss and all gradients captured once and replayed with
    new tokens: the bits of the eager step, with eager steps between."""
    tokens, vocab, hidden, inner, groups, topk = 256, 1000, 128, 64, 4, 2
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: (torch.randn(s, generator=gen, device="cuda") * s[-1] ** -0.5).bfloat16()
    ends = TiedVocab(table(vocab, hidden, "bf16").cuda(), tokens, embed_scale=hidden ** 0.5)
    layer = ExpertMLP(rnd(groups, 2 * inner, hidden), rnd(groups, hidden, inner), tokens, topk)
    ids, y = (torch.zeros(tokens, dtype=torch.int64, device="cuda") for _ in range(2))
    experts = torch.zeros(tokens, topk, dtype=torch.int64, device="cuda")
    weights = torch.full((tokens, topk), 0.5, device="cuda")
    dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")

    def step():
        Y = layer.forward(ends.embed(ids), experts, weights)
        loss, lse = ends.loss(Y, y)
        dX0, dw, dW1, dW2 = layer.backward(ends.loss_backward(dloss))
        return loss, lse, dw, dW1, dW2, ends.embed_backward(dX0)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        a, b = batch(tokens, vocab, seed)
        ids.copy_(a), y.copy_(b)
        experts.copy_(torch.stack([a % groups, (a + 1) % groups], 1).clamp(min=0))
        want = [x.clone() for x in step()]
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(out, want)), seed
        assert all(bool(torch.isfinite(x).all()) for x in want)
        assert float(want[0].max()) > 0 and float(want[-1].abs().max()) > 0


def test_gradient_of_both_ends_against_differences():
    """dE, the sum of both ends' gradients, against differences of the 64-bit
    loss along it: within dE's own bounds (the loss's, dX's rounding carried
    through the lookup, and the sums') and the difference's h^2 term, taken from
    two step widths."""
    tokens, vocab, hidden = 128, 400, 64
    E = table(vocab, hidden, "bf16")
    ids, y = batch(tokens, vocab, 1)
    ends = TiedVocab(E.cuda(), tokens)
    X0 = ends.embed(ids.cuda())
    loss, lse = ends.loss(X0, y.cuda())
    dloss = torch.ones(tokens)
    dX = ends.loss_backward(dloss.cuda())
    dE = ends.embed_backward(dX).double().cpu()
    gX, _, bX, bE = Xent(X0.cpu(), E, y, 1.0).grads(lse.cpu(), dloss, None, "bf16")
    carried, summed, _ = embed_grad_ref(ids, (bX + half_step("bf16", gX.abs() + bX)), vocab, 1.0)
    bound = bE + carried + summed + embed_grad_ref(ids, dX.cpu(), vocab, 1.0, dE)[1]

    def value(e):
        x = torch.where(((ids >= 0) & (ids < vocab)).unsqueeze(1), e[ids.clamp(0, vocab - 1)], 0.0)
        z = x @ e.t()
        zy = z.gather(1, y.clamp(max=vocab - 1).unsqueeze(1)).squeeze(1)
        return float((torch.logsumexp(z, 1) - zy)[y < vocab].sum())

    d = dE / dE.norm()
    diff = lambda h: (value(E.double() + h * d) - value(E.double() - h * d)) / (2 * h)
    d1, d2 = diff(1e-4), diff(2e-4)
    assert abs(float((dE * d).sum()) - d1) <= float((bound * d.abs()).sum()) + abs(d2 - d1)


def test_the_first_call_may_add_to_the_gradient():
    """embed_backward() alone, and loss_backward(accumulate=True), as a new
    object's first call: what the overwriting calls give."""
    tokens, vocab, hidden = 90, 300, 64
    E = table(vocab, hidden, "bf16").cuda()
    ids, y = (x.cuda() for x in batch(tokens, vocab, 2))
    gen = torch.Generator().manual_seed(4)
    X = torch.randn(tokens, hidden, generator=gen).bfloat16().cuda()
    dloss = torch.ones(tokens, device="cuda")

    def made():  # on memory that has been used
        junk = [torch.full((vocab * hidden,), float("nan"), device="cuda") for _ in range(4)]
        del junk
        return TiedVocab(E, tokens)

    out = []
    for accumulate in (False, True):
        ends = made()
        ends.embed(ids)
        looked_up = ends.embed_backward(X, accumulate=accumulate).clone()
        ends = made()
        ends.loss(X, y)
        ends.loss_backward(dloss, accumulate=accumulate)
        out.append((looked_up, ends.dE.clone()))
    for a, b in zip(*out):
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b)
