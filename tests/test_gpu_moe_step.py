"""The mixture-of-experts operators together: one training step of a gated
MLP with experts (sparse_tiled_gemm_amd.moe) against 64-bit autograd, on
another stream, and captured into a HIP graph."""
import pytest
import torch

import moe_ref as R
from gpu_util import say
from sparse_tiled_gemm_amd import gemm as G
from sparse_tiled_gemm_amd import moe

pytestmark = pytest.mark.gpu


def _problem(tokens, hidden, inner, groups, topk, dtype, seed, drop=0.0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s, k=1.0: (torch.randn(*s, generator=gen) * k)
    W1 = rnd(groups, 2 * inner, hidden, k=hidden ** -0.5).to(dtype)
    W2 = rnd(groups, hidden, inner, k=inner ** -0.5).to(dtype)
    X, dY = rnd(tokens, hidden).to(dtype), rnd(tokens, hidden).to(dtype)
    w, ids = torch.topk(rnd(tokens, groups), topk, dim=1)
    ids[torch.rand(tokens, topk, generator=gen) < drop] = -1
    return X, dY, torch.softmax(w, 1), ids, W1, W2


def _reference(X, dY, w, ids, W1, W2, codes=None):
    """64-bit autograd of the same layer."""
    X, w, W1, W2 = (t.double().requires_grad_(True) for t in (X, w, W1, W2))
    inner = W2.shape[2]
    Y = []
    for t in range(len(X)):
        y = torch.zeros(X.shape[1], dtype=torch.float64)
        for k, e in enumerate(ids[t].tolist()):
            if e >= 0:
                gu = W1[e] @ X[t]
                h = torch.nn.functional.silu(gu[:inner]) * gu[inner:]
                y = y + w[t, k] * (W2[e] @ h)
        Y.append(y)
    Y = torch.stack(Y)
    (Y * dY.double()).sum().backward()
    return Y.detach(), X.grad, w.grad, W1.grad, W2.grad


def _close(got, want, tol, what):
    err = (got.double().cpu() - want).norm() / want.norm().clamp(min=1e-30)
    assert err < tol, (what, float(err))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hidden,inner,groups,topk,drop", [
    (37, 64, 40, 5, 2, 0.1), (1, 128, 64, 8, 2, 0.0), (150, 72, 104, 3, 3, 0.3)])
def test_step(tokens, hidden, inner, groups, topk, drop, dtype):
    say("step", tokens, hidden, inner, groups, topk, drop, dtype)
    p = _problem(tokens, hidden, inner, groups, topk, dtype, tokens, drop)
    layer = moe.ExpertMLP(p[4].cuda(), p[5].cuda(), tokens, topk)
    for keep8 in (False, True):
        Y = layer.forward(p[0].cuda(), p[3].cuda(), p[2].cuda(), keep8=keep8)
        dX, dw, dW1, dW2 = layer.backward(p[1].cuda())
        torch.cuda.synchronize()
        rY, rX, rw, rW1, rW2 = _reference(*p)
        # 16-bit activations between the products: a few roundings of 2^-8
        # (bf16) or 2^-11 (fp16) each; the checkpoint adds 2^-4 per kept value,
        # which the sums average
        e16 = 2.0 ** (-6 if dtype == torch.bfloat16 else -9)
        _close(Y, rY, e16, "Y")
        e = e16 + 2.0 ** -4  # dGU and dW pass through the kept codes
        for got, want, what in [(dX, rX, "dX"), (dW1, rW1, "dW1"), (dW2, rW2, "dW2")]:
            _close(got, want, e, what)
        _close(dw, rw, e16, "dw")


def test_accumulates_weight_gradients():
    p = _problem(40, 64, 32, 4, 2, torch.bfloat16, 1)
    layer = moe.ExpertMLP(p[4].cuda(), p[5].cuda(), 40, 2)
    X, ids, w, dY = p[0].cuda(), p[3].cuda(), p[2].cuda(), p[1].cuda()
    layer.forward(X, ids, w)
    _, _, a1, a2 = [t.clone() for t in layer.backward(dY)]
    layer.forward(X, ids, w)
    _, _, b1, b2 = layer.backward(dY, accumulate=True)
    torch.cuda.synchronize()
    # fp32: the second pass starts from the first's gradients
    assert ((b1 - 2 * a1).norm() / a1.norm()) < 1e-5 and ((b2 - 2 * a2).norm() / a2.norm()) < 1e-5


def test_other_stream_and_graph():
    """The same bits on another stream and from replays of a captured step,
    with new inputs between the replays."""
    p = _problem(200, 128, 64, 6, 2, torch.bfloat16, 2, 0.1)
    layer = moe.ExpertMLP(p[4].cuda(), p[5].cuda(), 200, 2)
    X, ids, w, dY = p[0].cuda(), p[3].cuda(), p[2].cuda(), p[1].cuda()

    def step():
        y = layer.forward(X, ids, w)
        return [y] + list(layer.backward(dY))

    def eager():
        out = [t.clone() for t in step()]
        torch.cuda.synchronize()
        return out

    want = eager()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = [t.clone() for t in step()]
    s.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        if i:
            q = _problem(200, 128, 64, 6, 2, torch.bfloat16, 10 + i, 0.1 * i)
            for dst, src in zip((X, dY, w, ids), q[:4]):
                dst.copy_(src)
        want = eager()
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [1, 40])
def test_strides_of_rows(tokens):
    """Padded, broadcast and overlapping rows give what packed copies give."""
    p = _problem(tokens, 64, 32, 4, 2, torch.bfloat16, 5)
    layer = moe.ExpertMLP(p[4].cuda(), p[5].cuda(), tokens, 2)
    X, ids, w, dY = p[0].cuda(), p[3].cuda(), p[2].cuda(), p[1].cuda()
    wide = torch.full((tokens, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :64] = X
    lapped = torch.randn(64 + 3 * tokens, device="cuda").bfloat16()
    for x, dy in [(wide[:, :64], dY), (X, wide[:, :64]), (X[:1].expand(tokens, 64), dY),
                  (X, dY[:1].expand(tokens, 64)), (lapped.as_strided((tokens, 64), (3, 1)), dY)]:
        say("strides", x.stride(), dy.stride())
        step = lambda x_, dy_: [t.clone() for t in (layer.forward(x_, ids, w),) + layer.backward(dy_)]
        got, want = step(x, dy), step(x.clone().contiguous(), dy.clone().contiguous())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_first_backward_may_accumulate():
    p = _problem(40, 64, 32, 4, 2, torch.bfloat16, 6)
    X, ids, w, dY = p[0].cuda(), p[3].cuda(), p[2].cuda(), p[1].cuda()
    out = []
    for accumulate in (False, True):
        # what the allocator hands out next has been used
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (4 * 64 * 64, 4 * 64 * 32) * 2]
        del junk
        layer = moe.ExpertMLP(p[4].cuda(), p[5].cuda(), 40, 2)
        layer.forward(X, ids, w)
        out.append([t.clone() for t in layer.backward(dY, accumulate=accumulate)])
    torch.cuda.synchronize()
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_weights_changed_between_the_passes():
    """backward() is the gradient of the forward pass that was run, eagerly and
    from two graphs with the weights changed between their replays."""
    p = _problem(40, 64, 32, 4, 2, torch.bfloat16, 7)
    layer = moe.ExpertMLP(p[4].cuda(), p[5].cuda(), 40, 2)
    X, ids, w, dY = p[0].cuda(), p[3].cuda(), p[2].cuda(), p[1].cuda()
    layer.forward(X, ids, w)
    want = [t.clone() for t in layer.backward(dY)]
    layer.forward(X, ids, w)
    w.mul_(3)
    got = [t.clone() for t in layer.backward(dY)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    fwd, bwd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(fwd):
        layer.forward(X, ids, w)
    with torch.cuda.graph(bwd):
        out = layer.backward(dY)
    for i in range(3):
        w.copy_(p[2])
        torch.cuda.synchronize()
        fwd.replay()
        w.fill_(float(i))
        bwd.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
            a.fill_(5)


def _from_codes(layer, X, dY, w, ids, W1, W2):
    """dX, dW1 and dW2 in 64 bits from the values that the layer kept."""
    v = R.q8_values(layer.codes.cpu(), layer.scales.cpu())
    xv = R.q8_values(layer.xcodes.cpu(), layer.xscales.cpu()) if layer.keep8 else None
    pos = layer.pos.cpu().view(ids.shape)
    X, dY, w, W1, W2 = (t.double() for t in (X, dY, w, W1, W2))
    inner = W2.shape[2]
    dX, dW1, dW2 = torch.zeros_like(X), torch.zeros_like(W1), torch.zeros_like(W2)
    for t in range(len(X)):
        for k, e in enumerate(ids[t].tolist()):
            if e < 0:
                continue
            p = int(pos[t, k])
            dys = w[t, k] * dY[t]
            (dg, du, h), _ = R.swiglu_backward_ref(v[p, :inner], v[p, inner:], W2[e].t() @ dys)
            dgu = torch.cat([dg, du])
            dW2[e] += torch.outer(dys, h)
            dW1[e] += torch.outer(dgu, X[t] if xv is None else xv[p])
            dX[t] += W1[e].t() @ dgu
    return dX, dW1, dW2


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hidden,inner,groups,topk,drop", [
    (37, 64, 40, 5, 2, 0.1), (1, 128, 64, 8, 2, 0.0), (150, 72, 104, 3, 3, 0.3)])
def test_gradients_at_the_kept_values(tokens, hidden, inner, groups, topk, drop, dtype, keep8):
    """Against the gradient at the values the codes stand for, what is left
    are the roundings of the 16-bit tensors on the way, half a step each: dYs,
    dH, dGU, dXs, dX for dX; dYs, dH, dGU for dW1; dYs, H for dW2."""
    say("kept values", tokens, hidden, inner, groups, topk, drop, dtype, keep8)
    p = _problem(tokens, hidden, inner, groups, topk, dtype, tokens + 1, drop)
    layer = moe.ExpertMLP(p[4].cuda(), p[5].cuda(), tokens, topk)
    layer.forward(p[0].cuda(), p[3].cuda(), p[2].cuda(), keep8=keep8)
    dX, _, dW1, dW2 = layer.backward(p[1].cuda())
    torch.cuda.synchronize()
    half = torch.finfo(dtype).eps / 2
    for got, want, n, what in zip((dX, dW1, dW2), _from_codes(layer, *p), (5, 3, 2),
                                  ("dX", "dW1", "dW2")):
        _close(got, want, n * half, what)


def test_the_current_stream_is_torch_s():
    """The binding's look-up of the stream against torch's public one."""
    for s in (torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert G._stream(None) == s.cuda_stream == torch.cuda.current_stream().cuda_stream
            assert G._stream(s) == s.cuda_stream
