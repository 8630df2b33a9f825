"""A gated MLP with experts, one training step at a time, on the operators of
include/gemm_moe.h: the path that runs them together.

    layer = ExpertMLP(W1, W2, tokens, topk)
    Y = layer.forward(X, ids, weights)
    dX, dweights, dW1, dW2 = layer.backward(dY)

W1 (experts x 2F x H) holds each expert's gate and up projection, W2 (experts
x H x F) its down projection; X is tokens x H, ids (int32 or int64) and
weights (fp32) are tokens x topk, an id out of range drops its slot.  dW1 and
dW2 (fp32) have W1's and W2's layout.  Each forward() uses W1 and W2 as they
are then (contiguous ones are read where they lie, others copied first); they
must not change before its backward().

All buffers are made once and belong to the layer, those it returns among
them: Y is overwritten by the next forward(), the gradients by the next
backward().  A step only enqueues kernels, so it may be captured into a HIP
graph (rows of X or dY that share memory are copied out first).

backward() is the gradient of the last forward().  It reads the input of the
activation as 8-bit codes and, after forward(keep8=True), the sorted input
rows for dW1 as well: half the bytes, at 4 significant bits.  The 16-bit
buffers those come from (GU, and Xs) are then free between the passes, but
this layer keeps them, so that it takes no less memory for the codes.

`python -m sparse_tiled_gemm_amd.moe` runs a step and prints the time of each part.
"""
import torch

from . import gemm as G

_NAME = {torch.float16: "f16", torch.bfloat16: "bf16"}


def _rows(x):
    """x (rows with contiguous elements) and its leading dimension.  Rows that
    share memory (one row broadcast to all: a stride of 0, which the library
    takes for "packed") are copied out; a single row's stride means nothing."""
    rows, cols = x.shape
    if rows > 1 and x.stride(0) < cols:
        x = x.contiguous()
    return x, x.stride(0) if rows > 1 else cols


def _check_device(device, **tensors):
    """The library takes addresses: what lies elsewhere would fault in a kernel."""
    for name, x in tensors.items():
        if not x.is_cuda or x.device != device:
            raise ValueError("%s has to lie on the weights' GPU" % name)
    if device.type == "cuda" and device.index != torch.cuda.current_device():
        raise ValueError("the weights' GPU has to be the current one")


class ExpertMLP:
    def __init__(self, W1, W2, tokens, topk):
        self.groups, two_f, self.hidden = W1.shape
        self.inner = two_f // 2
        if W2.shape != (self.groups, self.hidden, self.inner) or W1.dtype != W2.dtype or \
                two_f % 2 or W1.dtype not in _NAME:
            raise ValueError("W1 (experts x 2F x H) and W2 (experts x H x F) in f16 or bf16")
        _check_device(W1.device, W1=W1, W2=W2)
        # weights that are not contiguous: copies, renewed by each forward pass
        self.W1, self.W2 = (w if w.is_contiguous() else w.detach().contiguous() for w in (W1, W2))
        self.copied = [(own, given) for own, given in ((self.W1, W1), (self.W2, W2))
                       if own is not given]
        self.tokens, self.topk = tokens, topk
        dt, dev = W1.dtype, W1.device
        self.dtype = _NAME[dt]
        n, g, h, f, t = tokens * topk, self.groups, self.hidden, self.inner, self.dtype
        mk = lambda *s, d=dt: torch.empty(s, dtype=d, device=dev)
        i32, u8, f32 = torch.int32, torch.uint8, torch.float32
        # rows past the last group are never written: zeros keep them finite
        z = lambda *s, d=dt: torch.zeros(s, dtype=d, device=dev)
        self.offsets, self.order, self.pos = mk(g + 1, d=i32), mk(n, d=i32), mk(n, d=i32)
        self.ws = mk(max(G.gemm_moe_sort_workspace(tokens, topk, g), 1), d=u8)
        self.Xs, self.GU, self.H, self.Ys = z(n, h), z(n, 2 * f), z(n, f), z(n, h)
        self.codes, self.scales = mk(n, 2 * f, d=u8), mk(n, (2 * f + 31) // 32, d=u8)
        self.xcodes, self.xscales = mk(n, h, d=u8), mk(n, (h + 31) // 32, d=u8)
        self.Y, self.dX, self.dw = mk(tokens, h), mk(tokens, h), mk(tokens, topk, d=f32)
        # the forward pass's own copy: the caller may change its tensor before
        # the backward pass
        self.weights = mk(tokens, topk, d=f32)
        self.dYs, self.dH, self.dGU, self.dXs = z(n, h), z(n, f), z(n, 2 * f), z(n, h)
        # in W1's and W2's layout; zeros, so that the first step may accumulate
        self.dW1, self.dW2 = z(g, 2 * f, h, d=f32), z(g, h, f, d=f32)
        plan = lambda *a, **k: G.gemm_grouped_plan(G.make_grouped_desc(*a, **k))
        self.p_up = plan("rows", n, 2 * f, h, g, t, t, t)
        self.p_down = plan("rows", n, h, f, g, t, t, t)
        self.p_dh = plan("rows", n, f, h, g, t, t, t, b_layout="row")
        self.p_dx = plan("rows", n, h, 2 * f, g, t, t, t, b_layout="row")
        self.p_dw1 = {(k8, acc): plan("weights", n, h, 2 * f, g, t, "e4m3" if k8 else t, "f32",
                                      has_c=acc) for k8 in (False, True) for acc in (False, True)}
        self.p_dw2 = {acc: plan("weights", n, f, h, g, t, t, "f32", has_c=acc)
                      for acc in (False, True)}
        self.keep8 = None  # of the last forward pass; None: there was none

    def forward(self, X, ids, weights, keep8=False):
        """Y = sum over each token's experts of weight * W2 (silu(W1g x) * W1u x)."""
        T, K, n, h, f, t = self.tokens, self.topk, len(self.pos), self.hidden, self.inner, self.dtype
        if X.shape != (T, h) or ids.shape != (T, K) or weights.shape != (T, K):
            raise ValueError("X is tokens x H, ids and weights tokens x topk")
        if X.dtype != self.W1.dtype or X.stride(1) != 1 or weights.dtype != torch.float32 or \
                not (ids.is_contiguous() and weights.is_contiguous()):
            raise ValueError("X in the weights' type with contiguous rows, ids and fp32 weights packed")
        if ids.dtype not in (torch.int32, torch.int64):
            raise ValueError("ids in int32 or int64")
        _check_device(self.W1.device, X=X, ids=ids, weights=weights)
        for own, given in self.copied:
            own.copy_(given.detach())
        self.weights.copy_(weights.detach())  # no graph of the caller's
        X, ldx = _rows(X)
        G.gemm_moe_dispatch(T, K, self.groups, h, t, ids, X, ldx, self.offsets, self.order,
                            self.pos, self.Xs, h, self.ws, id_bytes=ids.element_size())
        G.gemm_grouped_run(self.p_up, self.Xs, self.W1, None, self.offsets, None, self.GU)
        G.gemm_swiglu(n, f, t, self.GU, 2 * f, self.H, f, self.codes, self.scales)
        G.gemm_grouped_run(self.p_down, self.H, self.W2, None, self.offsets, None, self.Ys)
        G.gemm_moe_combine(T, K, h, t, self.pos, self.weights, self.Ys, h, n, self.Y, h)
        self.keep8 = bool(keep8)
        if self.keep8:  # the sorted inputs wait for the backward pass in 8 bits
            G.gemm_q8_store(n, h, t, self.Xs, h, self.xcodes, self.xscales)
        return self.Y

    def backward(self, dY, accumulate=False):
        """dX, the gradient of the weights of the choices, dW1 and dW2 (fp32);
        accumulate: dW1 and dW2 are added to what they held."""
        T, K, n, h, f, t = self.tokens, self.topk, len(self.pos), self.hidden, self.inner, self.dtype
        if dY.shape != (T, h) or dY.dtype != self.W1.dtype or dY.stride(1) != 1:
            raise ValueError("dY is tokens x H in the weights' type with contiguous rows")
        if self.keep8 is None:
            raise RuntimeError("backward before the first forward")
        _check_device(self.W1.device, dY=dY)
        accumulate = bool(accumulate)
        dY, lddy = _rows(dY)
        G.gemm_moe_combine_backward(T, K, h, t, self.pos, self.weights, dY, lddy, self.Ys, h, n,
                                    self.dYs, h, self.dw)
        G.gemm_grouped_run(self.p_dh, self.dYs, self.W2, None, self.offsets, None, self.dH)
        G.gemm_swiglu_backward(n, f, t, self.codes, self.scales, self.dH, f, self.dGU, 2 * f,
                               self.H, f)
        c = (lambda d: d) if accumulate else (lambda d: None)
        G.gemm_grouped_run(self.p_dw2[accumulate], self.dYs, self.H, None, self.offsets,
                           c(self.dW2), self.dW2)
        if self.keep8:
            G.gemm_grouped_run(self.p_dw1[True, accumulate], self.dGU, self.xcodes, self.xscales,
                               self.offsets, c(self.dW1), self.dW1)
        else:
            G.gemm_grouped_run(self.p_dw1[False, accumulate], self.dGU, self.Xs, None, self.offsets,
                               c(self.dW1), self.dW1)
        G.gemm_grouped_run(self.p_dx, self.dGU, self.W1, None, self.offsets, None, self.dXs)
        G.gemm_moe_combine(T, K, h, t, self.pos, None, self.dXs, h, n, self.dX, h)
        return self.dX, self.dw, self.dW1, self.dW2


def main(tokens=4096, hidden=4096, inner=2048, groups=16, topk=2, steps=10):
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s, k=1.0: (torch.randn(s, generator=gen, device="cuda") * k).bfloat16()
    layer = ExpertMLP(rnd(groups, 2 * inner, hidden, k=hidden ** -0.5),
                      rnd(groups, hidden, inner, k=inner ** -0.5), tokens, topk)
    X, dY = rnd(tokens, hidden), rnd(tokens, hidden)
    w, ids = torch.topk(torch.randn(tokens, groups, generator=gen, device="cuda"), topk, dim=1)
    w = torch.softmax(w, 1)
    for part, fn in [("forward", lambda: layer.forward(X, ids, w)),
                     ("backward", lambda: layer.backward(dY))]:
        for _ in range(3):
            fn()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(steps):
            fn()
        b.record()
        torch.cuda.synchronize()
        ms = a.elapsed_time(b) / steps
        flops = 6 * tokens * topk * hidden * inner * (1 if part == "forward" else 2)
        print("%s: %.3f ms, %.0f TFLOP/s (%d tokens, %d of %d experts, %d x %d, bf16)" %
              (part, ms, flops / ms / 1e9, tokens, topk, groups, hidden, inner), flush=True)


if __name__ == "__main__":
    main()
