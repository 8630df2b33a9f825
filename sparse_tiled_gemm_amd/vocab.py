"""The two ends of a language model on one matrix E (vocab x hidden), on the
operators of include/gemm_vocab.h: tokens in, loss out, and the gradients.

    ends = TiedVocab(E, tokens)
    X0 = ends.embed(ids)                 # scale * E[ids]
    ...                                  # the layers: X from X0
    loss, lse = ends.loss(X, targets)    # by token
    dX = ends.loss_backward(dloss)       # starts dE
    ...                                  # the layers' gradients: dX0 from dX
    dE = ends.embed_backward(dX0)        # completes dE

E is f16 or bf16, X and dX0 have its type, dE is fp32.  ids and targets are int32 or
int64; an id out of range is padding (a row of zeros, no gradient), a target
out of range a token that does not count (loss and lse 0, a row of zeros in
dX).  dE begins as zeros, so that a new object's first call may add to it.  dloss and dlse are fp32, by token: the mean of the losses has dloss =
1 / (number of targets).

All buffers are made once and belong to the object, those it returns among
them: each is overwritten by the next call of its kind.  (dE and the workspace of
the gradients are there for an object that only scores too.)  One workspace serves
all calls, so an object's calls belong on one stream at a time.  E has at most
2^20 rows and is read where it lies, at each call.  A step only enqueues kernels, so it may be captured into a HIP
graph; X, ids and targets must not change between a call and its gradient's.

`python -m sparse_tiled_gemm_amd.vocab` runs a step and prints the time of each part.
"""
import torch

from . import gemm as G
from .moe import _NAME, _check_device, _rows


class TiedVocab:
    def __init__(self, E, tokens, embed_scale=1.0, logit_scale=1.0):
        if E.dim() != 2 or E.dtype not in _NAME:
            raise ValueError("E (vocab x hidden) in f16 or bf16")
        if E.stride(1) != 1 or (len(E) > 1 and E.stride(0) < E.shape[1]):
            raise ValueError("E's rows have to be contiguous and apart")
        _check_device(E.device, E=E)
        self.E, self.tokens = E.detach(), tokens
        self.vocab, self.hidden = E.shape
        self.lde = _rows(self.E)[1]
        self.embed_scale, self.logit_scale = float(embed_scale), float(logit_scale)
        self.dtype, dev = _NAME[E.dtype], E.device
        mk = lambda *s, d=E.dtype: torch.empty(s, dtype=d, device=dev)
        f32, u8 = torch.float32, torch.uint8
        self.X0, self.dX = mk(tokens, self.hidden), mk(tokens, self.hidden)
        self.loss_, self.lse = mk(tokens, d=f32), mk(tokens, d=f32)
        # zeros, so that the first call may add to it
        self.dE = torch.zeros((self.vocab, self.hidden), dtype=f32, device=dev)
        self.plans = {}
        # (its size is the same for every plan of this object)
        self.ws = mk(max(G.gemm_embed_workspace(tokens, self.vocab, self.hidden),
                         *G.gemm_xent_workspace(self._plan(4, self.hidden, False)), 1), d=u8)
        self.ids = self.seen = None  # of the last embed() and loss()

    def _plan(self, id_bytes, ldx, accumulate):
        key = id_bytes, ldx, accumulate
        if key not in self.plans:
            self.plans[key] = G.gemm_xent_plan(G.make_xent_desc(
                self.tokens, self.vocab, self.hidden, self.dtype, self.dtype, "f32",
                scale=self.logit_scale, id_bytes=id_bytes, accumulate=accumulate, ldx=ldx, ldw=self.lde,
                unaligned=self.E.data_ptr() % 16 != 0))
        return self.plans[key]

    def _ids(self, name, x):
        if x.shape != (self.tokens,) or x.dtype not in (torch.int32, torch.int64) or \
                not x.is_contiguous():
            raise ValueError("%s: one int32 or int64 per token, packed" % name)
        _check_device(self.E.device, **{name: x})
        return x

    def _matrix(self, name, x):
        if x.shape != (self.tokens, self.hidden) or x.dtype != self.E.dtype or x.stride(1) != 1:
            raise ValueError("%s is tokens x hidden in E's type with contiguous rows" % name)
        _check_device(self.E.device, **{name: x})
        return _rows(x.detach())

    def _vector(self, name, x):
        if x.shape != (self.tokens,) or x.dtype != torch.float32 or not x.is_contiguous():
            raise ValueError("%s: one fp32 value per token, packed" % name)
        _check_device(self.E.device, **{name: x})
        return x.detach()

    def embed(self, ids):
        """X0 = embed_scale * E[ids]."""
        self.ids = self._ids("ids", ids)
        G.gemm_embed(self.tokens, self.vocab, self.hidden, self.dtype, self.dtype, ids, self.E, self.lde,
                     self.X0, 0, scale=self.embed_scale, id_bytes=ids.element_size())
        return self.X0

    def loss(self, X, targets):
        """loss and lse of softmax(logit_scale * X E^T) at the targets, by token."""
        self._ids("targets", targets)
        X, ldx = self._matrix("X", X)
        plan = self._plan(targets.element_size(), ldx, False)
        G.gemm_xent_forward(plan, X, self.E, targets, self.loss_, self.lse, self.ws)
        self.seen = X, ldx, targets
        return self.loss_, self.lse

    def loss_backward(self, dloss, dlse=None, accumulate=False):
        """dX of the last loss(); dE is overwritten, or added to (accumulate)."""
        if self.seen is None:
            raise RuntimeError("loss_backward before the first loss")
        dloss = self._vector("dloss", dloss)
        dlse = None if dlse is None else self._vector("dlse", dlse)
        X, ldx, targets = self.seen
        plan = self._plan(targets.element_size(), ldx, bool(accumulate))
        G.gemm_xent_backward(plan, X, self.E, targets, self.lse, dloss, dlse, self.dX, self.dE, self.ws)
        return self.dX

    def embed_backward(self, dX0, accumulate=True):
        """The gradient of the last embed(), added to dE (the default: what
        loss_backward() left there) or alone."""
        if self.ids is None:
            raise RuntimeError("embed_backward before the first embed")
        dX0, lddx = self._matrix("dX0", dX0)
        G.gemm_embed_backward(self.tokens, self.vocab, self.hidden, self.dtype, "f32", self.ids, dX0,
                              lddx, self.dE, 0, self.ws, scale=self.embed_scale,
                              accumulate=accumulate, id_bytes=self.ids.element_size())
        return self.dE


def main(tokens=8192, vocab=131072, hidden=4096, steps=5):
    gen = torch.Generator(device="cuda").manual_seed(0)
    E = (torch.randn(vocab, hidden, generator=gen, device="cuda") * hidden ** -0.5).bfloat16()
    ends = TiedVocab(E, tokens)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    X = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")
    flops = 2 * tokens * vocab * hidden
    for part, fn, f in [("embed", lambda: ends.embed(ids), 0), ("loss", lambda: ends.loss(X, ids), flops),
                        ("loss_backward", lambda: ends.loss_backward(dloss), 3 * flops),
                        ("embed_backward", lambda: ends.embed_backward(X), 0)]:
        for _ in range(2):
            fn()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(steps):
            fn()
        b.record()
        torch.cuda.synchronize()
        ms = a.elapsed_time(b) / steps
        print("%s: %.3f ms%s (%d tokens, %d x %d, bf16)" %
              (part, ms, ", %.0f TFLOP/s" % (f / ms / 1e9) if f else "", tokens, vocab, hidden),
              flush=True)


if __name__ == "__main__":
    main()
