"""Plain 64-bit references (on the CPU) of the operators over a vocabulary,
and the error bounds their tests use.

A rounding to a type is off by at most half a step: eps/2 relative, and half
the smallest subnormal below the normal range (half_step).  A sum of n products in
fp32 is off by at most n roundings of the sum of magnitudes, whatever its
order."""
import numpy as np
import torch

from moe_ref import DT, U32, half_step

LOG2E = 1.4426950408889634


def valid(ids, vocab):
    return (ids >= 0) & (ids < vocab)


def embed_ref(ids, E, scale):
    """Y (64 bits): the rows of E, zeros for ids that name none."""
    ok = valid(ids, len(E))
    Y = torch.zeros(len(ids), E.shape[1], dtype=torch.float64)
    Y[ok] = E[ids[ok]].double() * float(np.float32(scale))
    return Y


def embed_grad_ref(ids, dY, vocab, scale, before=None):
    """dE and its bound without the last rounding: n + 1 roundings of the sum
    of magnitudes (n additions of a row's tokens, the scale's product) and, with
    what was there before, one of the sum with that."""
    ok = valid(ids, vocab)
    k = float(np.float32(scale))
    D = torch.zeros(vocab, dY.shape[1], dtype=torch.float64)
    S = torch.zeros_like(D)
    n = torch.zeros(vocab, 1, dtype=torch.float64)
    D.index_add_(0, ids[ok], dY[ok].double())
    S.index_add_(0, ids[ok], dY[ok].double().abs())
    n.index_add_(0, ids[ok], torch.ones(int(ok.sum()), 1, dtype=torch.float64))
    D, S = D * k, S * abs(k)
    B = (n + 1) * U32 * S
    if before is not None:
        B += U32 * (before.double().abs() + S) * (n > 0)
        D += before.double()
    return D, B, n.squeeze(1) > 0


class Xent:
    """The linear cross entropy in 64 bits, with bounds of the kernels' errors."""

    def __init__(self, X, W, targets, scale):
        self.k = float(np.float32(scale))
        self.ok = valid(targets, len(W))
        self.rows = torch.nonzero(self.ok).squeeze(1)
        self.y = targets[self.rows]
        self.X, self.W = X[self.rows].double(), W.double()
        self.T = len(targets)
        self.z = self.X @ self.W.t() * self.k
        # hidden products summed in fp32, and the scale's product
        S = self.X.abs() @ self.W.abs().t() * abs(self.k)
        self.dz = (X.shape[1] + 1) * U32 * S
        self.lse_rows = torch.logsumexp(self.z, 1) if len(self.rows) else self.z.sum(1)

    def forward(self):
        """loss, lse and their bounds, by token."""
        V = self.W.shape[0]
        at = self.y.unsqueeze(1)
        spread = (self.z.amax(1) - self.z.amin(1)) * LOG2E if len(self.rows) else self.lse_rows
        # a term of the sum: the exponential instruction (2^-23) and its
        # argument (a subtraction and a product of at most `spread`); the sum:
        # fewer joins than a tile's 64 and one per tile of 64 columns; the
        # logarithm to two steps; the addition of the maximum
        rel = 2 * U32 + 3 * U32 * spread + (64 + V / 64 + 1) * U32
        b = self.dz.amax(1) if len(self.rows) else self.lse_rows
        logs = (self.lse_rows - self.z.amax(1)).abs() if len(self.rows) else self.lse_rows
        b_lse = b + 1.01 * rel + 4 * U32 * logs + U32 * self.lse_rows.abs() + 1e-30
        zy = self.z.gather(1, at).squeeze(1)
        loss = self.lse_rows - zy
        b_loss = b_lse + self.dz.gather(1, at).squeeze(1) + U32 * loss.abs()
        out = []
        for v in (loss, self.lse_rows, b_loss, b_lse):
            x = torch.zeros(self.T, dtype=torch.float64)
            x[self.rows] = v
            out.append(x)
        return out

    def grads(self, lse, dloss, dlse, x_type, pieces=1):
        """dX, dW in 64 bits from the given lse (fp32), and their bounds before
        the last rounding."""
        k, r = abs(self.k), self.rows
        L = lse[r].double().unsqueeze(1)
        g = dloss[r].double().unsqueeze(1)
        gl = (dlse[r].double().unsqueeze(1) if dlse is not None else 0 * g)
        a = (dloss[r] + dlse[r]).double().unsqueeze(1) if dlse is not None else g
        p = torch.exp(self.z - L)
        G = a * p
        hot = torch.zeros_like(G)
        if len(r):
            hot[torch.arange(len(r)), self.y] = 1.0
        # p: the logit, lse / ln 2 and the fused product rounded, the
        # exponential to a step; the products with the coefficients (each divided
        # by the largest one: two roundings more) and their difference
        rel = self.dz + U32 * (2 * L.abs() + (self.z - L).abs()) * 1.01 + 8 * U32
        eG = (a * p).abs() * rel + 4 * U32 * g.abs() * hot
        G = G - g * hot
        eG = eG + U32 * gl.abs() * p  # dloss + dlse in fp32
        fi = torch.finfo(DT[x_type])
        gmax = float(torch.maximum(a.abs().max(), g.abs().max())) if len(r) else 0.0
        unit = 16384.0 if x_type == "f16" else 1.0
        # G in 16 bits relative to gmax / unit
        eG = eG * 1.01 + (G.abs() + eG) * (fi.eps / 2) + gmax / unit * fi.smallest_normal * fi.eps / 2
        G, eG = G * self.k, eG * k
        V, n = self.W.shape[0], len(r)
        dX, dW = G @ self.W, G.t() @ self.X
        SX, SW = (G.abs() + eG) @ self.W.abs(), (G.abs() + eG).t() @ self.X.abs()
        # fp32 sums, the pieces' and splits' among them, and the factor's three roundings
        bX = eG @ self.W.abs() + (V + 64 + 4) * U32 * SX
        bW = eG.t() @ self.X.abs() + (n + 4) * U32 * SW
        full = lambda v: torch.zeros(self.T, v.shape[1], dtype=torch.float64).index_copy_(0, r, v)
        return full(dX), dW, full(bX), bW


def far(got, ref, bound, dtype):
    """Largest excess of |got - ref| over its bound with one rounding to dtype
    (<= 0: within)."""
    got = got.double().cpu()
    assert bool(torch.isfinite(got).all()), "not finite"
    d = (got - ref).abs() - (bound + half_step(dtype, ref.abs() + bound))
    return float(d.max()) if d.numel() else 0.0
