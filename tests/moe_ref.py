"""Plain 64-bit references (on the CPU) of the mixture-of-experts operators,
and the error bounds their tests use.

A rounding to a type is off by at most half a step: eps/2 relative, and half
the smallest subnormal below the normal range.  A sum of n products in fp32
is off by at most n roundings of the sum of magnitudes, whatever its order."""
import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24


def half_step(dtype, ref):
    """Bound of one rounding to `dtype` at values ref."""
    fi = torch.finfo(DT[dtype])
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def sort_ref(ids, groups):
    """offsets, order, pos of ids (any integer array), straight from the definition."""
    flat = np.asarray(ids).reshape(-1)
    slots = [(int(g), s) for s, g in enumerate(flat) if 0 <= g < groups]
    slots.sort()
    offsets = np.zeros(groups + 1, np.int32)
    for g, _ in slots:
        offsets[g + 1] += 1
    offsets = np.cumsum(offsets).astype(np.int32)
    order = np.full(len(flat), -1, np.int32)
    pos = np.full(len(flat), -1, np.int32)
    for p, (_, s) in enumerate(slots):
        order[p], pos[s] = s, p
    return offsets, order, pos


def combine_ref(pos, weights, Ys):
    """Y and the sum of magnitudes, 64 bits."""
    T, K = pos.shape
    Y = torch.zeros(T, Ys.shape[1], dtype=torch.float64)
    S = torch.zeros_like(Y)
    for t in range(T):
        for k in range(K):
            p = int(pos[t, k])
            if 0 <= p < len(Ys):
                w = 1.0 if weights is None else float(weights[t, k])
                Y[t] += w * Ys[p].double()
                S[t] += abs(w) * Ys[p].double().abs()
    return Y, S


def bounds_of(offsets, rows):
    """Clamped (begin, end) of each group."""
    o = [min(max(int(x), 0), rows) for x in offsets]
    return [(a, max(a, b)) for a, b in zip(o, o[1:])]


def rows_ref(A, B, offsets, b_layout):
    """{group: (first row, D, sum of magnitudes)} of the rows' product, 64 bits."""
    out = {}
    for g, (a, b) in enumerate(bounds_of(offsets, len(A))):
        if a < b:
            w = B[g].double().t() if b_layout == "col" else B[g].double()
            x = A[a:b].double()
            out[g] = (a, x @ w, x.abs() @ w.abs())
    return out


def weights_ref(A, B, offsets, C=None):
    G = len(offsets) - 1
    D = torch.zeros(G, A.shape[1], B.shape[1], dtype=torch.float64)
    S = torch.zeros_like(D)
    for g, (a, b) in enumerate(bounds_of(offsets, len(A))):
        D[g] = A[a:b].double().t() @ B[a:b].double()
        S[g] = A[a:b].double().abs().t() @ B[a:b].double().abs()
        if C is not None:
            D[g] += C[g].double()
            S[g] += C[g].double().abs()
    return D, S


def pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)


def q8_ref(X):
    """Codes and scales of a 16-bit tensor, by the definition."""
    rows, cols = X.shape
    nb = (cols + 31) // 32
    x = torch.zeros(rows, nb * 32, dtype=torch.float64)
    x[:, :cols] = X.double()
    x = x.view(rows, nb, 32)
    fin = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs()
    amax = fin.amax(2)
    e = torch.full((rows, nb), -127, dtype=torch.int32)
    for _ in range(256):  # the smallest e that fits, found by counting up
        small = amax > 448.0 * pow2(e)
        if not small.any():
            break
        e = torch.where(small, e + 1, e)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    q = torch.where(torch.isfinite(x), x * pow2(-e).unsqueeze(2), torch.full_like(x, float("nan")))
    codes = e4m3_codes(q).view(rows, nb * 32)[:, :cols].contiguous()
    return codes, (e + 127).to(torch.uint8)


def e4m3_values():
    """The 256 values of E4M3, from its fields."""
    v = torch.zeros(256, dtype=torch.float64)
    for c in range(256):
        s, ex, m = c >> 7, (c >> 3) & 15, c & 7
        x = float("nan") if ex == 15 and m == 7 else (m / 8 * 2.0 ** -6 if ex == 0
                                                      else (1 + m / 8) * 2.0 ** (ex - 7))
        v[c] = -x if s else x
    return v


def e4m3_codes(q):
    """Nearest E4M3 code (ties to even) of |q| <= 448; 0x7F for NaN (any sign)."""
    vals = e4m3_values()[:127]  # +0 .. 448, ascending
    a = q.abs()
    hi = torch.searchsorted(vals, a.contiguous()).clamp(0, 126)
    lo = (hi - 1).clamp(min=0)
    dh, dl = (vals[hi] - a).abs(), (a - vals[lo]).abs()
    c = torch.where(dh < dl, hi, lo)
    c = torch.where(dh == dl, torch.where(hi % 2 == 0, hi, lo), c)
    c = torch.where(torch.signbit(q), c + 128, c)
    return torch.where(torch.isnan(q), torch.full_like(c, 0x7F), c).to(torch.uint8)


def q8_values(codes, scales):
    """The values that codes and scales stand for, 64 bits."""
    cols = codes.shape[1]
    s = pow2(scales.int() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return e4m3_values()[codes.long()] * s.repeat_interleave(32, 1)[:, :cols]


def q8_load_ref(codes, scales, dtype):
    big = torch.finfo(DT[dtype]).max
    v = q8_values(codes, scales)
    return v.clamp(-big, big).to(DT[dtype])  # exact or one rounding (codes hold 4 bits)


def swiglu_ref(g, u):
    """H in 64 bits, and its relative bound before the last rounding: the
    exponential's argument is rounded once (|g| steps of its value), and
    sigmoid and products add a few more."""
    h = g * torch.sigmoid(g) * u
    return h, h.abs() * (g.abs() + 16) * U32


def swiglu_backward_ref(g, u, dh):
    s = torch.sigmoid(g)
    dg, du, h = dh * u * (s + g * s * (1 - s)), dh * g * s, g * s * u
    rel = (g.abs() + 16) * U32
    # 1 + g (1 - s) may cancel: its error counts against its terms
    return (dg, du, h), ((dh * u * s).abs() * (1 + g.abs()) * 2 * rel, du.abs() * rel, h.abs() * rel)
