"""8-bit checkpoints and the gated activation that keeps and uses them, on
the GPU, against plain 64-bit references (tests/moe_ref.py)."""
import numpy as np
import pytest
import torch

import moe_ref as R
from gpu_util import say
from sparse_tiled_gemm_amd import gemm as G

pytestmark = pytest.mark.gpu


def _store(X):
    rows, cols = X.shape
    dt = "f16" if X.dtype == torch.float16 else "bf16"
    codes = torch.full((rows, cols), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, (cols + 31) // 32), 0x5A, dtype=torch.uint8, device="cuda")
    G.gemm_q8_store(rows, cols, dt, X.cuda(), 0, codes, scales)
    torch.cuda.synchronize()
    return codes.cpu(), scales.cpu()


def _check_codes(codes, scales, X):
    rc, rs = R.q8_ref(X)
    assert torch.equal(scales, rs)
    nan = ~torch.isfinite(X)
    assert ((codes[nan] & 0x7F) == 0x7F).all()
    assert torch.equal(codes[~nan], rc[~nan])


def _load(codes, scales, dtype):
    out = torch.full(codes.shape, 3.0, dtype=R.DT[dtype], device="cuda")
    G.gemm_q8_load(codes.shape[0], codes.shape[1], dtype, codes.cuda(), scales.cuda(), out, 0)
    torch.cuda.synchronize()
    return out.cpu()


def _same(got, want):
    """Bit-equal except for which NaN."""
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan].view(torch.int16), want[~nan].view(torch.int16))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 64), (7, 127),
                                       (130, 200), (33, 1027), (4, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_store_load(rows, cols, dtype):
    say("store/load", rows, cols, dtype)
    gen = torch.Generator().manual_seed(rows + cols)
    X = (torch.randn(rows, cols, generator=gen) *
         torch.exp(3 * torch.randn(rows, 1, generator=gen))).to(R.DT[dtype])
    X[0, 0] = 0.0
    codes, scales = _store(X)
    _check_codes(codes, scales, X)
    back = _load(codes, scales, dtype)
    _same(back, R.q8_load_ref(codes, scales, dtype))
    # 4 significant bits, down to 2^-9 of the block's scale
    err = (back.double() - X.double()).abs()
    s = R.pow2(scales.int() - 127).repeat_interleave(32, 1)[:, :cols]
    assert (err <= X.double().abs() * 2.0 ** -4 + s * 2.0 ** -10 +
            R.half_step(dtype, X.double())).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_bit_pattern(dtype):
    """All 65536 values of the type, among them NaN, infinities and
    subnormals, in blocks of neighbours and in shuffled blocks."""
    bits = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16).copy())
    perm = torch.randperm(65536, generator=torch.Generator().manual_seed(1))
    for b in (bits, bits[perm]):
        X = b.view(R.DT[dtype]).view(64, 1024)
        codes, scales = _store(X)
        _check_codes(codes, scales, X)
        _same(_load(codes, scales, dtype), R.q8_load_ref(codes, scales, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_load_every_code_and_scale(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8)
    _same(_load(codes, scales, dtype), R.q8_load_ref(codes, scales, dtype))


def test_block_borders():
    """The scale steps exactly above 448 * 2^e."""
    vals = [448.0, 450.0, 224.0, 225.0, 1.75, 1.7578125, 2.0, 7.0, 0.0, -448.0, -450.0]
    X = torch.zeros(len(vals), 32)
    X[:, 5] = torch.tensor(vals)
    X = X.bfloat16()
    codes, scales = _store(X)
    _check_codes(codes, scales, X)
    assert scales[:, 0].tolist() == [127, 128, 126, 127, 119, 120, 120, 121, 127, 127, 128]


def _gu(gen, rows, cols, dtype, ld, off=0):
    buf = torch.full((rows * ld + 64,), 7.5, dtype=R.DT[dtype], device="cuda")
    v = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
    v.copy_((torch.randn(rows, cols, generator=gen) * 2).to(R.DT[dtype]))
    return v, buf


@pytest.mark.parametrize("rows,cols,ldx,off", [
    (1, 1, 0, 0), (1, 16, 0, 0), (3, 8, 0, 1), (2, 32, 8, 0), (9, 100, 0, 0), (17, 515, 3, 1),
    (300, 1416, 0, 0), (5, 2048, 0, 0), (1, 8200, 0, 0), (600, 48, 0, 0), (64, 1027, 0, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_swiglu_and_backward(rows, cols, ldx, off, dtype):
    say("swiglu", rows, cols, ldx, off, dtype)
    gen = torch.Generator().manual_seed(rows * 3 + cols)
    ldg, ldh = 2 * cols + ldx, cols + ldx
    GU, _ = _gu(gen, rows, 2 * cols, dtype, ldg, off)
    H, h_buf = _gu(gen, rows, cols, dtype, ldh, off)
    hb = h_buf.clone()
    codes = torch.full((rows, 2 * cols), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, (2 * cols + 31) // 32), 0x5A, dtype=torch.uint8, device="cuda")
    G.gemm_swiglu(rows, cols, dtype, GU, ldg, H, ldh, codes, scales)
    torch.cuda.synchronize()
    gu = GU.cpu()
    _check_codes(codes.cpu(), scales.cpu(), gu)
    ref, e32 = R.swiglu_ref(gu[:, :cols].double(), gu[:, cols:].double())
    err = (H.cpu().double() - ref).abs()
    assert (err <= R.half_step(dtype, ref) * 1.001 + e32).all()
    hb[off:off + rows * ldh].view(rows, ldh)[:, :cols] = H
    assert torch.equal(h_buf.view(torch.int16), hb.view(torch.int16))
    # without a checkpoint: the same H
    H2 = torch.empty(rows, cols, dtype=R.DT[dtype], device="cuda")
    G.gemm_swiglu(rows, cols, dtype, GU, ldg, H2, 0)
    assert torch.equal(H2, H)

    dH, _ = _gu(gen, rows, cols, dtype, ldh, off)
    dGU, d_buf = _gu(gen, rows, 2 * cols, dtype, ldg, off)
    db = d_buf.clone()
    H3 = torch.empty(rows, cols, dtype=R.DT[dtype], device="cuda")
    G.gemm_swiglu_backward(rows, cols, dtype, codes, scales, dH, ldh, dGU, ldg, H3, 0)
    torch.cuda.synchronize()
    v = R.q8_values(codes.cpu(), scales.cpu())
    refs, bounds = R.swiglu_backward_ref(v[:, :cols], v[:, cols:], dH.cpu().double())
    d = dGU.cpu().double()
    for got, want, b in zip((d[:, :cols], d[:, cols:], H3.cpu().double()), refs, bounds):
        assert ((got - want).abs() <= R.half_step(dtype, want) * 1.001 + b).all()
    db[off:off + rows * ldg].view(rows, ldg)[:, :2 * cols] = dGU
    assert torch.equal(d_buf.view(torch.int16), db.view(torch.int16))
    # without H
    dGU2 = torch.empty(rows, 2 * cols, dtype=R.DT[dtype], device="cuda")
    G.gemm_swiglu_backward(rows, cols, dtype, codes, scales, dH, ldh, dGU2, 0)
    assert torch.equal(dGU2, dGU)


def test_swiglu_far_values():
    """Gates far from zero: no overflow on the way, the limits on either side."""
    g = torch.tensor([-1e30, -3e4, -200.0, -100.0, -90.0, -88.0, -20.0, 0.0, 20.0, 89.0, 200.0, 3e38,
                      float("inf"), float("nan"), -0.0, 1e-30]).bfloat16()
    u = torch.ones(16).bfloat16()
    H = torch.empty(1, 16, dtype=torch.bfloat16, device="cuda")
    G.gemm_swiglu(1, 16, "bf16", torch.cat([g, u]).view(1, 32).cuda(), 0, H, 0)
    h = H.cpu().double().view(-1)
    ref, e32 = R.swiglu_ref(g.double(), u.double())
    fin = torch.isfinite(ref)
    assert ((h - ref).abs()[fin] <= (R.half_step("bf16", ref) * 1.001 + e32)[fin]).all()
    assert h[12] == float("inf") and torch.isnan(h[13])


def test_backward_against_differences():
    """dG and dU against differences of H at the kept values, in 64 bits."""
    gen = torch.Generator().manual_seed(2)
    rows, cols = 6, 40
    X = (torch.randn(rows, 2 * cols, generator=gen) * 2).half()
    codes, scales = _store(X)
    v = R.q8_values(codes, scales)
    g, u = v[:, :cols], v[:, cols:]
    dH = torch.randn(rows, cols, generator=gen).half()
    dGU = torch.empty(rows, 2 * cols, dtype=torch.float16, device="cuda")
    G.gemm_swiglu_backward(rows, cols, "f16", codes.cuda(), scales.cuda(), dH.cuda(), 0, dGU, 0)
    got = dGU.cpu().double()
    h = 1e-5
    f = lambda g_, u_: R.swiglu_ref(g_, u_)[0] * dH.double()
    dg = (f(g + h, u) - f(g - h, u)) / (2 * h)
    du = (f(g, u + h) - f(g, u - h)) / (2 * h)
    # differences: h^2 times the third derivative (below 1 for these), and 64-bit noise
    tol = lambda x: R.half_step("f16", x) * 1.01 + 1e-6 * (1 + (u * dH.double()).abs())
    assert ((got[:, :cols] - dg).abs() <= tol(dg)).all()
    assert ((got[:, cols:] - du).abs() <= tol(du)).all()


def _backward(GU, dH, dtype):
    """Codes of GU, the clamped values they stand for, and dG, dU, H (64 bits, CPU)."""
    rows, cols = dH.shape
    codes, scales = _store(GU)
    dGU = torch.empty(rows, 2 * cols, dtype=R.DT[dtype], device="cuda")
    H = torch.empty(rows, cols, dtype=R.DT[dtype], device="cuda")
    G.gemm_swiglu_backward(rows, cols, dtype, codes.cuda(), scales.cuda(), dH.cuda(), 0, dGU, 0, H, 0)
    torch.cuda.synchronize()
    v = R.q8_load_ref(codes, scales, dtype).double()
    d = dGU.cpu().double()
    return v[:, :cols], v[:, cols:], (d[:, :cols], d[:, cols:], H.cpu().double())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_backward_at_the_end_of_the_range(dtype):
    """Finite inputs whose code times its scale lies past the type's range
    (bfloat16: past fp32's as well) enter as the type's largest value."""
    big = torch.finfo(R.DT[dtype]).max
    pairs = [(big, 0.5), (big, -0.25), (0.97 * big, 0.5), (-big, 2.0), (1.0, big), (-2.0, big),
             (-2.0, -0.98 * big), (0.0, big), (0.0, -big)]
    cols = 64
    X = torch.tensor(pairs).repeat_interleave(cols, 1).to(R.DT[dtype])  # a value per block
    dH = torch.full((len(pairs), cols), 2.0 ** -10).to(R.DT[dtype])
    g, u, got = _backward(X, dH, dtype)
    refs, bounds = R.swiglu_backward_ref(g, u, dH.double())
    for x, want, b in zip(got, refs, bounds):
        # far gates: sigmoid is 0 or 1 to the last bit, and each result is at
        # most four fp32 roundings of its products away
        b = torch.where(g.abs() > 100, 4 * R.U32 * want.abs(), b)
        assert torch.isfinite(x).all()
        assert ((x - want).abs() <= R.half_step(dtype, want) * 1.001 + b).all()


def test_backward_products_that_overflow_on_the_way():
    """dH * u past fp32's range where the gate brings dG back into it."""
    cols = 32
    cases = [  # g, u, dH
        (-200.0, 1e35, 1e5), (-200.0, -1e35, 1e5), (-40.0, 1e20, 1e20), (-30.0, 1e24, -1e22),
        (-30.0, 1e22, 1e24), (-3e38, 1e30, 1e30), (-20.0, 3e38, 30.0)]
    t = torch.tensor(cases).bfloat16()
    X = t[:, :2].repeat_interleave(cols, 1)
    dH = t[:, 2:].repeat_interleave(cols, 1)
    g, u, (dg, du, h) = _backward(X, dH, "bf16")
    (rg, _, _), (bg, _, _) = R.swiglu_backward_ref(g, u, dH.double())
    bg = torch.where(g < -100, torch.zeros_like(bg), bg)  # the gate is zero
    rg = torch.where(g < -100, torch.zeros_like(rg), rg)
    assert (rg.abs() < torch.finfo(torch.bfloat16).max).all()
    assert ((dg - rg).abs() <= R.half_step("bf16", rg) * 1.001 + bg).all()
    # and past the type's range where it does not
    X = torch.tensor([[50.0, -1e20]]).bfloat16().repeat_interleave(cols, 1)
    _, _, (dg, _, _) = _backward(X, torch.full((1, cols), 1e20).bfloat16(), "bf16")
    assert (dg == -float("inf")).all()
