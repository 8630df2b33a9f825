"""Grouped products (gemm_grouped_run) on the GPU against plain 64-bit
products, group by group, for every kernel family that takes the sizes."""
import os

import pytest
import torch

import moe_ref as R
from gpu_util import say
from sparse_tiled_gemm_amd import gemm as G

pytestmark = pytest.mark.gpu

FAMILIES = ["auto", "generic", "skinny", "tiled64", "tiled128", "tiled256"]


def _plan(algo, *a, **kw):
    """A plan of the family (through the tuning override), or a skip where it
    does not take the sizes."""
    if algo != "auto":
        os.environ["STGEMM_FORCE_KERNEL"] = algo
    try:
        plan = G.gemm_grouped_plan(G.make_grouped_desc(*a, **kw))
    finally:
        os.environ.pop("STGEMM_FORCE_KERNEL", None)
    if algo != "auto" and "_%s_" % algo not in plan.name:
        pytest.skip("%s does not take these sizes" % algo)
    return plan


def _mat(gen, rows, cols, dtype, ld=0, scale=1.0, off=0):
    ld = ld or cols
    buf = torch.full((rows * ld + 64,), float("nan"), dtype=R.DT[dtype], device="cuda")
    v = buf[off:off + rows * ld].view(rows, ld)
    v[:, :cols] = (torch.randn(rows, cols, generator=gen) * scale).to(R.DT[dtype])
    return v[:, :cols], buf


def _bounds(counts, lead=0):
    o = [lead]
    for c in counts:
        o.append(o[-1] + c)
    return o


# rows outside every group (before the first, after the last), empty groups,
# groups of one row, groups that end inside a tile
ROWS = [  # counts, lead, tail, N, K, dtype, d_type, ld extra, element offset
    ([1], 0, 0, 64, 64, "bf16", "bf16", 0, 0),
    ([0, 1, 0, 3], 0, 0, 1024, 2048, "bf16", "bf16", 0, 0),
    ([1, 1, 1, 1, 0], 0, 0, 96, 256, "f16", "f16", 0, 0),
    ([5, 0, 17, 16, 40, 0, 1], 2, 3, 200, 136, "f16", "f32", 0, 0),
    ([130, 0, 64, 300], 0, 0, 264, 1416, "bf16", "bf16", 8, 0),
    ([257, 256, 0, 1, 500], 1, 9, 520, 72, "f16", "f16", 0, 0),
    ([40, 25], 0, 0, 33, 45, "bf16", "f32", 3, 1),       # nothing aligned
    ([70, 3], 0, 0, 128, 8, "bf16", "bf16", 0, 0),
    ([3] * 70, 0, 0, 64, 128, "bf16", "bf16", 0, 0),     # more groups than lanes
    ([0, 0], 0, 5, 64, 64, "f16", "f16", 0, 0),
    ([33, 600], 0, 0, 776, 1032, "f16", "f32", 0, 0),
    ([4, 9], 0, 0, 64, 0, "bf16", "f32", 0, 0),          # an empty sum
]


@pytest.mark.parametrize("algo", FAMILIES)
@pytest.mark.parametrize("b_layout", ["col", "row"])
@pytest.mark.parametrize("case", ROWS)
def test_rows(case, b_layout, algo):
    counts, lead, tail, N, K, dtype, d_type, ldx, off = case
    say("rows", algo, b_layout, case)
    gen = torch.Generator().manual_seed(N + K)
    g = len(counts)
    offsets = _bounds(counts, lead)
    rows = offsets[-1] + tail
    bw, bh = (K, N) if b_layout == "col" else (N, K)
    plan = _plan(algo, "rows", rows, N, K, g, dtype, dtype, d_type, b_layout=b_layout,
                 lda=K + ldx, ldb=bw + ldx, ldd=N + ldx)
    A, _ = _mat(gen, rows, K, dtype, K + ldx, 1.0, off)
    B, _ = _mat(gen, g * bh, bw, dtype, bw + ldx, max(K, 1) ** -0.5, off)
    D, d_buf = _mat(gen, rows, N, d_type, N + ldx, 1.0, off)
    before = d_buf.clone()
    off_d = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    G.gemm_grouped_run(plan, A, B, None, off_d, None, D)
    torch.cuda.synchronize()
    got = D.cpu().double()
    refs = R.rows_ref(A.cpu(), B.cpu().reshape(g, bh, bw), offsets, b_layout)
    want = before.clone()
    wv = want[off:off + rows * (N + ldx)].view(rows, N + ldx)
    for a, ref, S in refs.values():
        n = len(ref)
        bound = R.half_step(d_type, ref) * 1.001 + (K + 2) * 2 * R.U32 * S
        assert ((got[a:a + n] - ref).abs() <= bound).all(), plan.name
        wv[a:a + n, :N] = D[a:a + n]
    it = torch.int32 if d_type == "f32" else torch.int16
    assert torch.equal(d_buf.view(it), want.view(it))  # nothing else is written


@pytest.mark.parametrize("counts,N", [([700, 1, 300, 0, 255], 264), ([512] * 8, 4096),
                                      ([256 * 16 + 3, 5000], 4100)])
def test_last_round(counts, N):
    """The 256 x 256 tiles past the last full round of compute units go in
    halves: fewer tiles than one round, exactly one, some more."""
    say("last round", counts, N)
    gen = torch.Generator().manual_seed(N)
    offsets, K = _bounds(counts), 72
    rows = offsets[-1]
    plan = _plan("tiled256", "rows", rows, N, K, len(counts), "bf16", "bf16", "f32")
    A, _ = _mat(gen, rows, K, "bf16")
    B, _ = _mat(gen, len(counts) * N, K, "bf16", 0, K ** -0.5)
    D = torch.full((rows, N), float("nan"), device="cuda")
    G.gemm_grouped_run(plan, A, B, None, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                       None, D)
    torch.cuda.synchronize()
    d = D.cpu()
    for a, ref, S in R.rows_ref(A.cpu(), B.cpu().reshape(len(counts), N, K), offsets,
                                "col").values():
        err = (d[a:a + len(ref)].double() - ref).abs()
        assert (err <= R.half_step("f32", ref) + (K + 2) * 2 * R.U32 * S).all()


@pytest.mark.parametrize("offsets", [[0, 40, 20, 60], [-7, 10, 1000, 64], [64, 64, 64, 0],
                                     [2 ** 31 - 1, -2 ** 31, 30, 2 ** 31 - 1]])
@pytest.mark.parametrize("algo", FAMILIES)
@pytest.mark.parametrize("mode", ["rows", "weights"])
def test_bounds_are_clamped(mode, offsets, algo):
    """Bounds outside 0 .. rows or descending: clamped, empty, never out of range."""
    gen = torch.Generator().manual_seed(1)
    rows, N, K = 64, 64, 128
    A, _ = _mat(gen, rows, K, "bf16")
    off_d = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    if mode == "rows":
        plan = _plan(algo, mode, rows, N, K, 3, "bf16", "bf16", "f32")
        B, _ = _mat(gen, 3 * N, K, "bf16", 0, K ** -0.5)
        D = torch.full((rows, N), 7.0, device="cuda")
        G.gemm_grouped_run(plan, A, B, None, off_d, None, D)
        torch.cuda.synchronize()
        got = D.cpu().double()
        refs = R.rows_ref(A.cpu(), B.cpu().reshape(3, N, K), offsets, "col")
        hit = torch.zeros(rows, dtype=torch.int32)
        for a, ref, _ in refs.values():
            hit[a:a + len(ref)] += 1
        for a, ref, S in refs.values():
            sel = hit[a:a + len(ref)] == 1  # rows of two groups hold either's product
            err = (got[a:a + len(ref)] - ref).abs()
            assert (err[sel] <= (K + 2) * 2 * R.U32 * S[sel] + R.half_step("f32", ref)[sel]).all()
        assert (got[hit == 0] == 7).all()
    else:
        plan = _plan(algo, mode, rows, N, K, 3, "bf16", "bf16", "f32")
        B, _ = _mat(gen, rows, N, "bf16")
        D = torch.empty(3, K, N, device="cuda")
        G.gemm_grouped_run(plan, A, B, None, off_d, None, D)
        torch.cuda.synchronize()
        ref, S = R.weights_ref(A.cpu(), B.cpu(), offsets)
        assert ((D.cpu().double() - ref).abs() <= (rows + 2) * 2 * R.U32 * S +
                R.half_step("f32", ref)).all()


WEIGHTS = [  # counts, lead, tail, K, N, dtype, d_type, C, eight, ld extra, element offset
    ([1], 0, 0, 64, 64, "bf16", "f32", False, False, 0, 0),
    ([0, 3, 0, 33], 0, 0, 128, 256, "bf16", "f32", True, False, 0, 0),
    ([100, 0, 31, 200], 5, 2, 264, 136, "f16", "f32", False, False, 8, 0),
    ([7, 64, 65], 0, 0, 300, 45, "f16", "bf16", True, False, 3, 1),     # nothing aligned
    ([513, 40], 0, 0, 520, 776, "bf16", "f32", True, False, 0, 0),
    ([96, 32], 0, 0, 256, 256, "f16", "f16", False, False, 0, 0),
    ([0, 3, 0, 33], 0, 0, 128, 256, "bf16", "f32", True, True, 0, 0),
    ([300, 0, 75], 1, 1, 264, 424, "f16", "f32", False, True, 0, 0),
    ([90, 20], 0, 0, 72, 45, "bf16", "f32", False, True, 0, 0),
    ([257, 255], 0, 0, 512, 512, "bf16", "bf16", True, True, 0, 0),
    ([2] * 66, 0, 0, 64, 64, "bf16", "f32", False, False, 0, 0),
]


@pytest.mark.parametrize("algo", FAMILIES)
@pytest.mark.parametrize("case", WEIGHTS)
def test_weights(case, algo):
    counts, lead, tail, K, N, dtype, d_type, has_c, eight, ldx, off = case
    say("weights", algo, case)
    gen = torch.Generator().manual_seed(N + K)
    g = len(counts)
    offsets = _bounds(counts, lead)
    rows = offsets[-1] + tail
    plan = _plan(algo, "weights", rows, N, K, g, dtype, "e4m3" if eight else dtype, d_type,
                 has_c=has_c, lda=K + ldx, ldb=0 if eight else N + ldx, ldd=N + ldx)
    A, _ = _mat(gen, rows, K, dtype, K + ldx, 1.0, off)
    Bf, _ = _mat(gen, rows, N, dtype, N + ldx, 1.0, off)
    B, scales, Bv = Bf, None, Bf.cpu()
    if eight:
        B = torch.empty(rows, N, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows, (N + 31) // 32, dtype=torch.uint8, device="cuda")
        G.gemm_q8_store(rows, N, dtype, Bf, N + ldx, B, scales)
        torch.cuda.synchronize()
        Bv = R.q8_load_ref(B.cpu(), scales.cpu(), dtype)
    D, d_buf = _mat(gen, g * K, N, d_type, N + ldx, 1.0, off)
    C, _ = _mat(gen, g * K, N, d_type, N + ldx, 1.0, off)
    before = d_buf.clone()
    off_d = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    G.gemm_grouped_run(plan, A, B, scales, off_d, C if has_c else None, D)
    torch.cuda.synchronize()
    c64 = C.cpu().reshape(g, K, N) if has_c else None
    ref, S = R.weights_ref(A.cpu(), Bv, offsets, c64)
    L = max(counts) + 2
    bound = R.half_step(d_type, ref) * 1.001 + L * 2 * R.U32 * S
    assert ((D.cpu().double().reshape(g, K, N) - ref).abs() <= bound).all(), plan.name
    want = before.clone()
    want[off:off + g * K * (N + ldx)].view(g * K, N + ldx)[:, :N] = D
    it = torch.int32 if d_type == "f32" else torch.int16
    assert torch.equal(d_buf.view(it), want.view(it))
    if has_c:  # in place: the same bits
        E, _ = _mat(gen, g * K, N, d_type, N + ldx, 1.0, off)
        E.copy_(C)
        G.gemm_grouped_run(plan, A, B, scales, off_d, E, E)
        torch.cuda.synchronize()
        assert torch.equal(E, D)


@pytest.mark.parametrize("algo", FAMILIES)
def test_rows_of_other_groups_do_not_leak(algo):
    """NaN and infinity in one group's rows, in its weights and past K stay there."""
    gen = torch.Generator().manual_seed(4)
    N, K, lda = 72, 104, 112
    offsets = [0, 20, 41, 75]
    plan = _plan(algo, "rows", 75, N, K, 3, "bf16", "bf16", "f32", lda=lda, ldb=lda)
    A, _ = _mat(gen, 75, K, "bf16", lda)   # NaN past K
    B, _ = _mat(gen, 3 * N, K, "bf16", lda, K ** -0.5)
    A[25] = float("nan")
    A[30, 7] = float("inf")
    B[N + 5] = float("nan")
    D = torch.empty(75, N, device="cuda")
    G.gemm_grouped_run(plan, A, B, None, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                       None, D)
    torch.cuda.synchronize()
    d = D.cpu()
    assert torch.isfinite(d[:20]).all() and torch.isfinite(d[41:]).all()
    assert torch.isnan(d[25]).all() and torch.isnan(d[20:41, 5]).all()
    ok = [r for r in range(20, 41) if r not in (25, 30)]
    assert torch.isfinite(d[ok][:, [c for c in range(N) if c != 5]]).all()


@pytest.mark.parametrize("algo", FAMILIES)
@pytest.mark.parametrize("eight", [False, True])
def test_weights_of_other_groups_do_not_leak(algo, eight):
    gen = torch.Generator().manual_seed(4)
    N, K = 136, 72
    offsets = [0, 20, 41, 75]
    plan = _plan(algo, "weights", 80, N, K, 3, "f16", "e4m3" if eight else "f16", "f32")
    A, _ = _mat(gen, 80, K, "f16")
    Bf, _ = _mat(gen, 80, N, "f16")
    A[25] = float("nan")
    Bf[26, 3] = float("inf")
    A[77], Bf[78] = float("nan"), float("nan")  # rows of no group
    B, scales = Bf, None
    if eight:
        B = torch.empty(80, N, dtype=torch.uint8, device="cuda")
        scales = torch.empty(80, (N + 31) // 32, dtype=torch.uint8, device="cuda")
        G.gemm_q8_store(80, N, "f16", Bf, 0, B, scales)
    D = torch.empty(3, K, N, device="cuda")
    G.gemm_grouped_run(plan, A, B, scales, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                       None, D)
    torch.cuda.synchronize()
    d = D.cpu()
    assert torch.isfinite(d[0]).all() and torch.isfinite(d[2]).all() and torch.isnan(d[1]).all()


@pytest.mark.parametrize("algo", ["skinny", "tiled128", "tiled256"])
def test_forced_algorithms(algo):
    """The descriptor's algo code picks the family too, or is refused."""
    d = lambda mode, K=64: G.make_grouped_desc(mode, 64, 64, K, 4, "bf16", "bf16", "bf16", algo=algo)
    assert algo in G.gemm_grouped_plan(d("rows")).name
    with pytest.raises(G.GemmError):
        G.gemm_grouped_plan(d("rows", 65))  # rows of A not in whole 16 bytes
    if algo == "skinny":
        with pytest.raises(G.GemmError):
            G.gemm_grouped_plan(d("weights"))
    else:
        assert algo in G.gemm_grouped_plan(d("weights")).name


def _far(gen, rows, cols, ld, off=8):
    """rows x cols of a matrix of several GiB, NaN beside them."""
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    v = buf.view(rows, ld)
    v[:, :off + cols + 256] = float("nan")
    v[:, off:off + cols] = torch.randn(rows, cols, generator=gen).bfloat16()
    return v[:, off:off + cols]


@pytest.mark.parametrize("algo", FAMILIES)
def test_offsets_past_32_bits(algo):
    """Operands of 4.8 GB each: a group's last K rows lie past 2^32 bytes of
    its first, and its rows past 2^32 bytes of the operand's."""
    say("far", algo)
    gen = torch.Generator().manual_seed(9)
    rows, ld, offsets = 2400, 1000000, [0, 3, 2397]
    off_d = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    A, B = _far(gen, rows, 72, ld), _far(gen, rows, 136, ld)
    if algo != "skinny":
        plan = _plan(algo, "weights", rows, 136, 72, 2, "bf16", "bf16", "f32", lda=ld, ldb=ld)
        D = torch.empty(2, 72, 136, device="cuda")
        G.gemm_grouped_run(plan, A, B, None, off_d, None, D)
        torch.cuda.synchronize()
        ref, S = R.weights_ref(A.cpu(), B.cpu(), offsets)
        bound = R.half_step("f32", ref) * 1.001 + rows * 2 * R.U32 * S
        assert ((D.cpu().double() - ref).abs() <= bound).all(), plan.name
    # rows: B is one group's 2400 x 136 (row-major), A's rows a pitch of ld apart
    offsets = [3, 2397]
    X = A[:, :72]
    W = torch.randn(136, 72, generator=gen).bfloat16()
    plan = _plan(algo, "rows", rows, 136, 72, 1, "bf16", "bf16", "f32", lda=ld)
    D = torch.zeros(rows, 136, device="cuda")
    off_d = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    G.gemm_grouped_run(plan, X, W.cuda(), None, off_d, None, D)
    torch.cuda.synchronize()
    _, ref, S = R.rows_ref(X.cpu(), W[None], offsets, "col")[0]
    bound = R.half_step("f32", ref) * 1.001 + 74 * 2 * R.U32 * S
    assert ((D.cpu()[3:2397].double() - ref).abs() <= bound).all(), plan.name
    Y = torch.randn(40, rows, generator=gen).bfloat16()
    plan = _plan(algo, "rows", 40, 136, rows, 1, "bf16", "bf16", "f32", b_layout="row", ldb=ld)
    D = torch.zeros(40, 136, device="cuda")
    off_d = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    G.gemm_grouped_run(plan, Y.cuda(), B, None, off_d, None, D)
    torch.cuda.synchronize()
    _, ref, S = R.rows_ref(Y, B.cpu()[None], [0, 40], "row")[0]
    bound = R.half_step("f32", ref) * 1.001 + (rows + 2) * 2 * R.U32 * S
    assert ((D.cpu().double() - ref).abs() <= bound).all(), plan.name


@pytest.mark.parametrize("algo", ["auto", "tiled64", "tiled128", "tiled256"])
def test_codes_past_32_bits(algo):
    """4.4 GB of 8-bit codes: the first and last columns of the product."""
    say("far codes", algo)
    gen = torch.Generator().manual_seed(10)
    dgen = torch.Generator(device="cuda").manual_seed(10)
    rows, N, K, offsets = 4400, 1000000, 8, [0, 4400]
    plan = _plan(algo, "weights", rows, N, K, 1, "bf16", "e4m3", "f32")
    A = torch.randn(rows, K, generator=gen).bfloat16()
    B = torch.randint(0, 0x78, (rows, N), generator=dgen, dtype=torch.uint8, device="cuda")
    scales = torch.randint(118, 128, (rows, N // 32), generator=dgen, dtype=torch.uint8,
                           device="cuda")
    D = torch.empty(1, K, N, device="cuda")
    off_d = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    G.gemm_grouped_run(plan, A.cuda(), B, scales, off_d, None, D)
    torch.cuda.synchronize()
    for c in (0, N - 192):
        Bv = R.q8_load_ref(B[:, c:c + 192].cpu(), scales[:, c // 32:c // 32 + 6].cpu(), "bf16")
        ref, S = R.weights_ref(A, Bv, offsets)
        bound = R.half_step("f32", ref) * 1.001 + rows * 2 * R.U32 * S
        assert ((D[:, :, c:c + 192].cpu().double() - ref).abs() <= bound).all(), plan.name


EIGHT = ["auto", "generic", "tiled64", "tiled128", "tiled256"]


@pytest.mark.parametrize("algo", EIGHT)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_code_and_scale_of_an_8_bit_operand(dtype, algo):
    """Each value enters as the one gemm_q8_load gives: groups of one row and
    a single 1 in A leave it as it is."""
    say("codes", dtype, algo)
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8)
    K = 8
    A = torch.zeros(256, K, dtype=R.DT[dtype])
    A[:, 0] = 1
    plan = _plan(algo, "weights", 256, 256, K, 256, dtype, "e4m3", "f32")
    D = torch.full((256, K, 256), 5.0, device="cuda")
    off_d = torch.arange(257, dtype=torch.int32, device="cuda")
    G.gemm_grouped_run(plan, A.cuda(), codes.cuda(), scales.cuda(), off_d, None, D)
    torch.cuda.synchronize()
    want = R.q8_load_ref(codes, scales, dtype).float()
    got = D.cpu()[:, 0]
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan]), plan.name


@pytest.mark.parametrize("algo", EIGHT)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_code_in_every_row_of_a_tile(dtype, algo):
    """The same for one group of all rows and an identity for A (no NaN codes,
    which would reach every row)."""
    say("codes by row", dtype, algo)
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    codes[codes & 0x7F == 0x7F] = 0
    scales = torch.arange(256, dtype=torch.uint8).clamp(max=254).view(256, 1).repeat(1, 8)
    plan = _plan(algo, "weights", 256, 256, 256, 1, dtype, "e4m3", "f32")
    D = torch.full((256, 256), 5.0, device="cuda")
    off_d = torch.tensor([0, 256], dtype=torch.int32, device="cuda")
    G.gemm_grouped_run(plan, torch.eye(256, dtype=R.DT[dtype]).cuda(), codes.cuda(), scales.cuda(),
                       off_d, None, D)
    torch.cuda.synchronize()
    assert torch.equal(D.cpu(), R.q8_load_ref(codes, scales, dtype).float()), plan.name
