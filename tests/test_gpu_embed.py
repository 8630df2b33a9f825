"""Embedding lookup and its gradient (gemm_embed, gemm_embed_backward) against
64-bit references: types, odd sizes, strides, ids out of range, repeated ids
from none to all, on either side of the border between the single launch and
the sort."""
import pytest
import torch

from gpu_util import say
from moe_ref import DT
from sparse_tiled_gemm_amd import gemm as G
from vocab_ref import embed_grad_ref, embed_ref, far, valid

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]


def ids_of(tokens, vocab, kind, seed=0):
    gen = torch.Generator().manual_seed(seed)
    if kind == "one":       # all tokens the same
        return torch.full((tokens,), vocab // 2, dtype=torch.int64)
    if kind == "none":      # no token names a row
        return torch.where(torch.arange(tokens) % 2 == 0, -1, vocab)
    if kind == "ends":      # the first and the last row
        return torch.where(torch.rand(tokens, generator=gen) < 0.5, 0, vocab - 1)
    r = torch.rand(tokens, generator=gen, dtype=torch.float64)
    ids = (vocab * r ** 4).long().clamp(max=vocab - 1)  # many of the first rows
    if kind == "hot":
        ids[torch.rand(tokens, generator=gen) < 0.5] = vocab - 2 if vocab > 1 else 0
    if kind != "all":
        ids[torch.rand(tokens, generator=gen) < 0.1] = -100
        ids[torch.rand(tokens, generator=gen) < 0.05] = (1 << 40) + 1
    return ids


def dev_ids(ids, id_bytes):
    if id_bytes == 8:
        return ids.cuda()
    return ids.clamp(-(1 << 31), (1 << 31) - 1).to(torch.int32).cuda()


def strided(x, ld, fill):
    """x's rows ld elements apart in a buffer of `fill`, and the buffer."""
    buf = torch.full((max(len(x), 1) * ld + 8,), fill, dtype=x.dtype, device="cuda")
    view = buf.as_strided((len(x), x.shape[1]), (ld, 1))
    view.copy_(x)
    return view, buf


@pytest.mark.parametrize("e", TYPES)
@pytest.mark.parametrize("y", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols,pad,id_bytes", [
    (1, 100, 64, 0, 8), (7, 33, 1, 0, 4), (130, 1000, 130, 0, 8), (65, 17, 1027, 5, 4),
    (300, 2000, 512, 8, 8), (3, 1, 8, 1, 8)])
def test_lookup(e, y, tokens, vocab, cols, pad, id_bytes):
    say("lookup", e, y, tokens, vocab, cols, pad)
    gen = torch.Generator().manual_seed(1)
    E = torch.randn(vocab, cols, generator=gen).to(DT[e])
    ids = ids_of(tokens, vocab, "some")
    scale = 1.7
    Ed, _ = strided(E, cols + pad, 3.0)
    Y, buf = strided(torch.zeros(tokens, cols, dtype=DT[y]), cols + 2 * pad, 7.0)
    before = buf.clone()
    G.gemm_embed(tokens, vocab, cols, e, y, dev_ids(ids, id_bytes), Ed, cols + pad, Y, cols + 2 * pad,
                 scale=scale, id_bytes=id_bytes)
    ref = embed_ref(ids, E, scale)
    assert far(Y, ref, ref.abs() * 2.0 ** -24, y) <= 0
    assert bool((Y[~valid(ids, vocab).cuda()] == 0).all())
    # between the rows and behind the last nothing is written
    before.as_strided((tokens, cols), (cols + 2 * pad, 1)).copy_(Y)
    assert torch.equal(before, buf)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_lookup_copies_bits(dtype):
    """scale 1 and one type: the values themselves, the type's ends among them."""
    fi = torch.finfo(DT[dtype])
    E = torch.tensor([[fi.max, -fi.max, fi.smallest_normal, 0.0, 1.0, -fi.eps, float("inf"),
                       -float("inf"), 2.0, 3.0]], dtype=DT[dtype])
    Y = torch.empty(2, 10, dtype=DT[dtype], device="cuda")
    G.gemm_embed(2, 1, 10, dtype, dtype, torch.zeros(2, dtype=torch.int32, device="cuda"), E.cuda(), 0,
                 Y, 0)
    assert torch.equal(Y.cpu(), E.expand(2, 10))


@pytest.mark.parametrize("kind", ["some", "all", "hot", "one", "none", "ends"])
@pytest.mark.parametrize("tokens", [0, 1, 33, 1000, 1024, 1025, 5000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(kind, tokens, accumulate):
    run_gradient(kind, tokens, 777, 200, "bf16", "f32", accumulate, 8, 0, 0.5)


@pytest.mark.parametrize("y", TYPES)
@pytest.mark.parametrize("e", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols,pad", [(600, 300, 72, 3), (3000, 300, 72, 3)])
def test_gradient_types(y, e, tokens, vocab, cols, pad):
    run_gradient("hot", tokens, vocab, cols, y, e, False, 4, pad, 2.0)
    run_gradient("hot", tokens, vocab, cols, y, e, True, 4, pad, 2.0)


@pytest.mark.parametrize("kind", ["some", "hot"])
@pytest.mark.parametrize("tokens", [1024, 1025, 2048, 2049])
@pytest.mark.parametrize("cols", [512, 520, 1030, 2048, 2056])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_by_search_or_sort(kind, tokens, cols, accumulate):
    run_gradient(kind, tokens, 300, cols, "bf16", "bf16", accumulate, 8, 0, 0.5)


@pytest.mark.parametrize("tokens,vocab,cols,kind", [
    (2000, 1, 8, "one"), (2000, 2, 513, "all"), (1500, 3, 1, "all"), (40000, 65537, 24, "hot"),
    (70000, 1000, 40, "some"), (1100, 1 << 20, 8, "some"), (20000, 131072, 16, "ends"),
    (300000, 50021, 8, "hot"), (2000, 500, 1027, "hot"), (40000, 70000, 8, "one")])
def test_gradient_sizes(tokens, vocab, cols, kind):
    run_gradient(kind, tokens, vocab, cols, "f16", "f32", False, 8, 0, 1.0)


def run_gradient(kind, tokens, vocab, cols, y, e, accumulate, id_bytes, pad, scale):
    say("gradient", kind, tokens, vocab, cols, y, e, accumulate)
    gen = torch.Generator().manual_seed(2)
    dY = torch.randn(tokens, cols, generator=gen).to(DT[y])
    ids = ids_of(tokens, vocab, kind)
    D0 = torch.randn(vocab, cols, generator=gen).to(DT[e])
    dYd, _ = strided(dY, cols + pad, 3.0)
    D, buf = strided(D0 if accumulate else torch.full_like(D0, float("nan")), cols + 2 * pad, 7.0)
    before = buf.clone()
    ws = torch.full((G.gemm_embed_workspace(tokens, vocab, cols) + 16,), 0xA5, dtype=torch.uint8,
                    device="cuda")
    args = (tokens, vocab, cols, y, e, dev_ids(ids, id_bytes), dYd, cols + pad, D, cols + 2 * pad, ws)
    G.gemm_embed_backward(*args, scale=scale, accumulate=accumulate, id_bytes=id_bytes)
    torch.cuda.synchronize()
    ref, bound, named = embed_grad_ref(ids, dY, vocab, scale, D0 if accumulate else None)
    assert far(D, ref, bound, e) <= 0
    if accumulate:  # rows that no token names keep their bits
        assert torch.equal(D.cpu()[~named], D0[~named])
    assert bool((ws[-16:] == 0xA5).all())
    first = D.clone()
    before.as_strided((vocab, cols), (cols + 2 * pad, 1)).copy_(D)
    assert torch.equal(before, buf)  # nothing else is written
    D.copy_(D0)
    G.gemm_embed_backward(*args, scale=scale, accumulate=accumulate, id_bytes=id_bytes)
    assert torch.equal(first, D)  # the same bits again


def test_gradient_in_exact_sums():
    """Whole numbers below 2^24: any order gives the sum itself."""
    gen = torch.Generator().manual_seed(5)
    tokens, vocab, cols = 30000, 3000, 96
    ids = ids_of(tokens, vocab, "hot")
    dY = torch.randint(-8, 9, (tokens, cols), generator=gen).bfloat16()
    D = torch.empty(vocab, cols, device="cuda")
    ws = torch.empty(G.gemm_embed_workspace(tokens, vocab, cols), dtype=torch.uint8, device="cuda")
    G.gemm_embed_backward(tokens, vocab, cols, "bf16", "f32", ids.cuda(), dY.cuda(), 0, D, 0, ws,
                          id_bytes=8)
    ref, _, _ = embed_grad_ref(ids, dY, vocab, 1.0)
    assert torch.equal(D.cpu().double(), ref)


def test_gradient_replayed():
    """Captured once, replayed with other ids and rows between eager work; two
    graphs on one workspace, one after the other."""
    tokens, vocab, cols = 3000, 900, 64
    ids = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    dY = torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    D = torch.zeros(vocab, cols, device="cuda")
    Y = torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(G.gemm_embed_workspace(tokens, vocab, cols), dtype=torch.uint8, device="cuda")

    def step(acc):
        G.gemm_embed_backward(tokens, vocab, cols, "bf16", "f32", ids, dY, 0, D, 0, ws, id_bytes=8,
                              accumulate=acc)
        G.gemm_embed(tokens, vocab, cols, "f32", "bf16", ids, D, 0, Y, 0, id_bytes=8)

    graphs = []
    for acc in (False, True):
        step(acc)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(acc)
        graphs.append(g)
    for seed in range(3):
        new = ids_of(tokens, vocab, "hot", seed)
        gen = torch.Generator().manual_seed(seed)
        rows = torch.randint(-8, 9, (tokens, cols), generator=gen).bfloat16()
        ids.copy_(new)
        dY.copy_(rows)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        ref = 2 * embed_grad_ref(new, rows, vocab, 1.0)[0]
        assert torch.equal(D.cpu().double(), ref)
        assert torch.equal(Y.cpu().double(), embed_ref(new, ref.float(), 1.0).bfloat16().double())
        step(False)  # eager work between the replays


def test_on_another_stream():
    tokens, vocab, cols = 2000, 400, 64
    s = torch.cuda.Stream()
    gen = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    dY = torch.randint(-8, 9, (tokens, cols), generator=gen, device="cuda").half()
    D = torch.empty(vocab, cols, device="cuda")
    ws = torch.empty(G.gemm_embed_workspace(tokens, vocab, cols), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        G.gemm_embed_backward(tokens, vocab, cols, "f16", "f32", ids, dY, 0, D, 0, ws, id_bytes=8)
    s.synchronize()
    assert torch.equal(D.cpu().double(), embed_grad_ref(ids.cpu(), dY.cpu(), vocab, 1.0)[0])


def test_offsets_past_32_bits():
    """A table and rows of more than 2^32 bytes: the last rows."""
    vocab, cols = 1 << 20, 2056
    E = torch.zeros(vocab, cols, dtype=torch.bfloat16, device="cuda")
    E[-1], E[-2] = 1.5, 2.5
    ids = torch.tensor([vocab - 1, vocab - 2, 0, vocab], device="cuda")
    Y = torch.empty(4, cols, dtype=torch.bfloat16, device="cuda")
    G.gemm_embed(4, vocab, cols, "bf16", "bf16", ids, E, 0, Y, 0, id_bytes=8)
    assert Y.unique(dim=1).squeeze(1).tolist() == [1.5, 2.5, 0.0, 0.0]
    tokens = 1500
    many = torch.full((tokens,), vocab - 1, device="cuda")
    dY = torch.ones(tokens, cols, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(G.gemm_embed_workspace(tokens, vocab, cols), dtype=torch.uint8, device="cuda")
    G.gemm_embed_backward(tokens, vocab, cols, "bf16", "bf16", many, dY, 0, E, 0, ws, id_bytes=8)
    assert bool((E[-1] == 1504.0).all())  # 1500 to 8 bits
    assert not bool(E[:-1].any())
    G.gemm_embed_backward(3, vocab, cols, "bf16", "bf16", many, dY, 0, E, 0, None, id_bytes=8)
    assert bool((E[-1] == 3.0).all()) and not bool(E[:-1].any())
