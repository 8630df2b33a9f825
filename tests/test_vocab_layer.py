"""TiedVocab's handling of its arguments (sparse_tiled_gemm_amd.vocab), without
a GPU: the library's calls are recorded instead of made, with the tensors and
leading dimensions that the kernels would have read."""
import types

import pytest
import torch

from sparse_tiled_gemm_amd import gemm as G
from sparse_tiled_gemm_amd import vocab
from test_moe_layer import dev, read_back

T, V, H = 5, 11, 16


class Recorded(types.SimpleNamespace):
    def __init__(self):
        super().__init__(calls=[], make_xent_desc=G.make_xent_desc,
                         gemm_embed_workspace=lambda *a: 64, gemm_xent_workspace=lambda p: (128, 256),
                         gemm_xent_plan=lambda desc: types.SimpleNamespace(desc=desc))
        for name in ("gemm_embed", "gemm_embed_backward", "gemm_xent_forward", "gemm_xent_backward"):
            setattr(self, name, lambda *a, _n=name, **kw: self.calls.append((_n, a, kw)))

    def last(self, name):
        return [(a, kw) for n, a, kw in self.calls if n == name][-1]


@pytest.fixture
def lib(monkeypatch):
    lib = Recorded()
    monkeypatch.setattr(vocab, "G", lib)
    return lib


def ends_of(E=None, **kw):
    return vocab.TiedVocab(dev(torch.zeros(V, H, dtype=torch.bfloat16)) if E is None else E, T, **kw)


def matrix(seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=gen).bfloat16()


def views(x):
    wide = torch.zeros(len(x), H + 8, dtype=x.dtype)
    wide[:, :H] = x
    return {"packed": x, "padded": wide[:, :H], "every other": x.repeat_interleave(2, 0)[::2],
            "one row": x[:1].expand(len(x), H),
            "overlapping": torch.arange(H + 3 * T, dtype=x.dtype).as_strided((len(x), H), (3, 1))}


@pytest.mark.parametrize("kind", ["packed", "padded", "every other", "one row", "overlapping"])
def test_rows_are_read_where_they_lie(lib, kind):
    """X and dX0 of any row stride, broadcast rows among them."""
    ends, x = ends_of(), dev(views(matrix())[kind])
    want = x.clone()
    ids = dev(torch.arange(T))
    ends.loss(x, ids)
    a, _ = lib.last("gemm_xent_forward")
    d = a[0].desc
    assert torch.equal(read_back(a[1], d.ldx, T, H), want) and d.id_bytes == 8
    ends.embed(ids)
    ends.embed_backward(x)
    a, kw = lib.last("gemm_embed_backward")
    assert torch.equal(read_back(a[6], a[7], T, H), want) and kw["accumulate"] is True


def test_the_gradient_reads_what_the_forward_pass_read(lib):
    ends, x, y = ends_of(logit_scale=0.5), dev(matrix()), dev(torch.arange(T, dtype=torch.int32))
    loss, lse = ends.loss(x, y)
    g = dev(torch.ones(T))
    ends.loss_backward(g, accumulate=True)
    f, b = lib.last("gemm_xent_forward")[0], lib.last("gemm_xent_backward")[0]
    assert f[1].data_ptr() == b[1].data_ptr() == x.data_ptr()
    assert b[3] is y and b[4] is lse and b[6] is None and b[8] is ends.dE
    assert b[0].desc.accumulate == 1 and f[0].desc.accumulate == 0
    assert b[0].desc.scale == 0.5 and b[0].desc.id_bytes == 4
    assert b[0].desc.dw_type == G.DTYPES["f32"] and b[0].desc.dx_type == G.DTYPES["bf16"]


def test_a_padded_table(lib):
    wide = dev(torch.zeros(V, H + 8, dtype=torch.float16))
    ends = ends_of(wide[:, :H])
    ends.embed(dev(torch.zeros(T, dtype=torch.int64)))
    a, kw = lib.last("gemm_embed")
    assert a[7] == H + 8 and a[3] == "f16"
    assert ends._plan(8, H, False).desc.ldw == H + 8


def test_any_truth_value_picks_a_plan(lib):
    ends, x, y = ends_of(), dev(matrix()), dev(torch.arange(T))
    ends.loss(x, y)
    for acc in (1, 0, torch.tensor(True), "yes"):
        ends.loss_backward(dev(torch.ones(T)), accumulate=acc)
        assert lib.last("gemm_xent_backward")[0][0].desc.accumulate == int(bool(acc))


def test_refusals(lib):
    ends, x, y = ends_of(), dev(matrix()), dev(torch.arange(T))
    g = dev(torch.ones(T))
    with pytest.raises(RuntimeError):
        ends.loss_backward(g)
    with pytest.raises(RuntimeError):
        ends.embed_backward(x)
    ends.loss(x, y)
    for bad in (y[:4], y.float(), y.to(torch.int16), dev(torch.arange(2 * T))[::2], y.view(1, T)):
        with pytest.raises(ValueError):
            ends.embed(bad)
        with pytest.raises(ValueError):
            ends.loss(x, bad)
    for bad in (x[:4], x.float(), x.half(), x.t().contiguous().t(), x[:, :8]):
        with pytest.raises(ValueError):
            ends.loss(bad, y)
    for bad in (g[:4], g.double(), g.half(), dev(torch.ones(2 * T))[::2]):
        with pytest.raises(ValueError):
            ends.loss_backward(bad)
        with pytest.raises(ValueError):
            ends.loss_backward(g, bad)
    with pytest.raises(ValueError):  # on the host
        ends.loss(matrix(), y)
    with pytest.raises(ValueError):
        ends.loss(x, torch.arange(T))
    for bad in (torch.zeros(V, H), torch.zeros(V, dtype=torch.float16),
                torch.zeros(H, V, dtype=torch.float16).t(),
                torch.zeros(1, H, dtype=torch.float16).expand(V, H)):
        with pytest.raises(ValueError):
            ends_of(dev(bad))
    with pytest.raises(ValueError):
        ends_of(torch.zeros(V, H, dtype=torch.float16))


def test_no_graph_of_the_callers_is_kept(lib):
    E = dev(torch.zeros(V, H, dtype=torch.bfloat16)).requires_grad_()
    ends = ends_of(E)
    x = dev(matrix()).requires_grad_()
    ends.loss(x, dev(torch.arange(T)))
    ends.loss_backward(dev(torch.ones(T)).requires_grad_())
    a = lib.last("gemm_xent_backward")[0]
    assert not any(isinstance(t, torch.Tensor) and t.requires_grad for t in a)


def test_the_gradient_starts_at_zero(lib):
    """The first call may add to dE: embed_backward() does by default."""
    torch.use_deterministic_algorithms(True)  # torch.empty's memory is filled with NaN
    try:
        ends = ends_of()
    finally:
        torch.use_deterministic_algorithms(False)
    assert (ends.dE == 0).all()
