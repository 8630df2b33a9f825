"""The layer's handling of its arguments (sparse_tiled_gemm_amd.moe), without
a GPU: the library's calls are recorded instead of made, with the tensors and
leading dimensions that the kernels would have read."""
import types

import pytest
import torch

from sparse_tiled_gemm_amd import gemm as G
from sparse_tiled_gemm_amd import moe

T, K, E, H, F = 5, 2, 3, 16, 8


class Recorded(types.SimpleNamespace):
    def __init__(self):
        super().__init__(calls=[], make_grouped_desc=G.make_grouped_desc,
                         gemm_moe_sort_workspace=lambda *a: 0,
                         gemm_grouped_plan=lambda desc: types.SimpleNamespace(desc=desc))
        for name in ("gemm_moe_dispatch", "gemm_grouped_run", "gemm_swiglu", "gemm_moe_combine",
                     "gemm_q8_store", "gemm_moe_combine_backward", "gemm_swiglu_backward"):
            setattr(self, name, lambda *a, _n=name, **kw: self.calls.append((_n, a, kw)))

    def args(self, name):
        return [a for n, a, _ in self.calls if n == name][-1]


class OnDevice(torch.Tensor):
    """A tensor in host memory that says it is on the device."""
    is_cuda = True


def dev(x):
    return x.as_subclass(OnDevice)


@pytest.fixture
def lib(monkeypatch):
    lib = Recorded()
    monkeypatch.setattr(moe, "G", lib)
    return lib


def layer_of(tokens=T):
    return moe.ExpertMLP(dev(torch.zeros(E, 2 * F, H, dtype=torch.bfloat16)),
                         dev(torch.zeros(E, H, F, dtype=torch.bfloat16)), tokens, K)


def inputs(tokens=T):
    gen = torch.Generator().manual_seed(0)
    return (dev(torch.randn(tokens, H, generator=gen).bfloat16()),
            dev(torch.randint(0, E, (tokens, K), generator=gen)),
            dev(torch.rand(tokens, K, generator=gen)))


def read_back(x, ld, rows, cols):
    """What a kernel reads at x with leading dimension ld (0: packed)."""
    ld = ld or cols
    assert ld >= cols
    last = x.storage_offset() + (rows - 1) * ld + cols
    assert last * x.element_size() <= x.untyped_storage().nbytes(), "read past the buffer"
    return x.as_strided((rows, cols), (ld, 1))


def views(x):
    """The same rows in other strides."""
    wide = torch.zeros(len(x), H + 8, dtype=x.dtype)
    wide[:, :H] = x
    row = x[:1]
    lapped = torch.arange(H + 3 * T, dtype=x.dtype)
    return {"packed": x, "padded": dev(wide[:, :H]), "every other": dev(x.repeat_interleave(2, 0)[::2]),
            "one row": row.expand(len(x), H),
            "overlapping": dev(lapped.as_strided((len(x), H), (3, 1)))}


@pytest.mark.parametrize("kind", ["packed", "padded", "every other", "one row", "overlapping"])
def test_rows_are_read_where_they_lie(lib, kind):
    """X and dY of any row stride, broadcast rows among them."""
    layer, (X, ids, w) = layer_of(), inputs()
    x = views(X)[kind]
    layer.forward(x, ids, w)
    a = lib.args("gemm_moe_dispatch")
    assert torch.equal(read_back(a[6], a[7], T, H), x)
    layer.backward(x)
    a = lib.args("gemm_moe_combine_backward")
    assert torch.equal(read_back(a[6], a[7], T, H), x)


def test_one_token_of_any_stride(lib):
    """The row stride of a single row means nothing."""
    layer, (X, ids, w) = layer_of(1), inputs(1)
    for stride in (1, 0, H - 1, 1000):
        x = dev(X.as_strided((1, H), (stride, 1)))
        layer.forward(x, ids, w)
        a = lib.args("gemm_moe_dispatch")
        assert torch.equal(read_back(a[6], a[7], 1, H), x)
        layer.backward(x)
        a = lib.args("gemm_moe_combine_backward")
        assert torch.equal(read_back(a[6], a[7], 1, H), x)


def test_tensors_off_the_device_are_refused(lib):
    """Host memory never reaches a kernel."""
    W1, W2 = torch.zeros(E, 2 * F, H).bfloat16(), torch.zeros(E, H, F).bfloat16()
    for a, b in [(W1, W2), (dev(W1), W2), (W1, dev(W2))]:
        with pytest.raises(ValueError):
            moe.ExpertMLP(a, b, T, K)
    layer, (X, ids, w) = layer_of(), inputs()
    host = [t.as_subclass(torch.Tensor) for t in (X, ids, w)]
    meta = [torch.empty_like(t, device="meta") for t in host]  # another device
    lib.calls.clear()
    for i in range(3):
        for other in (host, meta):
            a = [X, ids, w]
            a[i] = other[i]
            with pytest.raises(ValueError):
                layer.forward(*a)
    assert not lib.calls
    layer.forward(X, ids, w)
    lib.calls.clear()
    for dY in (host[0], meta[0]):
        with pytest.raises(ValueError):
            layer.backward(dY)
    assert not lib.calls


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64, torch.int16, torch.uint8, torch.bool])
def test_ids_of_another_type_are_refused(lib, dtype):
    """Floats of an integer's size are not read as its bits."""
    layer, (X, ids, w) = layer_of(), inputs()
    with pytest.raises(ValueError):
        layer.forward(X, dev(ids.to(dtype)), w)
    assert not lib.calls
    for ok, size in ((torch.int32, 4), (torch.int64, 8)):
        layer.forward(X, dev(ids.to(ok)), w)
        assert [kw for n, _, kw in lib.calls if n == "gemm_moe_dispatch"][-1]["id_bytes"] == size


def test_weight_gradients_start_at_zero(lib):
    """The first backward pass may accumulate."""
    torch.use_deterministic_algorithms(True)  # torch.empty's memory is filled with NaN
    try:
        layer = layer_of()
    finally:
        torch.use_deterministic_algorithms(False)
    assert (layer.dW1 == 0).all() and (layer.dW2 == 0).all()


def test_weights_are_kept_as_they_were(lib):
    """The gradient is that of the forward pass, whatever the caller does to
    the weights in between."""
    layer, (X, ids, w) = layer_of(), inputs()
    want = w.clone()
    layer.forward(X, ids, w)
    a = lib.args("gemm_moe_combine")
    assert torch.equal(read_back(a[5].view(T, K), 0, T, K), want)
    w.fill_(7)
    layer.backward(X)
    a = lib.args("gemm_moe_combine_backward")
    assert torch.equal(read_back(a[5].view(T, K), 0, T, K), want)
    layer.forward(X, ids, w.clone().requires_grad_(True))
    assert not layer.weights.requires_grad


def test_backward_needs_a_forward(lib):
    layer, (X, ids, w) = layer_of(), inputs()
    with pytest.raises(RuntimeError):
        layer.backward(X)
    assert not lib.calls
    layer.forward(X, ids, w)
    layer.backward(X)
    layer.backward(X)  # of the same forward pass once more


def test_accumulate_and_keep8_are_truth_values(lib):
    """Any truth value picks a plan."""
    layer, (X, ids, w) = layer_of(), inputs()
    layer.forward(X, ids, w, keep8=torch.tensor(1))
    layer.backward(X, accumulate=2)
    run = [a for n, a, _ in lib.calls if n == "gemm_grouped_run"]
    dw1 = [a for a in run if a[6] is layer.dW1]
    assert dw1[0][0].desc.has_c == 1 and dw1[0][5] is layer.dW1 and dw1[0][2] is layer.xcodes


def test_weights_in_any_layout_follow_updates(lib):
    """Weights changed in place between steps are the ones the next step
    uses, contiguous or not."""
    gen = torch.Generator().manual_seed(1)
    w1 = torch.randn(E, H, 2 * F, generator=gen).bfloat16()
    w2 = torch.randn(H, E, F, generator=gen).bfloat16()
    for W1, W2 in [(w1.transpose(1, 2), w2.transpose(0, 1)),
                   (w1.transpose(1, 2).contiguous(), w2.transpose(0, 1).contiguous())]:
        layer = moe.ExpertMLP(dev(W1), dev(W2), T, K)
        X, ids, w = inputs()
        for _ in range(2):
            lib.calls.clear()
            layer.forward(X, ids, w)
            layer.backward(X)
            products = [a[2] for n, a, _ in lib.calls if n == "gemm_grouped_run"]
            for got, want in [(products[0], W1), (products[1], W2), (products[2], W2),
                              (products[5], W1)]:
                assert torch.equal(got, want) and got.is_contiguous()
            W1.mul_(-2)
            W2.add_(1)
    assert layer.W1.data_ptr() == W1.data_ptr()  # contiguous ones are read where they lie


def test_the_weights_gpu_is_the_current_one(monkeypatch):
    """The library launches on the current device: addresses of another
    device's memory do not go to it."""
    x = types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", 1))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        moe._check_device(x.device, X=x)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    moe._check_device(x.device, X=x)
