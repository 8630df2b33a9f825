"""Refusals of the mixture-of-experts entry points (include/gemm_moe.h): bad
sizes, types, pointers, alignment and overlaps are refused on the host before
anything is launched.  CPU only; the addresses are never dereferenced."""
import ctypes

import pytest

from sparse_tiled_gemm_amd import gemm as G


def P(i, off=0):
    """A fake device address, 2^42 bytes from the next."""
    return ((i + 1) << 42) + off


def _status(fn, *a, **kw):
    try:
        fn(*a, stream=0, **kw)
    except G.GemmError as e:
        return e.status
    return G.GEMM_OK


ROUTE = dict(tokens=8, topk=2, groups=4, cols=64, dtype="bf16", ids=P(0), X=P(1), ldx=0,
             offsets=P(2), order=P(3), pos=P(4), Xs=P(5), ldxs=0, workspace=P(6), id_bytes=8)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), G.GEMM_ERR_INVALID_VALUE),
    (dict(topk=0), G.GEMM_ERR_INVALID_VALUE),
    (dict(groups=0), G.GEMM_ERR_INVALID_VALUE),
    (dict(groups=1025), G.GEMM_ERR_UNSUPPORTED),
    (dict(tokens=1 << 30), G.GEMM_ERR_UNSUPPORTED),
    (dict(cols=-1), G.GEMM_ERR_INVALID_VALUE),
    (dict(cols=(1 << 23) + 1), G.GEMM_ERR_UNSUPPORTED),
    (dict(dtype="f32"), G.GEMM_ERR_UNSUPPORTED),
    (dict(ldx=63), G.GEMM_ERR_INVALID_VALUE),
    (dict(ldxs=-64), G.GEMM_ERR_INVALID_VALUE),
    (dict(ldxs=1 << 41), G.GEMM_ERR_INVALID_VALUE),
    (dict(id_bytes=2), G.GEMM_ERR_INVALID_VALUE),
    (dict(ids=None), G.GEMM_ERR_NULL_POINTER),
    (dict(X=None), G.GEMM_ERR_NULL_POINTER),
    (dict(offsets=None), G.GEMM_ERR_NULL_POINTER),
    (dict(order=None), G.GEMM_ERR_NULL_POINTER),
    (dict(pos=None), G.GEMM_ERR_NULL_POINTER),
    (dict(Xs=None), G.GEMM_ERR_NULL_POINTER),
    (dict(tokens=4096, workspace=None), G.GEMM_ERR_NULL_POINTER),
    (dict(ids=P(0, 4)), G.GEMM_ERR_MISALIGNED),
    (dict(X=P(1, 1)), G.GEMM_ERR_MISALIGNED),
    (dict(pos=P(4, 2)), G.GEMM_ERR_MISALIGNED),
    (dict(Xs=P(1, 64)), G.GEMM_ERR_UNSUPPORTED),           # overlaps X
    (dict(order=P(4, 32)), G.GEMM_ERR_UNSUPPORTED),        # overlaps pos
    (dict(offsets=P(0, 64)), G.GEMM_ERR_UNSUPPORTED),      # overlaps ids
])
def test_dispatch_refusals(change, status):
    a = dict(ROUTE, **change)
    kw = dict(id_bytes=a.pop("id_bytes"))
    assert _status(G.gemm_moe_dispatch, *a.values(), **kw) == status, G.gemm_last_error()


def test_sort_workspace():
    assert G.gemm_moe_sort_workspace(0, 1, 1) == 0
    assert G.gemm_moe_sort_workspace(4096, 1, 64) == 0
    assert G.gemm_moe_sort_workspace(4097, 1, 64) == 5 * 64 * 4
    # at most 256 chunks
    assert G.gemm_moe_sort_workspace(1 << 20, 8, 1024) <= 256 * 1024 * 4
    for bad in [(-1, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 30, 4, 1), (1, 1, 1025)]:
        with pytest.raises(G.GemmError):
            G.gemm_moe_sort_workspace(*bad)
    assert G.load().gemm_moe_sort_workspace(1, 1, 1, None) == G.GEMM_ERR_NULL_POINTER


def test_sort_refusals():
    base = [8, 2, 4, P(0), P(2), P(3), P(4), None]
    for i, v, st in [(0, -1, G.GEMM_ERR_INVALID_VALUE), (3, None, G.GEMM_ERR_NULL_POINTER),
                     (4, P(0, 60), G.GEMM_ERR_UNSUPPORTED), (6, P(4, 1), G.GEMM_ERR_MISALIGNED)]:
        a = list(base)
        a[i] = v
        assert _status(G.gemm_moe_sort, *a, id_bytes=4) == st


COMBINE = dict(tokens=8, topk=2, cols=64, dtype="f16", pos=P(0), weights=P(1), Ys=P(2), ldys=0,
               rows=16, Y=P(3), ldy=0)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), G.GEMM_ERR_INVALID_VALUE),
    (dict(ldys=8), G.GEMM_ERR_INVALID_VALUE),
    (dict(ldy=8), G.GEMM_ERR_INVALID_VALUE),
    (dict(dtype="e4m3"), G.GEMM_ERR_UNSUPPORTED),
    (dict(pos=None), G.GEMM_ERR_NULL_POINTER),
    (dict(Ys=None), G.GEMM_ERR_NULL_POINTER),
    (dict(Y=None), G.GEMM_ERR_NULL_POINTER),
    (dict(weights=P(1, 2)), G.GEMM_ERR_MISALIGNED),
    (dict(Y=P(2)), G.GEMM_ERR_UNSUPPORTED),
    (dict(Y=P(1)), G.GEMM_ERR_UNSUPPORTED),
])
def test_combine_refusals(change, status):
    assert _status(G.gemm_moe_combine, *dict(COMBINE, **change).values()) == status


COMBINE_BW = dict(tokens=8, topk=2, cols=64, dtype="f16", pos=P(0), weights=P(1), dY=P(2), lddy=0,
                  Ys=P(3), ldys=0, rows=16, dYs=P(4), lddys=0, dw=P(5))


@pytest.mark.parametrize("change,status", [
    (dict(weights=None), G.GEMM_ERR_NULL_POINTER),
    (dict(dw=None), G.GEMM_ERR_NULL_POINTER),
    (dict(dw=P(1)), G.GEMM_ERR_UNSUPPORTED),
    (dict(dYs=P(3)), G.GEMM_ERR_UNSUPPORTED),   # not in place
    (dict(dYs=P(2, 128)), G.GEMM_ERR_UNSUPPORTED),
    (dict(lddy=63), G.GEMM_ERR_INVALID_VALUE),
    (dict(lddys=63), G.GEMM_ERR_INVALID_VALUE),
    (dict(dY=P(2, 1)), G.GEMM_ERR_MISALIGNED),
])
def test_combine_backward_refusals(change, status):
    assert _status(G.gemm_moe_combine_backward, *dict(COMBINE_BW, **change).values()) == status


def _desc(mode="rows", rows=64, N=64, K=64, groups=4, a="bf16", b=None, d="bf16", **kw):
    return G.make_grouped_desc(mode, rows, N, K, groups, a, b or a, d, **kw)


@pytest.mark.parametrize("desc,status", [
    (dict(), G.GEMM_OK),
    (dict(rows=0, N=0, K=0), G.GEMM_OK),
    (dict(a="f16", d="f32", b_layout="row"), G.GEMM_OK),
    (dict(mode="weights", d="f32", has_c=True), G.GEMM_OK),
    (dict(mode="weights", b="e4m3", d="f32"), G.GEMM_OK),
    (dict(rows=-1), G.GEMM_ERR_INVALID_VALUE),
    (dict(K=1 << 31), G.GEMM_ERR_INVALID_VALUE),
    (dict(groups=0), G.GEMM_ERR_INVALID_VALUE),
    (dict(groups=65536), G.GEMM_ERR_INVALID_VALUE),
    (dict(lda=63), G.GEMM_ERR_INVALID_VALUE),
    (dict(ldb=63), G.GEMM_ERR_INVALID_VALUE),
    (dict(ldd=1), G.GEMM_ERR_INVALID_VALUE),
    (dict(ldd=-64), G.GEMM_ERR_INVALID_VALUE),
    (dict(lda=1 << 41), G.GEMM_ERR_INVALID_VALUE),
    (dict(rows=1 << 30, lda=1 << 12), G.GEMM_ERR_INVALID_VALUE),
    (dict(algo=6), G.GEMM_ERR_INVALID_VALUE),
    (dict(a="f32"), G.GEMM_ERR_UNSUPPORTED),
    (dict(a="bf16", b="f16"), G.GEMM_ERR_UNSUPPORTED),
    (dict(b="e4m3"), G.GEMM_ERR_UNSUPPORTED),               # 8-bit B: weights only
    (dict(d="e4m3"), G.GEMM_ERR_UNSUPPORTED),
    (dict(has_c=True), G.GEMM_ERR_UNSUPPORTED),
    (dict(mode="weights", b_layout="col"), G.GEMM_ERR_UNSUPPORTED),
    (dict(mode="weights", b="e4m3", ldb=72), G.GEMM_ERR_UNSUPPORTED),
    (dict(rows=1 << 24, N=1 << 13, K=8), G.GEMM_ERR_UNSUPPORTED),  # too many tiles
])
def test_grouped_desc(desc, status):
    assert G.gemm_grouped_validate_desc(_desc(**desc)) == status, G.gemm_last_error()


def test_grouped_null_and_bad_enums():
    L = G.load()
    assert G.gemm_grouped_validate_desc(None) == G.GEMM_ERR_NULL_POINTER
    for f, v in [("mode", 2), ("a_type", 0), ("b_layout", 5), ("has_c", 2), ("algo", -1)]:
        d = _desc()
        setattr(d, f, v)
        assert G.gemm_grouped_validate_desc(d) == G.GEMM_ERR_INVALID_VALUE, f
    assert L.gemm_grouped_plan(None, ctypes.byref(ctypes.c_void_p())) == G.GEMM_ERR_NULL_POINTER
    assert L.gemm_grouped_plan(ctypes.byref(_desc()), None) == G.GEMM_ERR_NULL_POINTER
    assert L.gemm_grouped_run(None, P(0), P(1), None, P(2), None, P(3), None) == \
        G.GEMM_ERR_NULL_POINTER
    assert L.gemm_grouped_plan_describe(None, None, 0) == G.GEMM_ERR_NULL_POINTER
    assert L.gemm_grouped_plan_destroy(None) == G.GEMM_OK


Q8 = dict(rows=8, cols=64, dtype="bf16")


@pytest.mark.parametrize("fn,args,status", [
    (G.gemm_q8_store, dict(X=P(0), ldx=0, codes=P(1), scales=None), G.GEMM_ERR_NULL_POINTER),
    (G.gemm_q8_store, dict(X=P(0), ldx=63, codes=P(1), scales=P(2)), G.GEMM_ERR_INVALID_VALUE),
    (G.gemm_q8_store, dict(X=P(0), ldx=0, codes=P(0), scales=P(2)), G.GEMM_ERR_UNSUPPORTED),
    (G.gemm_q8_store, dict(X=P(0, 1), ldx=0, codes=P(1), scales=P(2)), G.GEMM_ERR_MISALIGNED),
    (G.gemm_q8_load, dict(codes=None, scales=P(1), X=P(2), ldx=0), G.GEMM_ERR_NULL_POINTER),
    (G.gemm_q8_load, dict(codes=P(0), scales=P(2, 16), X=P(2), ldx=0), G.GEMM_ERR_UNSUPPORTED),
    (G.gemm_swiglu, dict(GU=P(0), ldgu=127, H=P(1), ldh=0), G.GEMM_ERR_INVALID_VALUE),
    (G.gemm_swiglu, dict(GU=P(0), ldgu=0, H=P(1), ldh=0, codes=P(2)), G.GEMM_ERR_NULL_POINTER),
    (G.gemm_swiglu, dict(GU=P(0), ldgu=0, H=P(0), ldh=0), G.GEMM_ERR_UNSUPPORTED),
    (G.gemm_swiglu, dict(GU=P(0), ldgu=0, H=None, ldh=0), G.GEMM_ERR_NULL_POINTER),
    (G.gemm_swiglu_backward, dict(codes=P(0), scales=P(1), dH=P(2), lddh=0, dGU=P(2), lddgu=0),
     G.GEMM_ERR_UNSUPPORTED),
    (G.gemm_swiglu_backward, dict(codes=P(0), scales=P(1), dH=P(2), lddh=0, dGU=P(3), lddgu=64),
     G.GEMM_ERR_INVALID_VALUE),
    (G.gemm_swiglu_backward, dict(codes=P(0), scales=P(1), dH=P(2), lddh=0, dGU=P(3), lddgu=0,
                                  H=P(3)), G.GEMM_ERR_UNSUPPORTED),
])
def test_q8_refusals(fn, args, status):
    a = dict(Q8, **args)
    assert _status(fn, *a.values()) == status, G.gemm_last_error()
    for change, st in [(dict(rows=-1), G.GEMM_ERR_INVALID_VALUE),
                       (dict(dtype="f32"), G.GEMM_ERR_UNSUPPORTED),
                       (dict(cols=-2), G.GEMM_ERR_INVALID_VALUE),
                       (dict(rows=1 << 40), G.GEMM_ERR_INVALID_VALUE)]:
        assert _status(fn, *dict(a, **change).values()) == st


def test_arguments_of_the_wrong_kind():
    """Integers, addresses, None and tensors only; nothing is cut to an integer."""
    from sparse_tiled_gemm_amd import _pycall
    torch = pytest.importorskip("torch")
    a = dict(COMBINE, tokens=0, rows=0)
    x = torch.zeros(4)
    assert _status(G.gemm_moe_combine, *dict(a, pos=x, weights=x, Ys=x, Y=x).values()) == G.GEMM_OK
    for k, v in [("tokens", 2.0), ("pos", "0"), ("weights", [1.0]), ("Ys", b"")]:
        with pytest.raises(TypeError):
            G.gemm_moe_combine(*dict(a, **{k: v}).values(), stream=0)
    for bad in [(), ("f",), (1,) * 22]:
        with pytest.raises(TypeError):
            _pycall.call(*bad)
    with pytest.raises(ValueError):
        _pycall.call(0, 1)


def test_calls_let_other_threads_run():
    """A call that waits (a full queue, a first launch) stops its own thread only."""
    import threading
    import time

    from sparse_tiled_gemm_amd import _pycall
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    begun, seen = threading.Event(), []

    def other():
        begun.wait()
        for _ in range(4):
            time.sleep(0.05)
            seen.append(time.monotonic())

    t = threading.Thread(target=other)
    t.start()
    begun.set()
    assert _pycall.call(usleep, 900000) == 0
    end = time.monotonic()
    t.join()
    assert seen[0] < end - 0.3
