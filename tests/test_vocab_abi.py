"""Refusals of the entry points over a vocabulary (include/gemm_vocab.h): bad
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


INVALID, UNSUPPORTED = G.GEMM_ERR_INVALID_VALUE, G.GEMM_ERR_UNSUPPORTED
NULL, MISALIGNED = G.GEMM_ERR_NULL_POINTER, G.GEMM_ERR_MISALIGNED
EMBED = dict(tokens=8, vocab=100, cols=64, e_dtype="bf16", y_dtype="f16", ids=P(0), E=P(1), lde=0,
             Y=P(2), ldy=0, id_bytes=8)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), INVALID), (dict(vocab=-1), INVALID), (dict(cols=-1), INVALID),
    (dict(tokens=(1 << 25) + 1), UNSUPPORTED), (dict(vocab=(1 << 20) + 1), UNSUPPORTED),
    (dict(cols=(1 << 23) + 1), UNSUPPORTED), (dict(e_dtype="s8"), UNSUPPORTED),
    (dict(y_dtype="e4m3"), UNSUPPORTED), (dict(id_bytes=2), INVALID), (dict(lde=63), INVALID),
    (dict(ldy=-64), INVALID), (dict(ldy=1 << 41), INVALID), (dict(ids=None), NULL),
    (dict(E=None), NULL), (dict(Y=None), NULL), (dict(ids=P(0, 4)), MISALIGNED),
    (dict(E=P(1, 1)), MISALIGNED), (dict(e_dtype="f32", E=P(1, 2)), MISALIGNED),
    (dict(Y=P(2, 1)), MISALIGNED), (dict(Y=P(1, 128)), UNSUPPORTED), (dict(Y=P(0, 8)), UNSUPPORTED),
])
def test_embed_refusals(change, status):
    a = dict(EMBED, **change)
    kw = dict(id_bytes=a.pop("id_bytes"))
    assert _status(G.gemm_embed, *a.values(), **kw) == status, G.gemm_last_error()


def test_nothing_to_do():
    """No tokens or no columns: no pointer is needed, no device touched."""
    G.gemm_embed(0, 10, 64, "bf16", "bf16", None, P(1), 0, None, 0, stream=0)
    G.gemm_embed(4, 10, 0, "bf16", "bf16", P(0), None, 0, None, 0, stream=0)
    G.gemm_embed_backward(0, 10, 64, "bf16", "f32", None, None, 0, P(2), 0, None, accumulate=True,
                          stream=0)
    G.gemm_embed_backward(4, 0, 64, "bf16", "f32", P(0), P(1), 0, None, 0, None, stream=0)


BACK = dict(tokens=2000, vocab=100, cols=64, y_dtype="bf16", e_dtype="f32", ids=P(0), dY=P(1), lddy=0,
            dE=P(2), ldde=0, workspace=P(3), id_bytes=4)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), INVALID), (dict(e_dtype="u4"), UNSUPPORTED), (dict(lddy=1), INVALID),
    (dict(ldde=63), INVALID), (dict(ids=None), NULL), (dict(dY=None), NULL), (dict(dE=None), NULL),
    (dict(workspace=None), NULL), (dict(workspace=P(3, 8)), MISALIGNED),
    (dict(dE=P(2, 2)), MISALIGNED), (dict(dY=P(1, 1)), MISALIGNED), (dict(ids=P(0, 2)), MISALIGNED),
    (dict(dE=P(1, 64)), UNSUPPORTED), (dict(workspace=P(2, 64)), UNSUPPORTED),
    (dict(workspace=P(0)), UNSUPPORTED), (dict(dE=P(0)), UNSUPPORTED),
])
def test_embed_backward_refusals(change, status):
    a = dict(BACK, **change)
    kw = dict(id_bytes=a.pop("id_bytes"))
    assert _status(G.gemm_embed_backward, *a.values(), **kw) == status, G.gemm_last_error()


def test_embed_backward_accumulate_is_a_truth_value():
    L = G.load()
    assert L.gemm_embed_backward(8, 10, 64, 2, 6, 4, P(0), P(1), 0, P(2), 0, 2, None, 1.0,
                                 None) == INVALID


def test_embed_workspace():
    assert G.gemm_embed_workspace(0, 10, 64) == 0
    assert G.gemm_embed_workspace(1024, 1 << 20, 64) == 0
    assert G.gemm_embed_workspace(1025, 100, 64) > 0
    n = G.gemm_embed_workspace(65536, 131072, 4096)
    # two fp32 rows per 32 tokens, three ints per token, the counts
    assert 65536 // 32 * 2 * 4096 * 4 <= n <= 65536 // 32 * 2 * 4096 * 4 + 16 * 65536 + 4 * 64 * 1024
    for bad in [(-1, 1, 1), (1, (1 << 20) + 1, 1), (1, 1, -1), ((1 << 25) + 1, 1, 1)]:
        with pytest.raises(G.GemmError):
            G.gemm_embed_workspace(*bad)
    assert G.load().gemm_embed_workspace(1, 1, 1, None) == NULL


def desc(**kw):
    d = G.make_xent_desc(64, 1000, 128, "bf16")
    for k, v in kw.items():
        setattr(d, k, G.DTYPES[v] if isinstance(v, str) else v)
    return d


@pytest.mark.parametrize("change,status", [
    (dict(), G.GEMM_OK), (dict(tokens=0), G.GEMM_OK), (dict(hidden=129), G.GEMM_OK),
    (dict(vocab=1), G.GEMM_OK), (dict(ldx=130, ldw=136), G.GEMM_OK), (dict(piece=1), G.GEMM_OK),
    (dict(dx_type="f32", dw_type="f16", id_bytes=8, accumulate=1, unaligned=1), G.GEMM_OK),
    (dict(tokens=-1), INVALID), (dict(vocab=0), INVALID), (dict(hidden=0), INVALID),
    (dict(x_type=0), INVALID), (dict(dw_type=13), INVALID), (dict(id_bytes=0), INVALID),
    (dict(accumulate=2), INVALID), (dict(unaligned=-1), INVALID), (dict(ldx=127), INVALID),
    (dict(ldw=-1), INVALID), (dict(lddx=1), INVALID), (dict(lddw=1 << 41), INVALID),
    (dict(piece=-1), INVALID), (dict(x_type="f32"), UNSUPPORTED), (dict(dx_type="s32"), UNSUPPORTED),
    (dict(dw_type="e5m2"), UNSUPPORTED), (dict(tokens=(1 << 20) + 1), UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1), UNSUPPORTED), (dict(hidden=(1 << 15) + 1), UNSUPPORTED),
    (dict(tokens=1 << 20, vocab=1 << 24, hidden=8), UNSUPPORTED),
])
def test_xent_desc(change, status):
    assert G.gemm_xent_validate_desc(desc(**change)) == status, G.gemm_last_error()


def test_null_arguments():
    L = G.load()
    assert G.gemm_xent_validate_desc(None) == NULL
    assert L.gemm_xent_plan(ctypes.byref(desc()), None) == NULL
    h = ctypes.c_void_p(1)
    assert L.gemm_xent_plan(None, ctypes.byref(h)) == NULL and not h.value
    assert L.gemm_xent_plan_destroy(None) == G.GEMM_OK
    assert L.gemm_xent_plan_describe(None, None, 0) == NULL
    assert L.gemm_xent_workspace(None, None, None) == NULL
    assert L.gemm_xent_forward(*[None] * 8) == NULL
    assert L.gemm_xent_backward(*[None] * 11) == NULL


def test_one_float_among_the_arguments():
    """The binding passes a function's float wherever it stands, and refuses
    floats in the place of integers."""
    for tokens in (1.5, 0.0):
        with pytest.raises(TypeError):
            G.gemm_embed(tokens, 10, 64, "bf16", "bf16", None, None, 0, None, 0, stream=0)
        with pytest.raises(TypeError):
            G.gemm_q8_store(tokens, 64, "bf16", None, 0, None, None, stream=0)
    G.gemm_embed(0, 10, 64, "bf16", "bf16", None, P(1), 0, None, 0, scale=2, stream=0)


def test_descriptor_size_matches_the_header(tmp_path):
    """gemm_xent_desc_t as the C compiler lays it out."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include "gemm_vocab.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu", sizeof(gemm_xent_desc_t),'
                   'offsetof(gemm_xent_desc_t, ldx), offsetof(gemm_xent_desc_t, piece),'
                   'offsetof(gemm_xent_desc_t, scale));return 0;}')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    T = G.gemm_xent_desc_t
    assert got == [ctypes.sizeof(T), T.ldx.offset, T.piece.offset, T.scale.offset]
