"""Python binding of libstgemm.so (include/gemm.h, include/gemm_moe.h, include/gemm_vocab.h).  Argument marshalling only:
every step of the computation runs in the library's HIP kernels.  Device
buffers are passed as torch tensors (their data pointers) or raw integer
addresses; PyTorch provides memory and streams only.

The functions carry the C names: gemm_validate_desc, gemm_plan,
gemm_plan_destroy, gemm_plan_describe, gemm_run, gemm_sparse24_sizes,
gemm_sparse24_compress, gemm_sparse24_compress_noalloc, gemm_sparse24_run, gemm_mx_run, gemm_w4a16_run, gemm_status_string,
gemm_last_error, and from gemm_moe.h gemm_moe_sort_workspace,
gemm_moe_sort, gemm_moe_dispatch, gemm_moe_combine, gemm_moe_combine_backward,
gemm_grouped_validate_desc, gemm_grouped_plan, gemm_grouped_run,
gemm_q8_store, gemm_q8_load, gemm_swiglu, gemm_swiglu_backward, and from
gemm_vocab.h gemm_embed, gemm_embed_workspace, gemm_embed_backward,
gemm_xent_validate_desc, gemm_xent_plan, gemm_xent_workspace,
gemm_xent_forward, gemm_xent_backward.  Non-OK statuses raise GemmError (except
those of gemm_validate_desc, gemm_grouped_validate_desc and
gemm_xent_validate_desc, which return the status).
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libstgemm.so")

# gemm_status_t
GEMM_OK = 0
GEMM_ERR_NULL_POINTER = 1
GEMM_ERR_INVALID_VALUE = 2
GEMM_ERR_UNSUPPORTED = 3
GEMM_ERR_MISALIGNED = 4
GEMM_ERR_NOT_SPARSE24 = 5
GEMM_ERR_DEVICE = 6
GEMM_ERR_HIP = 7

# gemm_dtype_t
DTYPES = {"f16": 1, "bf16": 2, "e4m3": 3, "e5m2": 4, "s8": 5, "f32": 6, "s32": 7,
          "e2m3": 8, "e3m2": 9, "e2m1": 10, "u4": 11, "u8": 12}
ROW_MAJOR, COL_MAJOR = 0, 1
ACT_NONE, ACT_RELU = 0, 1
# gemm_grouped_mode_t
GROUPED = {"rows": 0, "weights": 1}
# gemm_algo_t
ALGO = {"auto": 0, "tiled": 1, "generic": 2, "skinny": 3, "tiled128": 4, "tiled256": 5}

ELEM_BYTES = {"f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1, "s8": 1, "u8": 1, "f32": 4, "s32": 4}


class GemmError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (_status_name(status), message))
        self.status = status


class gemm_desc_t(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32),
        ("c_type", ctypes.c_int32), ("d_type", ctypes.c_int32),
        ("a_layout", ctypes.c_int32), ("b_layout", ctypes.c_int32),
        ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
        ("ldc", ctypes.c_int64), ("ldd", ctypes.c_int64),
        ("alpha", ctypes.c_float),
        ("has_c", ctypes.c_int32), ("has_bias", ctypes.c_int32), ("act", ctypes.c_int32),
        ("sparse_a", ctypes.c_int32), ("algo", ctypes.c_int32),
        ("block_scale", ctypes.c_int32), ("saturate", ctypes.c_int32),
    ]


class gemm_grouped_desc_t(ctypes.Structure):
    _fields_ = [
        ("mode", ctypes.c_int32), ("groups", ctypes.c_int32),
        ("rows", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32), ("d_type", ctypes.c_int32),
        ("b_layout", ctypes.c_int32), ("has_c", ctypes.c_int32), ("algo", ctypes.c_int32),
        ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldd", ctypes.c_int64),
    ]


class gemm_xent_desc_t(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("vocab", ctypes.c_int64), ("hidden", ctypes.c_int64),
        ("x_type", ctypes.c_int32), ("dx_type", ctypes.c_int32), ("dw_type", ctypes.c_int32),
        ("id_bytes", ctypes.c_int32), ("accumulate", ctypes.c_int32), ("unaligned", ctypes.c_int32),
        ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64),
        ("lddx", ctypes.c_int64), ("lddw", ctypes.c_int64),
        ("piece", ctypes.c_int64), ("scale", ctypes.c_float),
    ]


_lib = None


def load():
    """Load libstgemm.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libstgemm.so is not built (%s); run "
                           "`python -m sparse_tiled_gemm_amd.build`" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    st = ctypes.c_int
    dp = ctypes.POINTER(gemm_desc_t)
    gdp = ctypes.POINTER(gemm_grouped_desc_t)
    xdp = ctypes.POINTER(gemm_xent_desc_t)
    sz = ctypes.POINTER(ctypes.c_size_t)
    f32 = ctypes.c_float
    sig = {
        "gemm_validate_desc": (st, [dp]),
        "gemm_plan": (st, [dp, ctypes.POINTER(vp)]),
        "gemm_plan_destroy": (st, [vp]),
        "gemm_plan_describe": (st, [vp, ctypes.c_char_p, ctypes.c_size_t]),
        "gemm_run": (st, [vp, vp, vp, vp, vp, vp, vp]),
        "gemm_mx_run": (st, [vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "gemm_w4a16_run": (st, [vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "gemm_sparse24_sizes": (st, [i64, i64, i32, ctypes.POINTER(ctypes.c_size_t),
                                     ctypes.POINTER(ctypes.c_size_t)]),
        "gemm_sparse24_compress": (st, [i64, i64, i32, vp, vp, vp, vp]),
        "gemm_sparse24_compress_noalloc": (st, [i64, i64, i32, vp, vp, vp, vp]),
        "gemm_sparse24_run": (st, [vp, vp, vp, vp, vp, vp, vp, vp]),
        "gemm_moe_sort_workspace": (st, [i64, i64, i64, sz]),
        "gemm_moe_sort": (st, [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp]),
        "gemm_moe_dispatch": (st, [i64, i64, i64, i64, i32, i32, vp, vp, i64, vp, vp, vp, vp, i64,
                                   vp, vp]),
        "gemm_moe_combine": (st, [i64, i64, i64, i32, vp, vp, vp, i64, i64, vp, i64, vp]),
        "gemm_moe_combine_backward": (st, [i64, i64, i64, i32, vp, vp, vp, i64, vp, i64, i64, vp,
                                           i64, vp, vp]),
        "gemm_grouped_validate_desc": (st, [gdp]),
        "gemm_grouped_plan": (st, [gdp, ctypes.POINTER(vp)]),
        "gemm_grouped_plan_destroy": (st, [vp]),
        "gemm_grouped_plan_describe": (st, [vp, ctypes.c_char_p, ctypes.c_size_t]),
        "gemm_grouped_run": (st, [vp, vp, vp, vp, vp, vp, vp, vp]),
        "gemm_q8_store": (st, [i64, i64, i32, vp, i64, vp, vp, vp]),
        "gemm_q8_load": (st, [i64, i64, i32, vp, vp, vp, i64, vp]),
        "gemm_swiglu": (st, [i64, i64, i32, vp, i64, vp, i64, vp, vp, vp]),
        "gemm_swiglu_backward": (st, [i64, i64, i32, vp, vp, vp, i64, vp, i64, vp, i64, vp]),
        "gemm_embed": (st, [i64, i64, i64, i32, i32, i32, vp, vp, i64, vp, i64, f32, vp]),
        "gemm_embed_workspace": (st, [i64, i64, i64, sz]),
        "gemm_embed_backward": (st, [i64, i64, i64, i32, i32, i32, vp, vp, i64, vp, i64, i32, vp,
                                     f32, vp]),
        "gemm_xent_validate_desc": (st, [xdp]),
        "gemm_xent_plan": (st, [xdp, ctypes.POINTER(vp)]),
        "gemm_xent_plan_destroy": (st, [vp]),
        "gemm_xent_plan_describe": (st, [vp, ctypes.c_char_p, ctypes.c_size_t]),
        "gemm_xent_workspace": (st, [vp, sz, sz]),
        "gemm_xent_forward": (st, [vp, vp, vp, vp, vp, vp, vp, vp]),
        "gemm_xent_backward": (st, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "gemm_diag_mfma_loop": (st, [i32, i32, i64, vp, vp]),
        "gemm_status_string": (ctypes.c_char_p, [st]),
        "gemm_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _status_name(s):
    try:
        return load().gemm_status_string(s).decode()
    except Exception:
        return "status %d" % s


def gemm_status_string(status):
    return load().gemm_status_string(status).decode()


def gemm_last_error():
    return load().gemm_last_error().decode()


def _check(status):
    if status != GEMM_OK:
        raise GemmError(status, gemm_last_error())


def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        # the current stream's handle without a torch.cuda.Stream object for
        # it: 0.3 against 2.8 us per call
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_desc(M, N, K, a_type, b_type, d_type, *, c_type=None, has_c=True, has_bias=False,
              alpha=1.0, act="none", a_layout="row", b_layout="col", lda=0, ldb=0, ldc=0,
              ldd=0, sparse_a=False, algo="auto", block_scale=0, saturate=False):
    """Build a gemm_desc_t from readable arguments (type names as in DTYPES)."""
    integer = a_type in ("s8", "u8") and d_type == "s32"
    if c_type is None:
        c_type = "s32" if integer else "f32"
    d = gemm_desc_t()
    d.M, d.N, d.K = M, N, K
    d.a_type, d.b_type = DTYPES[a_type], DTYPES[b_type]
    d.c_type, d.d_type = DTYPES[c_type], DTYPES[d_type]
    d.a_layout = ROW_MAJOR if a_layout == "row" else COL_MAJOR
    d.b_layout = ROW_MAJOR if b_layout == "row" else COL_MAJOR
    d.lda, d.ldb, d.ldc, d.ldd = lda, ldb, ldc, ldd
    d.alpha = alpha
    d.has_c, d.has_bias = int(bool(has_c)), int(bool(has_bias))
    d.act = ACT_RELU if act == "relu" else ACT_NONE
    d.sparse_a = int(bool(sparse_a))
    d.algo = ALGO[algo] if isinstance(algo, str) else int(algo)
    d.block_scale = int(block_scale)
    d.saturate = int(bool(saturate))
    return d


def gemm_validate_desc(desc):
    """Returns the status code (GEMM_OK or an error); never raises."""
    return load().gemm_validate_desc(ctypes.byref(desc) if desc is not None else None)


class Plan:
    """Owns a gemm_plan_t*; released by gemm_plan_destroy / close()."""

    def __init__(self, handle, desc):
        self.handle = handle
        self.desc = desc

    def close(self):
        if self.handle:
            load().gemm_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def name(self):
        return gemm_plan_describe(self)


def gemm_plan(desc):
    L = load()
    h = ctypes.c_void_p()
    _check(L.gemm_plan(ctypes.byref(desc), ctypes.byref(h)))
    return Plan(h.value, desc)


def gemm_plan_destroy(plan):
    plan.close()


def gemm_plan_describe(plan):
    buf = ctypes.create_string_buffer(128)
    _check(load().gemm_plan_describe(plan.handle, buf, len(buf)))
    return buf.value.decode()


def gemm_run(plan, A, B, C, bias, D, stream=None):
    _check(load().gemm_run(plan.handle, _ptr(A), _ptr(B), _ptr(C), _ptr(bias), _ptr(D),
                           _stream(stream)))


def gemm_sparse24_sizes(M, K, a_type="f16"):
    vb, mb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().gemm_sparse24_sizes(M, K, DTYPES[a_type], ctypes.byref(vb), ctypes.byref(mb)))
    return vb.value, mb.value


def gemm_sparse24_compress(M, K, a_type, A, values, meta, stream=None):
    _check(load().gemm_sparse24_compress(M, K, DTYPES[a_type], _ptr(A), _ptr(values), _ptr(meta),
                                         _stream(stream)))


def gemm_sparse24_compress_noalloc(M, K, a_type, A, values, meta, stream=None):
    _check(load().gemm_sparse24_compress_noalloc(M, K, DTYPES[a_type], _ptr(A), _ptr(values),
                                                 _ptr(meta), _stream(stream)))


def gemm_sparse24_run(plan, values, meta, B, C, bias, D, stream=None):
    _check(load().gemm_sparse24_run(plan.handle, _ptr(values), _ptr(meta), _ptr(B), _ptr(C),
                                    _ptr(bias), _ptr(D), _stream(stream)))


def gemm_mx_run(plan, A, scale_a, B, scale_b, C, bias, D, stream=None):
    _check(load().gemm_mx_run(plan.handle, _ptr(A), _ptr(scale_a), _ptr(B), _ptr(scale_b),
                              _ptr(C), _ptr(bias), _ptr(D), _stream(stream)))


def gemm_w4a16_run(plan, A, B, scales, zeros, C, bias, D, stream=None):
    _check(load().gemm_w4a16_run(plan.handle, _ptr(A), _ptr(B), _ptr(scales), _ptr(zeros),
                                 _ptr(C), _ptr(bias), _ptr(D), _stream(stream)))


# ---------------------------------------------------------------- gemm_moe.h
# Argument order is the C functions'; a leading dimension of 0 means packed.
# Calls go through the extension module _pycall (csrc/pycall.c), which takes
# tensors, addresses, integers and None as they are.

class _Addresses(dict):
    """Address of each C function, looked up at its first use."""

    def __missing__(self, name):
        a = self[name] = ctypes.cast(getattr(load(), name), ctypes.c_void_p).value
        return a


_at = _Addresses()


def _call(address, *args):
    global _call
    try:
        from . import _pycall
    except ImportError as e:
        raise RuntimeError("_pycall.so is not built; run `python -m sparse_tiled_gemm_amd.build`") from e
    _call = _pycall.call  # from now on directly
    return _call(address, *args)


def _call_float(address, *args):
    """The same for a function with one float among its arguments."""
    global _call_float
    try:
        from . import _pycall
    except ImportError as e:
        raise RuntimeError("_pycall.so is not built; run `python -m sparse_tiled_gemm_amd.build`") from e
    _call_float = _pycall.call_float
    return _call_float(address, *args)


def gemm_moe_sort_workspace(tokens, topk, groups):
    """Bytes of workspace of gemm_moe_sort and gemm_moe_dispatch."""
    n = ctypes.c_size_t()
    _check(load().gemm_moe_sort_workspace(tokens, topk, groups, ctypes.byref(n)))
    return n.value


def gemm_moe_sort(tokens, topk, groups, ids, offsets, order, pos, workspace, id_bytes=4,
                  stream=None):
    _check(_call(_at["gemm_moe_sort"], tokens, topk, groups, id_bytes, ids, offsets,
                                order, pos, workspace, _stream(stream)))


def gemm_moe_dispatch(tokens, topk, groups, cols, dtype, ids, X, ldx, offsets, order, pos, Xs,
                      ldxs, workspace, id_bytes=4, stream=None):
    _check(_call(_at["gemm_moe_dispatch"], tokens, topk, groups, cols, DTYPES[dtype], id_bytes, ids,
                                    X, ldx, offsets, order, pos, Xs,
                                    ldxs, workspace, _stream(stream)))


def gemm_moe_combine(tokens, topk, cols, dtype, pos, weights, Ys, ldys, rows, Y, ldy, stream=None):
    _check(_call(_at["gemm_moe_combine"], tokens, topk, cols, DTYPES[dtype], pos, weights,
                                   Ys, ldys, rows, Y, ldy, _stream(stream)))


def gemm_moe_combine_backward(tokens, topk, cols, dtype, pos, weights, dY, lddy, Ys, ldys, rows,
                              dYs, lddys, dw, stream=None):
    _check(_call(_at["gemm_moe_combine_backward"], tokens, topk, cols, DTYPES[dtype], pos,
                                            weights, dY, lddy, Ys, ldys, rows,
                                            dYs, lddys, dw, _stream(stream)))


def make_grouped_desc(mode, rows, N, K, groups, a_type, b_type, d_type, *, b_layout=None,
                      has_c=False, lda=0, ldb=0, ldd=0, algo="auto"):
    """Build a gemm_grouped_desc_t; mode "rows" (D[r] = A[r] B_g, B_g N x K
    for b_layout "col", the default there, K x N for "row") or "weights"
    (D_g = A_g^T B_g (+ C_g), K x N)."""
    d = gemm_grouped_desc_t()
    d.mode, d.groups = GROUPED[mode], groups
    d.rows, d.N, d.K = rows, N, K
    d.a_type, d.b_type, d.d_type = DTYPES[a_type], DTYPES[b_type], DTYPES[d_type]
    if b_layout is None:
        b_layout = "col" if mode == "rows" else "row"
    d.b_layout = ROW_MAJOR if b_layout == "row" else COL_MAJOR
    d.has_c = int(bool(has_c))
    d.algo = ALGO[algo] if isinstance(algo, str) else int(algo)
    d.lda, d.ldb, d.ldd = lda, ldb, ldd
    return d


def gemm_grouped_validate_desc(desc):
    """Returns the status code (GEMM_OK or an error); never raises."""
    return load().gemm_grouped_validate_desc(ctypes.byref(desc) if desc is not None else None)


class GroupedPlan:
    """Owns a gemm_grouped_plan_t*; released by close()."""

    def __init__(self, handle, desc):
        self.handle = handle
        self.desc = desc

    def close(self):
        if self.handle:
            load().gemm_grouped_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def name(self):
        buf = ctypes.create_string_buffer(128)
        _check(load().gemm_grouped_plan_describe(self.handle, buf, len(buf)))
        return buf.value.decode()


def gemm_grouped_plan(desc):
    h = ctypes.c_void_p()
    _check(load().gemm_grouped_plan(ctypes.byref(desc), ctypes.byref(h)))
    return GroupedPlan(h.value, desc)


def gemm_grouped_run(plan, A, B, scales, offsets, C, D, stream=None):
    _check(_call(_at["gemm_grouped_run"], plan.handle, A, B, scales, offsets,
                                   C, D, _stream(stream)))


def gemm_q8_store(rows, cols, dtype, X, ldx, codes, scales, stream=None):
    _check(_call(_at["gemm_q8_store"], rows, cols, DTYPES[dtype], X, ldx, codes, scales,
                                _stream(stream)))


def gemm_q8_load(rows, cols, dtype, codes, scales, X, ldx, stream=None):
    _check(_call(_at["gemm_q8_load"], rows, cols, DTYPES[dtype], codes, scales, X, ldx,
                               _stream(stream)))


def gemm_swiglu(rows, cols, dtype, GU, ldgu, H, ldh, codes=None, scales=None, stream=None):
    _check(_call(_at["gemm_swiglu"], rows, cols, DTYPES[dtype], GU, ldgu, H, ldh, codes,
                              scales, _stream(stream)))


def gemm_swiglu_backward(rows, cols, dtype, codes, scales, dH, lddh, dGU, lddgu, H=None, ldh=0,
                         stream=None):
    _check(_call(_at["gemm_swiglu_backward"], rows, cols, DTYPES[dtype], codes, scales,
                                       dH, lddh, dGU, lddgu, H, ldh,
                                       _stream(stream)))


# ---------------------------------------------------------------- gemm_vocab.h
# Argument order is the C functions', with keywords behind; a leading
# dimension of 0 means packed.

def gemm_embed(tokens, vocab, cols, e_dtype, y_dtype, ids, E, lde, Y, ldy, scale=1.0, id_bytes=4,
               stream=None):
    _check(_call_float(_at["gemm_embed"], tokens, vocab, cols, DTYPES[e_dtype], DTYPES[y_dtype],
                       id_bytes, ids, E, lde, Y, ldy, float(scale), _stream(stream)))


def gemm_embed_workspace(tokens, vocab, cols):
    """Bytes of workspace of gemm_embed_backward."""
    n = ctypes.c_size_t()
    _check(load().gemm_embed_workspace(tokens, vocab, cols, ctypes.byref(n)))
    return n.value


def gemm_embed_backward(tokens, vocab, cols, y_dtype, e_dtype, ids, dY, lddy, dE, ldde, workspace,
                        scale=1.0, accumulate=False, id_bytes=4, stream=None):
    _check(_call_float(_at["gemm_embed_backward"], tokens, vocab, cols, DTYPES[y_dtype],
                       DTYPES[e_dtype], id_bytes, ids, dY, lddy, dE, ldde, int(bool(accumulate)),
                       workspace, float(scale), _stream(stream)))


def make_xent_desc(tokens, vocab, hidden, dtype, dx_dtype=None, dw_dtype=None, *, scale=1.0,
                   accumulate=False, id_bytes=4, unaligned=False, ldx=0, ldw=0, lddx=0, lddw=0,
                   piece=0):
    """Build a gemm_xent_desc_t; dx_dtype and dw_dtype default to dtype, that
    of X and W."""
    d = gemm_xent_desc_t()
    d.tokens, d.vocab, d.hidden = tokens, vocab, hidden
    d.x_type = DTYPES[dtype]
    d.dx_type, d.dw_type = DTYPES[dx_dtype or dtype], DTYPES[dw_dtype or dtype]
    d.id_bytes = id_bytes
    d.accumulate, d.unaligned = int(bool(accumulate)), int(bool(unaligned))
    d.ldx, d.ldw, d.lddx, d.lddw = ldx, ldw, lddx, lddw
    d.piece, d.scale = piece, scale
    return d


def gemm_xent_validate_desc(desc):
    """Returns the status code (GEMM_OK or an error); never raises."""
    return load().gemm_xent_validate_desc(ctypes.byref(desc) if desc is not None else None)


class XentPlan:
    """Owns a gemm_xent_plan_t*; released by close()."""

    def __init__(self, handle, desc):
        self.handle = handle
        self.desc = desc

    def close(self):
        if self.handle:
            load().gemm_xent_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def name(self):
        buf = ctypes.create_string_buffer(128)
        _check(load().gemm_xent_plan_describe(self.handle, buf, len(buf)))
        return buf.value.decode()


def gemm_xent_plan(desc):
    h = ctypes.c_void_p()
    _check(load().gemm_xent_plan(ctypes.byref(desc), ctypes.byref(h)))
    return XentPlan(h.value, desc)


def gemm_xent_workspace(plan):
    """Bytes of workspace of gemm_xent_forward and of gemm_xent_backward."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().gemm_xent_workspace(plan.handle, ctypes.byref(f), ctypes.byref(b)))
    return f.value, b.value


def gemm_xent_forward(plan, X, W, targets, loss, lse, workspace, stream=None):
    _check(_call(_at["gemm_xent_forward"], plan.handle, X, W, targets, loss, lse, workspace,
                 _stream(stream)))


def gemm_xent_backward(plan, X, W, targets, lse, dloss, dlse, dX, dW, workspace, stream=None):
    _check(_call(_at["gemm_xent_backward"], plan.handle, X, W, targets, lse, dloss, dlse, dX, dW,
                 workspace, _stream(stream)))


def gemm_diag_mfma_loop(kind, blocks, iters, out, stream=None):
    """Diagnostic MFMA-only loop (include/gemm_diag.h); kind 0 bf16, 1 fp8,
    2 int8 (32x32 forms), 3..5 the same types' 16x16 forms; out: a device
    float tensor of blocks * 512 elements."""
    _check(load().gemm_diag_mfma_loop(kind, blocks, iters, _ptr(out), _stream(stream)))
