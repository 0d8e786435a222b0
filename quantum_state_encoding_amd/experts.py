"""8-bit integer products and products grouped by expert, around the
Walsh-Hadamard rotation.

Bindings of ``include/fwt_experts.h``: rotation with quantisation to 8-bit
integers (a scale for each row), the product of two such operands, and the
products of rows that are sorted by expert, with their gradients.  Arguments,
streams and scratch are as in ``ffn``: outputs are torch allocations on the
call's stream, nothing waits, the operands' memory is kept until a given stream
has passed the call, and operands with a forward-mode tangent are refused, and in
grad mode those that require gradients, since the calls record no graph
(grouped_matmul_backward takes both; its results are not differentiable
themselves).

Example (the down projection of a served model's experts, 8-bit)::

    wq, ws = qse.rotate_quantize_int8(w_down.view(experts * n, k), bits=10)
    hq, hs = qse.rotate_quantize_int8(h, bits=10)       # h: tokens by expert
    y = qse.grouped_matmul(hq, wq.view(experts, n, k), ends, x_scales=hs,
                           w_scales=ws.view(experts, n))
"""
import ctypes
import operator

import quantum_state_encoding_amd as _qse

from . import ffn as _ffn

__all__ = ["rotate_quantize_int8", "int8_matmul", "grouped_matmul", "grouped_matmul_backward",
           "EXPERTS_SYMBOLS", "INT8"]

INT8 = 5                  # FWT_INT8

# Every symbol include/fwt_experts.h declares.
EXPERTS_SYMBOLS = ("fwt_rotate_quantize_int8", "fwt_int8_matmul_workspace", "fwt_int8_matmul",
                   "fwt_grouped_matmul_workspace", "fwt_grouped_matmul_workspace_for",
                   "fwt_grouped_matmul", "fwt_grouped_matmul_backward_workspace",
                   "fwt_grouped_matmul_backward_workspace_for", "fwt_grouped_matmul_backward")

_lib = None
# of torch, set by _load
_types = _i8 = _i32 = _floats = _halves = _f32 = None


def _load():
    global _lib, _types, _i8, _i32, _floats, _halves, _f32
    if _lib is None:
        import torch
        lib = _ffn._load()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        psz = ctypes.POINTER(sz)
        lib.fwt_rotate_quantize_int8.argtypes = [vp, i32, i64, i64, i64, i32, vp, i64, vp, vp]
        lib.fwt_int8_matmul_workspace.argtypes = [i64, i64, i64, i32, psz]
        lib.fwt_int8_matmul.argtypes = [vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, i32, i64, vp,
                                        sz, vp]
        lib.fwt_grouped_matmul_workspace.argtypes = [i32, i64, i64, i64, i64, psz]
        lib.fwt_grouped_matmul_workspace_for.argtypes = [vp, i64, vp, i64, i64, i64, i32, i64, i64,
                                                         i64, psz]
        lib.fwt_grouped_matmul.argtypes = [vp, i64, vp, vp, i64, i64, vp, vp, i64, i32, i64, i64,
                                           i64, vp, i32, i64, i32, vp, sz, vp]
        lib.fwt_grouped_matmul_backward_workspace.argtypes = [i64, i64, i64, i64, psz]
        lib.fwt_grouped_matmul_backward_workspace_for.argtypes = [
            vp, i64, vp, i64, i64, i64, vp, i64, i64, i64, i64, i32, i32, psz]
        lib.fwt_grouped_matmul_backward.argtypes = [vp, i64, vp, i64, i64, vp, i64, vp, i64, i32,
                                                    i64, i64, i64, vp, i64, vp, i64, i64, vp, sz,
                                                    vp]
        for name in EXPERTS_SYMBOLS:
            getattr(lib, name).restype = i32
        _types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: INT8}
        _i8, _i32, _f32 = torch.int8, torch.int32, torch.float32
        _halves = (torch.bfloat16, torch.float16)
        _floats = _halves + (_f32,)
        _lib = lib
    return _lib


def _scales(s, name, dev, shape):
    """Checks the scales of an operand's rows."""
    if s.dtype is not _f32 or not s.is_contiguous():
        raise ValueError("%s must be contiguous float32" % name)
    if s.get_device() != dev:
        raise ValueError("%s must be a tensor of the current device" % name)
    if tuple(s.shape) != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, shape, tuple(s.shape)))


def _weights(w, name, dtype, dev, k):
    """Checks the experts' weights; returns experts, n and the strides of a
    row and of an expert."""
    if w.dtype is not dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if w.get_device() != dev:
        raise ValueError("%s must be a tensor of the current device" % name)
    shape, strides = w.shape, w.stride()
    if len(shape) != 3 or shape[2] != k or shape[0] < 1:
        raise ValueError("%s must have shape (experts, n, %d)" % (name, k))
    experts, n, _ = shape
    if strides[2] != 1 and k > 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    ld = strides[1] if n > 1 else -(-k // 16) * 16
    if ld < k:
        raise ValueError("the rows of %s overlap" % name)
    between = strides[0] if experts > 1 else 0
    if experts > 1 and n and between < (n - 1) * ld + k:
        raise ValueError("the experts of %s overlap" % name)
    return experts, n, ld, between


def _check_ends(ends, dev, experts):
    if ends.dtype is not _i32 or ends.dim() != 1 or not ends.is_contiguous():
        raise ValueError("ends must be a contiguous int32 vector")
    if ends.get_device() != dev:
        raise ValueError("ends must be a tensor of the current device")
    if ends.shape[0] != experts:
        raise ValueError("ends must have one element for each of the %d experts" % experts)


def _no_graph(what, *tensors):
    _ffn._no_tangents(what, tensors)
    if _ffn._grad_mode():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("%s records no graph: call it under torch.no_grad() or with "
                                 "detached tensors (grouped_matmul_backward has "
                                 "grouped_matmul's gradients)" % what)


def _out_dtype(out_dtype, out):
    dtype = out_dtype or (_floats[0] if out is None else out.dtype)
    if dtype not in _floats:
        raise ValueError("out_dtype must be bfloat16, float16 or float32")
    return dtype


def _may_share(m, n, k, dtype):
    """Whether a grouped product could want scratch for shares of its steps.  Up to 16
    rows run in strips until these take longer than the second launch that shares need
    (calls, microseconds without and with: bf16 m 1 e 1 n 64 k 16384 20.0 and 15.4, m 2
    e 2 n 256 k 8192 12.0 and 15.4; kernels: int8 m 12 e 1 n 213 k 32608 21.3 and 10.3,
    m 3 e 29 n 346 k 11328 8.0 and 10.9)."""
    if m > 16:
        return _ffn._may_share(m, n, k)
    return k >= (28672 if dtype is _i8 else 14336) and m * n <= 1 << 21


def rotate_quantize_int8(x, bits=0, stream=None):
    """8-bit integers and scales of ``x (I (x) H_bits) 2^(-bits/2)``.

    ``x`` is (m, k), bf16, f16 or f32: tokens of activations, or channels of
    weights.  Returns (codes, scales): codes are int8 of shape (m, k), in rows
    padded with zeros to a multiple of 16 bytes, scales float32 of shape (m,).
    See fwt_rotate_quantize_int8.
    """
    lib = _lib or _load()
    bits = operator.index(bits)
    if not 0 <= bits <= _ffn.ROTATE_MAX_BITS:
        _ffn._raise(_qse.FWT_EINVAL, "rotate_quantize_int8: bits %d" % bits)
    dev = _ffn._current()
    m, k, ld = _ffn._matrix(x, "x", _floats, dev)
    _no_graph("rotate_quantize_int8", x)
    handle, where = _ffn._on(stream, dev, x)
    with where:
        ldq = -(-k // 16) * 16
        codes = x.new_empty((m, ldq), dtype=_i8)
        s = x.new_empty((m,), dtype=_f32)
    _ffn._raise(lib.fwt_rotate_quantize_int8(x.data_ptr(), _types[x.dtype], m, k, ld, bits,
                                             codes.data_ptr(), ldq, s.data_ptr(), handle),
                "fwt_rotate_quantize_int8")
    return (codes if ldq == k else codes[:, :k]), s


def int8_matmul(a, a_scales, b, b_scales, out_dtype=None, out=None, stream=None):
    """``a b^T`` of 8-bit integers times their rows' scales: a (m, k) with
    a_scales (m,), b (n, k) with b_scales (n,).  The sums are exact.
    ``out_dtype``: bfloat16 (default), float16 or float32.  See
    fwt_int8_matmul."""
    lib = _lib or _load()
    dev = _ffn._current()
    m, k, lda = _ffn._matrix(a, "a", (_i8,), dev)
    n, kb, ldb = _ffn._matrix(b, "b", (_i8,), dev)
    if k != kb:
        raise ValueError("a and b must have the same number of columns")
    _scales(a_scales, "a_scales", dev, (m,))
    _scales(b_scales, "b_scales", dev, (n,))
    dtype = _out_dtype(out_dtype, out)
    _no_graph("int8_matmul", a_scales, b_scales, out)
    need = 0
    if _ffn._may_share(m, n, k):
        size = ctypes.c_size_t(0)
        _ffn._raise(lib.fwt_int8_matmul_workspace(m, n, k, _types[dtype], ctypes.byref(size)),
                    "fwt_int8_matmul_workspace")
        need = size.value
    handle, where = _ffn._on(stream, dev, a, a_scales, b, b_scales, out)
    with where:
        c, ldc = _ffn._result(out, "out", dev, m, n, dtype, a)
        ws, wp = _ffn._scratch(need, a)
    _ffn._raise(lib.fwt_int8_matmul(a.data_ptr(), lda, a_scales.data_ptr(), b.data_ptr(), ldb,
                                    b_scales.data_ptr(), m, n, k, c.data_ptr(), _types[dtype],
                                    ldc, wp, need, handle), "fwt_int8_matmul")
    _ffn._written(out)
    return c


def grouped_matmul(x, w, ends, x_scales=None, w_scales=None, out_dtype=None, out=None,
                   stream=None):
    """``x[i] w[e]^T`` for the rows i of expert e: x (m, k) sorted by expert,
    w (experts, n, k).

    ``ends``: int32 of shape (experts,) on the device; expert e has the rows
    from ends[e - 1] (0 for the first) up to ends[e].  Rows from ends[-1] on
    belong to none: they are zeros in a new output, and left as they were in
    ``out``.  bf16 or f16 operands give an output of their dtype.  int8 codes
    come with ``x_scales`` (m,) and ``w_scales`` (experts, n) and give
    ``out_dtype`` (bfloat16 by default).  See fwt_grouped_matmul.
    """
    lib = _lib or _load()
    dev = _ffn._current()
    m, k, ldx = _ffn._matrix(x, "x", _halves + (_i8,), dev)
    experts, n, ldw, between = _weights(w, "w", x.dtype, dev, k)
    _check_ends(ends, dev, experts)
    sp = (None, None)
    if x.dtype is _i8:
        if x_scales is None or w_scales is None:
            raise ValueError("int8 operands need x_scales and w_scales")
        _scales(x_scales, "x_scales", dev, (m,))
        _scales(w_scales, "w_scales", dev, (experts, n))
        sp = (x_scales.data_ptr(), w_scales.data_ptr())
        dtype = _out_dtype(out_dtype, out)
    else:
        if x_scales is not None or w_scales is not None:
            raise ValueError("scales belong to int8 operands")
        dtype = out_dtype or x.dtype
        if dtype is not x.dtype:
            raise ValueError("the output has the operands' dtype")
    _no_graph("grouped_matmul", x, w, x_scales, w_scales, out)
    need = 0
    if _may_share(m, n, k, x.dtype) or (k % 8 and x.dtype is not _i8):
        size = ctypes.c_size_t(0)
        _ffn._raise(lib.fwt_grouped_matmul_workspace(_types[x.dtype], experts, m, n, k,
                                                     ctypes.byref(size)),
                    "fwt_grouped_matmul_workspace")
        if k % 8 and size.value >= 2 * (m + experts * n) * k:      # (copies may be in it)
            _ffn._raise(lib.fwt_grouped_matmul_workspace_for(
                x.data_ptr(), ldx, w.data_ptr(), ldw, between, experts, _types[x.dtype], m, n, k,
                ctypes.byref(size)), "fwt_grouped_matmul_workspace_for")
        need = size.value
    handle, where = _ffn._on(stream, dev, x, w, ends, x_scales, w_scales, out)
    with where:
        y, ldy = _ffn._result(out, "out", dev, m, n, dtype, x)
        ws, wp = _ffn._scratch(need, x)
    _ffn._raise(lib.fwt_grouped_matmul(x.data_ptr(), ldx, sp[0], w.data_ptr(), ldw, between,
                                       sp[1], ends.data_ptr(), experts, _types[x.dtype], m, n, k,
                                       y.data_ptr(), _types[dtype], ldy, 1 if out is None else 0,
                                       wp, need, handle), "fwt_grouped_matmul")
    _ffn._written(out)
    return y


def grouped_matmul_backward(x, w, ends, grad, stream=None):
    """Gradients (dx, dw) of ``grouped_matmul`` on bf16 or f16 operands for
    ``grad``, that of its output (m, n).  Rows of no expert and experts without
    rows get zeros.  See fwt_grouped_matmul_backward."""
    lib = _lib or _load()
    dev = _ffn._current()
    m, k, ldx = _ffn._matrix(x, "x", _halves, dev)
    experts, n, ldw, between = _weights(w, "w", x.dtype, dev, k)
    _check_ends(ends, dev, experts)
    mg, ng, ldd = _ffn._matrix(grad, "grad", (x.dtype,), dev)
    if (mg, ng) != (m, n):
        raise ValueError("grad must have shape %s" % ((m, n),))
    size = ctypes.c_size_t(0)
    _ffn._raise(lib.fwt_grouped_matmul_backward_workspace(experts, m, n, k, ctypes.byref(size)),
                "fwt_grouped_matmul_backward_workspace")
    copies = (2 * (m + experts * n) * k if k % 8 else 0) + (2 * m * n if n % 8 else 0)
    if copies and size.value >= copies:                  # (they may be in it)
        _ffn._raise(lib.fwt_grouped_matmul_backward_workspace_for(
            x.data_ptr(), ldx, w.data_ptr(), ldw, between, experts, grad.data_ptr(), ldd, m, n, k,
            1, 1, ctypes.byref(size)), "fwt_grouped_matmul_backward_workspace_for")
    handle, where = _ffn._on(stream, dev, x, w, ends, grad)
    with where:
        dx = x.new_empty((m, k))
        dw = x.new_empty((experts, n, k))
        ws, wp = _ffn._scratch(size.value, x)
    _ffn._raise(lib.fwt_grouped_matmul_backward(x.data_ptr(), ldx, w.data_ptr(), ldw, between,
                                                ends.data_ptr(), experts, grad.data_ptr(), ldd,
                                                _types[x.dtype], m, n, k, dx.data_ptr(), k,
                                                dw.data_ptr(), k, n * k, wp, size.value, handle),
                "fwt_grouped_matmul_backward")
    return dx, dw
