"""The feed-forward block around the Walsh-Hadamard rotation, in 8 and 16 bits.

Bindings of ``include/fwt_ffn.h``: rotation with quantisation to e4m3, the
product of two quantised operands, the gated block and its gradients.  Like
the rest of the package they only marshal arguments; outputs and scratch are
torch allocations on the call's stream.  ``stream`` (the current one by
default) is one of the current device; it is not made to wait for the operands,
nor another stream for the results, but the operands' memory is kept until it
has passed the call.  The calls record nothing for autograd: operands with a
forward-mode tangent are refused, and in grad mode those that require gradients
(gated_ffn_backward takes both; its results are not differentiable themselves).

Example (one feed-forward block of a served model; weights prepared once)::

    wq, ws = qse.rotate_quantize(w_down, bits=12, scales="tile")
    h = qse.gated_ffn(x, w_gate, w_up)                  # bf16
    hq, hs = qse.rotate_quantize(h, bits=12)
    y = qse.scaled_matmul(hq, hs, wq, ws)               # h w_down^T
"""
import contextlib
import ctypes
import operator

import quantum_state_encoding_amd as _qse

__all__ = ["rotate_quantize", "scaled_matmul", "gated_ffn", "gated_ffn_backward",
           "ROTATE_MAX_BITS", "ROTATE_MAX_BITS_T", "FFN_SYMBOLS"]

ROTATE_MAX_BITS, ROTATE_MAX_BITS_T = 14, 7   # FWT_ROTATE_MAX_BITS, .._T
BLOCK = 128                                  # elements of k that share a scale

# Every symbol include/fwt_ffn.h declares.
FFN_SYMBOLS = ("fwt_rotate_quantize_workspace", "fwt_rotate_quantize",
               "fwt_scaled_matmul_workspace", "fwt_scaled_matmul", "fwt_gated_ffn_workspace",
               "fwt_gated_ffn", "fwt_gated_ffn_backward_workspace", "fwt_gated_ffn_backward")

_SCALES = {"row": 0, "tile": 1}
_ACTS = {"silu": 0, "gelu": 1}
_lib = None
# of torch, set by _load
_types = _f32 = _f8 = _floats = _halves = _gated = _raw_stream = _device = _grad_mode = None
_forward = None           # torch.autograd.forward_ad
_here = contextlib.nullcontext()


def _load():
    global _lib, _types, _f32, _f8, _floats, _halves, _gated, _raw_stream, _device, _grad_mode
    global _forward
    if _lib is None:
        import torch
        lib = _qse.load_library()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        psz = ctypes.POINTER(sz)
        lib.fwt_rotate_quantize_workspace.argtypes = [i64, i64, i32, i32, i32, psz]
        lib.fwt_rotate_quantize.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, vp, i64, vp,
                                            vp, sz, vp]
        lib.fwt_scaled_matmul_workspace.argtypes = [i64, i64, i64, i32, i32, psz]
        lib.fwt_scaled_matmul.argtypes = [vp, i64, vp, vp, i64, vp, i32, i64, i64, i64, vp, i32,
                                          i64, vp, sz, vp]
        lib.fwt_gated_ffn_workspace.argtypes = [i32, i64, i64, i64, i32, psz]
        lib.fwt_gated_ffn.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, vp, i32, i64, i64, i64,
                                      i32, vp, i32, i64, vp, sz, vp]
        lib.fwt_gated_ffn_backward_workspace.argtypes = [i64, i64, i64, psz]
        lib.fwt_gated_ffn_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i32, i64, i64,
                                               i64, i32, vp, i64, vp, i64, vp, i64, vp, sz, vp]
        for name in FFN_SYMBOLS:
            getattr(lib, name).restype = i32
        _types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
        _f32, _f8, _device = torch.float32, torch.float8_e4m3fn, torch.cuda.current_device
        _halves = (torch.bfloat16, torch.float16)
        _floats, _gated = _halves + (_f32,), _halves + (_f8,)
        _raw_stream = torch._C._cuda_getCurrentRawStream   # the handle alone: no Stream object
        _grad_mode, _forward = torch.is_grad_enabled, torch.autograd.forward_ad
        _lib = lib
    return _lib


def _matrix(t, name, dtypes, dev):
    """Checks a 2-d operand; returns its rows, columns and row stride."""
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s" % (name, " or ".join(str(d) for d in dtypes)))
    if t.get_device() != dev:
        raise ValueError("%s must be a tensor of the current device" % name)
    shape, strides = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError("%s must have two dimensions" % name)
    rows, cols = shape
    if strides[1] != 1 and cols > 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    if rows > 1:
        ld = strides[0]
        if ld < cols:
            raise ValueError("the rows of %s overlap" % name)
        return rows, cols, ld
    return rows, cols, -(-cols // 16) * 16


def _scales_of(s, name, dev, blocks, rows, kinds):
    """Checks a scale array; returns its kind ("row" or "tile")."""
    if s.dtype is not _f32 or not s.is_contiguous():
        raise ValueError("%s must be a contiguous float32 matrix" % name)
    if s.get_device() != dev:
        raise ValueError("%s must be a tensor of the current device" % name)
    shape = tuple(s.shape)
    for kind in kinds:
        if shape == (blocks, rows if kind == "row" else -(-rows // BLOCK)):
            return kind
    raise ValueError("%s must have shape %s, not %s" % (name, " or ".join(
        str((blocks, rows if k == "row" else -(-rows // BLOCK))) for k in kinds), shape))


def _on(stream, dev, *tensors):
    """(stream handle, a context in which torch allocates for that stream).
    The memory of the call's tensors is kept until a given stream has passed
    the call."""
    if stream is None:
        return _raw_stream(dev), _here
    import torch
    if stream.device_index != dev:
        raise ValueError("stream must be one of the current device")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _result(out, name, dev, rows, cols, dtype, like):
    """The output tensor and its row stride."""
    if out is None:
        return like.new_empty((rows, cols), dtype=dtype), cols
    r, c, ld = _matrix(out, name, (dtype,), dev)
    if (r, c) != (rows, cols):
        raise ValueError("%s must have shape %s" % (name, (rows, cols)))
    return out, ld


def _out_dtype(out_dtype, out):
    dtype = out_dtype or (_floats[0] if out is None else out.dtype)
    if dtype not in _floats:
        raise ValueError("out_dtype must be bfloat16, float16 or float32")
    return dtype


def _no_tangents(what, tensors):
    """Refuses operands with a tangent, in any grad mode: the results would have
    none."""
    # (outside a level, asking each tensor would take 0.4 us)
    if getattr(_forward, "_current_level", 0) >= 0:
        for t in tensors:
            if t is not None and _forward.unpack_dual(t).tangent is not None:
                raise ValueError("%s hands no tangents on: call it with detached tensors" % what)


def _no_graph(what, *tensors):
    """Refuses operands whose gradients would be lost: the calls record
    nothing for autograd."""
    _no_tangents(what, tensors)
    if _grad_mode():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("%s records no graph: call it under torch.no_grad() or with "
                                 "detached tensors (gated_ffn_backward has gated_ffn's "
                                 "gradients)" % what)


def _written(out):
    """Tells autograd that `out`, which may be saved for a backward pass, has
    other values now."""
    if out is not None:
        import torch
        torch.autograd.graph.increment_version(out)


def _raise(status, what):
    if status != _qse.FWT_OK:
        raise _qse.FwtError(status, what)


def _act(act):
    if act not in _ACTS:
        raise ValueError("act must be 'silu' or 'gelu'")
    return _ACTS[act]


def _scratch(nbytes, like):
    import torch
    if not nbytes:
        return None, None
    ws = like.new_empty(nbytes, dtype=torch.uint8)
    return ws, ws.data_ptr()


def _may_share(m, n, k):
    """Whether a product of these sizes could want scratch: only where few
    tiles (of 64 x 64 and more) have many steps."""
    return m > 16 and k >= 512 and m * n <= 1 << 21


def _current():
    """The current device, or the reason that there is none."""
    try:
        return _device()
    except Exception as e:      # torch has no device to ask
        raise ValueError("no current device: %s" % e)


def rotate_quantize(x, bits=0, scales="row", transpose=False, stream=None):
    """e4m3 codes and scales of ``x (I (x) H_bits) 2^(-bits/2)``.

    ``x`` is (m, k), or (k, m) with ``transpose``; bf16, f16 or f32.
    ``scales`` "row" gives one scale for 128 elements of a row, shape
    (ceil(k/128), m); "tile" one for 128 rows of them, shape
    (ceil(k/128), ceil(m/128)).  Returns (codes, scales): codes are
    float8_e4m3fn of shape (m, k), in rows padded with zeros to a multiple of
    16 bytes.  See fwt_rotate_quantize.
    """
    lib = _lib or _load()
    if scales not in _SCALES:
        raise ValueError("scales must be 'row' or 'tile'")
    bits = operator.index(bits)
    if not 0 <= bits <= ROTATE_MAX_BITS:
        _raise(_qse.FWT_EINVAL, "rotate_quantize: bits %d" % bits)
    dev = _current()
    m, k, ld = _matrix(x, "x", _floats, dev)
    _no_graph("rotate_quantize", x)
    if transpose:
        m, k = k, m
    kind, t = _SCALES[scales], 1 if transpose else 0
    need = 0
    if kind and bits > ROTATE_MAX_BITS_T:
        size = ctypes.c_size_t(0)
        _raise(lib.fwt_rotate_quantize_workspace(m, k, bits, kind, t, ctypes.byref(size)),
               "fwt_rotate_quantize_workspace")
        need = size.value
    handle, where = _on(stream, dev, x)
    with where:
        ldq = -(-k // 16) * 16
        codes = x.new_empty((m, ldq), dtype=_f8)
        s = x.new_empty((-(-k // BLOCK), -(-m // BLOCK) if kind else m), dtype=_f32)
        ws, wp = _scratch(need, x)
    _raise(lib.fwt_rotate_quantize(x.data_ptr(), _types[x.dtype], m, k, ld, t, bits, kind,
                                   codes.data_ptr(), ldq, s.data_ptr(), wp, need, handle),
           "fwt_rotate_quantize")
    return (codes if ldq == k else codes[:, :k]), s


def scaled_matmul(a, a_scales, b, b_scales, out_dtype=None, out=None, stream=None):
    """``a b^T`` of e4m3 codes: a (m, k) with row scales, b (n, k) with row
    or tile scales (told by their shape).  ``out_dtype``: bfloat16 (default,
    twice the rate: its products lose what bfloat16 cannot show), float16 or
    float32.  See fwt_scaled_matmul."""
    lib = _lib or _load()
    dev = _current()
    m, k, lda = _matrix(a, "a", (_f8,), dev)
    n, kb, ldb = _matrix(b, "b", (_f8,), dev)
    if k != kb:
        raise ValueError("a and b must have the same number of columns")
    nblocks = -(-k // BLOCK)
    _scales_of(a_scales, "a_scales", dev, nblocks, m, ("row",))
    kind = _scales_of(b_scales, "b_scales", dev, nblocks, n, ("tile", "row"))
    dtype = _out_dtype(out_dtype, out)
    _no_graph("scaled_matmul", a, a_scales, b, b_scales, out)
    need = 0
    if _may_share(m, n, k):
        size = ctypes.c_size_t(0)
        _raise(lib.fwt_scaled_matmul_workspace(m, n, k, _SCALES[kind], _types[dtype],
                                               ctypes.byref(size)), "fwt_scaled_matmul_workspace")
        need = size.value
    handle, where = _on(stream, dev, a, a_scales, b, b_scales, out)
    with where:
        c, ldc = _result(out, "out", dev, m, n, dtype, a)
        ws, wp = _scratch(need, a)
    _raise(lib.fwt_scaled_matmul(a.data_ptr(), lda, a_scales.data_ptr(), b.data_ptr(), ldb,
                                 b_scales.data_ptr(), _SCALES[kind], m, n, k, c.data_ptr(),
                                 _types[dtype], ldc, wp, need, handle), "fwt_scaled_matmul")
    _written(out)
    return c


def gated_ffn(x, gate, up, act="silu", x_scales=None, gate_scales=None, up_scales=None,
              out_dtype=None, out=None, stream=None):
    """``act(x gate^T) * (x up^T)`` for x (m, k), gate and up (n, k).

    bf16 or f16 operands give an output of their dtype.  e4m3 codes come with
    ``x_scales`` ("row") and ``gate_scales``/``up_scales`` ("tile") and give
    ``out_dtype`` (bfloat16 by default).  ``act``: "silu" or "gelu".  See
    fwt_gated_ffn.
    """
    lib = _lib or _load()
    dev = _current()
    m, k, ldx = _matrix(x, "x", _gated, dev)
    n, kg, ldg = _matrix(gate, "gate", (x.dtype,), dev)
    nu, ku, ldu = _matrix(up, "up", (x.dtype,), dev)
    if kg != k or ku != k or nu != n:
        raise ValueError("gate and up must have shape (n, %d)" % k)
    sp = (None, None, None)
    if x.dtype is _f8:
        if x_scales is None or gate_scales is None or up_scales is None:
            raise ValueError("e4m3 operands need x_scales, gate_scales and up_scales")
        nblocks = -(-k // BLOCK)
        _scales_of(x_scales, "x_scales", dev, nblocks, m, ("row",))
        _scales_of(gate_scales, "gate_scales", dev, nblocks, n, ("tile",))
        _scales_of(up_scales, "up_scales", dev, nblocks, n, ("tile",))
        sp = (x_scales.data_ptr(), gate_scales.data_ptr(), up_scales.data_ptr())
        dtype = _out_dtype(out_dtype, out)
    else:
        if x_scales is not None or gate_scales is not None or up_scales is not None:
            raise ValueError("scales belong to e4m3 operands")
        dtype = out_dtype or x.dtype
        if dtype is not x.dtype:
            raise ValueError("the output has the operands' dtype")
    code = _act(act)
    _no_graph("gated_ffn", x, gate, up, x_scales, gate_scales, up_scales, out)
    need = 0
    if _may_share(m, n, k):
        size = ctypes.c_size_t(0)
        _raise(lib.fwt_gated_ffn_workspace(_types[x.dtype], m, n, k, _types[dtype],
                                           ctypes.byref(size)), "fwt_gated_ffn_workspace")
        need = size.value
    handle, where = _on(stream, dev, x, gate, up, x_scales, gate_scales, up_scales, out)
    with where:
        h, ldh = _result(out, "out", dev, m, n, dtype, x)
        ws, wp = _scratch(need, x)
    _raise(lib.fwt_gated_ffn(x.data_ptr(), ldx, sp[0], gate.data_ptr(), ldg, sp[1],
                             up.data_ptr(), ldu, sp[2], _types[x.dtype], m, n, k, code,
                             h.data_ptr(), _types[dtype], ldh, wp, need, handle),
           "fwt_gated_ffn")
    _written(out)
    return h


def gated_ffn_backward(x, gate, up, grad, act="silu", stream=None):
    """Gradients (dx, dgate, dup) of ``gated_ffn`` on bf16 or f16 operands
    for ``grad``, that of its output (m, n).  See fwt_gated_ffn_backward."""
    lib = _lib or _load()
    dev = _current()
    m, k, ldx = _matrix(x, "x", _halves, dev)
    n, kg, ldg = _matrix(gate, "gate", (x.dtype,), dev)
    nu, ku, ldu = _matrix(up, "up", (x.dtype,), dev)
    mg, ng, ldd = _matrix(grad, "grad", (x.dtype,), dev)
    if kg != k or ku != k or nu != n:
        raise ValueError("gate and up must have shape (n, %d)" % k)
    if (mg, ng) != (m, n):
        raise ValueError("grad must have shape %s" % ((m, n),))
    code = _act(act)
    size = ctypes.c_size_t(0)
    _raise(lib.fwt_gated_ffn_backward_workspace(m, n, k, ctypes.byref(size)),
           "fwt_gated_ffn_backward_workspace")
    handle, where = _on(stream, dev, x, gate, up, grad)
    with where:
        dx = x.new_empty((m, k))
        dgate = x.new_empty((n, k))
        dup = x.new_empty((n, k))
        ws, wp = _scratch(size.value, x)
    _raise(lib.fwt_gated_ffn_backward(x.data_ptr(), ldx, gate.data_ptr(), ldg, up.data_ptr(),
                                      ldu, grad.data_ptr(), ldd, _types[x.dtype], m, n, k, code,
                                      dx.data_ptr(), k, dgate.data_ptr(), k, dup.data_ptr(), k,
                                      wp, size.value, handle), "fwt_gated_ffn_backward")
    return dx, dgate, dup
