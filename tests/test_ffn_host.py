"""Host-side tests of the feed-forward entry points (no GPU): exported
symbols, workspace sizes, and the refusals that come before any HIP call."""
import ctypes
import os
import re

import pytest

import quantum_state_encoding_amd as qse
from quantum_state_encoding_amd import ffn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EALIGN, EUNSUPPORTED = 0, -1, -2, -3
BF16, F16, F32, E4M3 = 0, 1, 2, 3
P = 0x10000          # an aligned address that is never read: refusals come first


@pytest.fixture(scope="module")
def L(lib):
    pytest.importorskip("torch")
    return ffn._load()


def test_header_declares_the_binding_symbols(lib):
    text = open(os.path.join(ROOT, "include", "fwt_ffn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(fwt_[a-z_]+)\s*\(", text)))
    assert names == sorted(ffn.FFN_SYMBOLS)
    for name in names:
        assert hasattr(lib, name)
    head = open(os.path.join(ROOT, "include", "fwt_ffn.h")).read()
    assert "FWT_ROTATE_MAX_BITS %d" % qse.ffn.ROTATE_MAX_BITS in head
    assert "FWT_ROTATE_MAX_BITS_T %d" % qse.ffn.ROTATE_MAX_BITS_T in head


def rotate(L, x=P, dtype=BF16, m=4, k=256, ldx=256, t=0, bits=3, scales=0, q=P, ldq=256, s=P,
           ws=None, wsb=0):
    return L.fwt_rotate_quantize(x, dtype, m, k, ldx, t, bits, scales, q, ldq, s, ws, wsb, None)


def test_rotate_refusals(L):
    assert rotate(L, m=0) == OK
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(dtype=E4M3), dict(dtype=9),
                dict(m=-1), dict(k=0), dict(k=-5), dict(bits=-1), dict(bits=15),
                dict(bits=8, t=1), dict(scales=2), dict(k=252, bits=3), dict(k=300, bits=9),
                dict(bits=8, scales=1), dict(bits=8, scales=1, ws=P, wsb=8), dict(m=1 << 31)):
        assert rotate(L, **bad) == EINVAL, bad
    for bad in (dict(q=P + 8), dict(ldq=264), dict(bits=8, scales=1, ws=P + 4, wsb=1 << 20)):
        assert rotate(L, **bad) == EALIGN, bad
    far = dict(x=1 << 40, q=1 << 42, s=1 << 44)
    for bad in (dict(m=1 << 29, k=128, ldx=128, ldq=128), dict(m=1 << 20, k=1 << 16, bits=0),
                dict(m=(65535 * 128) + 1, scales=1), dict(m=(65535 * 128) + 1, t=1, ldx=1 << 30),
                dict(m=1, k=1 << 29, scales=1)):
        assert rotate(L, **dict(far, **bad)) == EUNSUPPORTED, bad
    for ldx in (-1, 255, (1 << 40) + 1, (1 << 63) - 1, -(1 << 63)):
        assert rotate(L, **dict(far, ldx=ldx)) == EINVAL
    # written arrays that overlap, or overlap what is read
    assert rotate(L, q=P, s=P + 64) == EINVAL
    assert rotate(L, x=P, q=P) == EINVAL


def test_rotate_workspace(L):
    def size(m, k, bits, scales, t=0):
        out = ctypes.c_size_t(77)
        st = L.fwt_rotate_quantize_workspace(m, k, bits, scales, t, ctypes.byref(out))
        return st, out.value
    assert size(100, 4096, 12, 0) == (OK, 0)
    assert size(100, 4096, 7, 1) == (OK, 0)
    assert size(100, 4096, 8, 1) == (OK, 100 * 32 * 4)
    assert size(100, 4352, 8, 1) == (OK, 100 * 34 * 4)
    assert size(0, 4096, 8, 1) == (OK, 0)
    assert size(100, 4096, 15, 0)[0] == EINVAL
    assert size(100, 4096, 8, 0, 1)[0] == EINVAL
    assert L.fwt_rotate_quantize_workspace(1, 1, 0, 0, 0, None) == EINVAL


def matmul(L, a=P, lda=256, sa=2 * P, b=3 * P, ldb=256, sb=4 * P, kind=0, m=4, n=8, k=256,
           c=5 * P, ctype=BF16, ldc=8, ws=None, wsb=0):
    return L.fwt_scaled_matmul(a, lda, sa, b, ldb, sb, kind, m, n, k, c, ctype, ldc, ws, wsb,
                               None)


def test_matmul_refusals(L):
    assert matmul(L, m=0) == OK and matmul(L, n=0) == OK
    for bad in (dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(c=None),
                dict(kind=2), dict(m=-1), dict(n=-1), dict(k=0), dict(ctype=E4M3),
                dict(ctype=7), dict(c=P), dict(c=3 * P + 16), dict(c=4 * P)):
        assert matmul(L, **bad) == EINVAL, bad
    for bad in (dict(a=P + 1), dict(b=P + 8), dict(lda=264), dict(ldb=257)):
        assert matmul(L, **bad) == EALIGN, bad
    assert matmul(L, lda=1 << 23) == EUNSUPPORTED
    assert matmul(L, ldb=1 << 23) == EUNSUPPORTED
    assert matmul(L, m=1 << 20, n=1 << 15, ldc=1 << 15) == EUNSUPPORTED
    assert matmul(L, m=1 << 29, n=1) == EUNSUPPORTED
    for ld in (-16, 240, -(1 << 63)):
        assert matmul(L, lda=ld) == EINVAL
    for ld in (7, -8, (1 << 63) - 1):
        assert matmul(L, ldc=ld) == EINVAL


def gated(L, x=P, ldx=64, xs=None, g=2 * P, ldg=64, gs=None, u=3 * P, ldu=64, us=None,
          dtype=BF16, m=4, n=8, k=64, act=0, h=4 * P, htype=BF16, ldh=8, ws=None, wsb=0):
    return L.fwt_gated_ffn(x, ldx, xs, g, ldg, gs, u, ldu, us, dtype, m, n, k, act, h, htype,
                           ldh, ws, wsb, None)


def test_gated_refusals(L):
    assert gated(L, m=0) == OK and gated(L, n=0) == OK
    f8 = dict(dtype=E4M3, xs=5 * P, gs=6 * P, us=7 * P)
    for bad in (dict(x=None), dict(g=None), dict(u=None), dict(h=None), dict(dtype=F32),
                dict(htype=F16), dict(act=2), dict(k=0), dict(m=-1), dict(xs=5 * P),
                dict(dtype=E4M3), dict(f8, gs=None), dict(f8, htype=E4M3), dict(h=P),
                dict(h=2 * P)):
        assert gated(L, **bad) == EINVAL, bad
    assert gated(L, **dict(f8, x=P + 4)) == EALIGN
    assert gated(L, **dict(f8, ldu=72)) == EALIGN
    assert gated(L, ldx=1 << 22) == EUNSUPPORTED
    assert gated(L, ldg=1 << 22) == EUNSUPPORTED
    assert gated(L, m=1 << 20, n=1 << 15, ldh=1 << 15) == EUNSUPPORTED


def backward(L, x=P, ldx=64, g=2 * P, ldg=64, u=3 * P, ldu=64, dh=4 * P, lddh=8, dtype=BF16,
             m=4, n=8, k=64, act=0, dx=5 * P, lddx=64, dg=6 * P, lddg=64, du=7 * P, lddu=64,
             ws=8 * P, wsb=1 << 20):
    return L.fwt_gated_ffn_backward(x, ldx, g, ldg, u, ldu, dh, lddh, dtype, m, n, k, act, dx,
                                    lddx, dg, lddg, du, lddu, ws, wsb, None)


def test_backward_refusals(L):
    assert backward(L, m=0, n=0) == OK
    for bad in (dict(x=None), dict(g=None), dict(u=None), dict(dh=None), dict(dx=None),
                dict(dg=None), dict(du=None), dict(ws=None), dict(wsb=64), dict(dtype=E4M3),
                dict(dtype=F32), dict(act=3), dict(k=0), dict(n=-1), dict(dx=P), dict(dg=7 * P),
                dict(ws=4 * P), dict(m=0, dg=None), dict(n=0, dx=None)):
        assert backward(L, **bad) == EINVAL, bad
    assert backward(L, ws=8 * P + 8) == EALIGN
    assert backward(L, ldx=1 << 22) == EUNSUPPORTED
    assert backward(L, m=1 << 20, k=1 << 15, ldx=1 << 15, wsb=1 << 40) == EUNSUPPORTED
    assert backward(L, n=1 << 21, wsb=1 << 40) == EUNSUPPORTED
    out = ctypes.c_size_t()
    assert L.fwt_gated_ffn_backward_workspace(4, 8, 64, ctypes.byref(out)) == OK
    assert out.value > 0 and out.value % 2 == 0
    assert L.fwt_gated_ffn_backward_workspace(0, 8, 64, ctypes.byref(out)) == OK
    assert out.value == 0
    assert L.fwt_gated_ffn_backward_workspace(4, 8, 0, ctypes.byref(out)) == EINVAL


def test_workspaces_of_shared_contractions(L):
    def size(fn, *a):
        out = ctypes.c_size_t(77)
        return fn(*a, ctypes.byref(out)), out.value
    mm, gf = L.fwt_scaled_matmul_workspace, L.fwt_gated_ffn_workspace
    # few tiles with many steps; not: few rows, few steps, many tiles
    for dtype in (BF16, F16, F32):
        st, n = size(mm, 300, 200, 16000, 0, dtype)
        assert st == OK and 0 < n <= 16 << 20
    assert size(mm, 4, 200, 16000, 0, BF16) == (OK, 0)
    assert size(mm, 300, 200, 256, 1, BF16) == (OK, 0)
    assert size(mm, 4096, 4096, 16384, 1, BF16) == (OK, 0)
    assert size(mm, 0, 200, 16000, 1, BF16) == (OK, 0)
    assert size(mm, 300, 200, 0, 1, BF16)[0] == EINVAL
    assert size(mm, 300, 200, 16000, 3, BF16)[0] == EINVAL
    assert size(mm, 300, 200, 16000, 0, E4M3)[0] == EINVAL
    assert mm(1, 1, 1, 0, BF16, None) == EINVAL
    st, n = size(gf, BF16, 64, 64, 8016, BF16)
    assert st == OK and 0 < n <= 16 << 20
    assert size(gf, E4M3, 300, 128, 16384, F32)[1] > 0
    assert size(gf, BF16, 64, 64, 8016, F16)[0] == EINVAL
    assert gf(BF16, 1, 1, 1, BF16, None) == EINVAL
    # a workspace that is given has to be whole and aligned
    big = dict(m=300, n=200, k=16000, lda=16000, ldb=16000, ldc=200)
    far = {n: (i + 1) << 28 for i, n in enumerate(("a", "sa", "b", "sb", "c", "ws"))}
    assert matmul(L, **big, **dict(far, wsb=16)) == EINVAL
    assert matmul(L, **big, **dict(far, ws=far["ws"] + 4, wsb=1 << 24)) == EALIGN
    assert matmul(L, **big, **dict(far, ws=far["a"], wsb=1 << 24)) == EINVAL
    far = {n: (i + 1) << 28 for i, n in enumerate(("x", "g", "u", "h", "ws"))}
    big = dict(m=64, n=64, k=8016, ldx=8016, ldg=8016, ldu=8016, ldh=64)
    assert gated(L, **big, **dict(far, wsb=16)) == EINVAL
    assert gated(L, **big, **dict(far, ws=far["ws"] + 8, wsb=1 << 24)) == EALIGN


def test_host_tensors_are_refused(L):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qse.rotate_quantize(x, bits=4)
    with pytest.raises(ValueError):
        qse.gated_ffn(x, x, x)
    with pytest.raises(ValueError):
        qse.gated_ffn_backward(x, x, x, x)
    q = x.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        qse.scaled_matmul(q, torch.zeros(1, 4), q, torch.zeros(1, 4))
    with pytest.raises(ValueError):
        qse.rotate_quantize(x, scales="column")
    for bits in (-1, 15, 1 << 32, (1 << 32) + 3):     # (no wrap to a valid number)
        with pytest.raises(qse.FwtError):
            qse.rotate_quantize(x, bits=bits)
    with pytest.raises(TypeError):
        qse.rotate_quantize(x, bits=2.5)
