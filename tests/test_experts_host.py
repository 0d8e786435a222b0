"""Host-side tests of the entry points of include/fwt_experts.h (no GPU):
exported symbols, workspace sizes, and the refusals that come before any HIP
call."""
import ctypes
import os
import re

import pytest

import quantum_state_encoding_amd as qse
from quantum_state_encoding_amd import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EALIGN, EUNSUPPORTED = 0, -1, -2, -3
BF16, F16, F32, E4M3, INT8 = 0, 1, 2, 3, 5
P = 0x10000          # an aligned address that is never read: refusals come first


@pytest.fixture(scope="module")
def L(lib):
    pytest.importorskip("torch")
    return experts._load()


def test_header_declares_the_binding_symbols(lib):
    head = open(os.path.join(ROOT, "include", "fwt_experts.h")).read()
    text = re.sub(r"/\*.*?\*/", "", head, flags=re.S)
    names = sorted(set(re.findall(r"\b(fwt_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(experts.EXPERTS_SYMBOLS)
    for name in names:
        assert hasattr(lib, name)
    assert "FWT_INT8 %d" % experts.INT8 in head
    for name in experts.__all__[:4]:
        assert getattr(qse, name) is getattr(experts, name) and name in qse.__all__


def quantize(L, x=P, dtype=BF16, m=4, k=256, ldx=256, bits=3, q=2 * P, ldq=256, s=3 * P):
    return L.fwt_rotate_quantize_int8(x, dtype, m, k, ldx, bits, q, ldq, s, None)


def test_quantize_refusals(L):
    assert quantize(L, m=0) == OK
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(dtype=E4M3), dict(dtype=INT8),
                dict(dtype=9), dict(m=-1), dict(k=0), dict(k=-8), dict(bits=-1), dict(bits=15),
                dict(k=252), dict(k=300, bits=9), dict(m=1 << 31), dict(ldx=255), dict(ldq=240),
                dict(ldx=-256), dict(q=P), dict(s=P), dict(s=2 * P + 16)):
        assert quantize(L, **bad) == EINVAL, bad
    for bad in (dict(q=2 * P + 8), dict(ldq=264), dict(s=3 * P + 2), dict(x=P + 1)):
        assert quantize(L, **bad) == EALIGN, bad
    far = dict(x=1 << 40, q=1 << 43, s=1 << 45)
    # a workgroup for each long row, for 2^8 / 2^shift short ones
    assert quantize(L, **far, m=1 << 22, k=4096, ldx=4096, ldq=4096) == EUNSUPPORTED
    assert quantize(L, **far, m=1 << 24, k=2048, ldx=2048, ldq=2048) == EUNSUPPORTED
    assert quantize(L, **far, m=1 << 30, k=32, ldx=32, ldq=32) == EUNSUPPORTED
    for ldx in ((1 << 40) + 1, (1 << 63) - 1, -(1 << 63)):
        assert quantize(L, **dict(far, ldx=ldx)) == EINVAL


def matmul(L, a=P, lda=256, sa=2 * P, b=3 * P, ldb=256, sb=4 * P, m=4, n=8, k=256, c=5 * P,
           ctype=BF16, ldc=8, ws=None, wsb=0):
    return L.fwt_int8_matmul(a, lda, sa, b, ldb, sb, m, n, k, c, ctype, ldc, ws, wsb, None)


def test_matmul_refusals(L):
    assert matmul(L, m=0) == OK and matmul(L, n=0) == OK
    for bad in (dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(c=None),
                dict(m=-1), dict(n=-1), dict(k=0), dict(ctype=E4M3), dict(ctype=INT8),
                dict(c=P), dict(c=3 * P + 16), dict(c=4 * P), dict(lda=240), dict(ldb=-256),
                dict(ldc=7)):
        assert matmul(L, **bad) == EINVAL, bad
    for bad in (dict(a=P + 1), dict(b=3 * P + 8), dict(lda=264), dict(ldb=257),
                dict(sa=2 * P + 2), dict(c=5 * P + 1)):
        assert matmul(L, **bad) == EALIGN, bad
    for bad in (dict(lda=1 << 23), dict(ldb=1 << 23), dict(m=1 << 20, n=1 << 15, ldc=1 << 15),
                dict(k=1 << 17, lda=1 << 17, ldb=1 << 17)):
        assert matmul(L, **bad) == EUNSUPPORTED, bad
    # a workspace that is given has to be whole, aligned and apart
    big = dict(m=300, n=200, k=16000, lda=16000, ldb=16000, ldc=200)
    far = {n: (i + 1) << 28 for i, n in enumerate(("a", "sa", "b", "sb", "c", "ws"))}
    assert matmul(L, **big, **dict(far, wsb=16)) == EINVAL
    assert matmul(L, **big, **dict(far, ws=far["ws"] + 4, wsb=1 << 24)) == EALIGN
    assert matmul(L, **big, **dict(far, ws=far["a"], wsb=1 << 24)) == EINVAL


def size(fn, *a):
    out = ctypes.c_size_t(77)
    return fn(*a, ctypes.byref(out)), out.value


def test_workspaces(L):
    mm = L.fwt_int8_matmul_workspace
    for dtype in (BF16, F16, F32):
        st, n = size(mm, 300, 200, 16000, dtype)
        assert st == OK and 0 < n <= 16 << 20
    assert size(mm, 4, 200, 16000, BF16) == (OK, 0)
    assert size(mm, 300, 200, 256, BF16) == (OK, 0)
    assert size(mm, 4096, 4096, 16384, BF16) == (OK, 0)
    assert size(mm, 0, 200, 16000, BF16) == (OK, 0)
    assert size(mm, 300, 200, 0, BF16)[0] == EINVAL
    assert size(mm, 300, 200, 16000, E4M3)[0] == EINVAL
    assert mm(1, 1, 1, BF16, None) == EINVAL
    gm = L.fwt_grouped_matmul_workspace
    for dtype in (BF16, F16, INT8):
        st, n = size(gm, dtype, 2, 100, 100, 16000)
        assert st == OK and 0 < n <= 32 << 20
        assert size(gm, dtype, 8, 4096, 4096, 4096) == (OK, 0)
        assert size(gm, dtype, 8, 0, 4096, 4096) == (OK, 0)
        assert size(gm, dtype, 0, 10, 10, 10)[0] == EINVAL
    assert size(gm, F32, 2, 100, 100, 16000)[0] == EINVAL
    assert gm(BF16, 1, 1, 1, 1, None) == EINVAL
    gb = L.fwt_grouped_matmul_backward_workspace
    st, n = size(gb, 1, 16384, 64, 64)      # few results of many rows
    assert st == OK and 0 < n <= 32 << 20
    assert size(gb, 4, 0, 64, 64) == (OK, 0)
    assert size(gb, 0, 10, 64, 64)[0] == EINVAL
    assert size(gb, 1, 10, 64, 0)[0] == EINVAL
    assert gb(1, 1, 1, 1, None) == EINVAL


def grouped(L, x=P, ldx=64, xs=None, w=2 * P, ldw=64, sw=512, wsc=None, ends=3 * P, e=3,
            dtype=BF16, m=4, n=8, k=64, y=4 * P, ytype=BF16, ldy=8, zero=1, ws=None, wsb=0):
    return L.fwt_grouped_matmul(x, ldx, xs, w, ldw, sw, wsc, ends, e, dtype, m, n, k, y, ytype,
                                ldy, zero, ws, wsb, None)


def test_grouped_refusals(L):
    assert grouped(L, m=0) == OK and grouped(L, n=0) == OK
    i8 = dict(dtype=INT8, xs=5 * P, wsc=6 * P)
    for bad in (dict(x=None), dict(w=None), dict(ends=None), dict(y=None), dict(dtype=F32),
                dict(dtype=E4M3), dict(ytype=F16), dict(ytype=F32), dict(k=0), dict(m=-1),
                dict(e=0), dict(e=-1), dict(xs=5 * P), dict(wsc=5 * P), dict(dtype=INT8),
                dict(i8, xs=None), dict(i8, wsc=None), dict(i8, ytype=E4M3), dict(y=P),
                dict(y=2 * P), dict(y=3 * P), dict(i8, y=6 * P), dict(sw=511), dict(sw=-512),
                dict(ldw=63), dict(ldw=-64), dict(ldx=63), dict(ldy=7),
                dict(sw=(1 << 40) + 1), dict(ldw=1 << 41), dict(sw=(1 << 63) - 1)):
        assert grouped(L, **bad) in (EINVAL, EUNSUPPORTED), bad
        if not set(bad) & {"ldw", "ldx"}:
            assert grouped(L, **bad) == EINVAL, bad
    for bad in (dict(i8, x=P + 4), dict(i8, ldw=72), dict(i8, sw=520), dict(ends=3 * P + 2),
                dict(x=P + 1), dict(y=4 * P + 1)):
        assert grouped(L, **bad) == EALIGN, bad
    for bad in (dict(ldx=1 << 22), dict(ldw=1 << 22, sw=1 << 27), dict(i8, ldx=1 << 23),
                dict(m=1 << 20, n=1 << 15, ldy=1 << 15, sw=1 << 21), dict(e=(1 << 16) + 1),
                dict(m=1 << 16, e=1 << 16, n=1 << 13, ldy=1 << 13, sw=1 << 19),
                dict(i8, k=1 << 17, ldx=1 << 17, ldw=1 << 17, sw=1 << 20)):
        assert grouped(L, **bad) == EUNSUPPORTED, bad
    big = dict(e=2, m=100, n=100, k=16000, ldx=16000, ldw=16000, sw=1600000, ldy=100)
    far = {n: (i + 1) << 28 for i, n in enumerate(("x", "w", "ends", "y", "ws"))}
    assert grouped(L, **big, **dict(far, wsb=16)) == EINVAL
    assert grouped(L, **big, **dict(far, ws=far["ws"] + 8, wsb=1 << 26)) == EALIGN
    assert grouped(L, **big, **dict(far, ws=far["x"], wsb=1 << 26)) == EINVAL


def backward(L, x=P, ldx=64, w=2 * P, ldw=64, sw=512, ends=3 * P, e=3, dy=4 * P, lddy=8,
             dtype=BF16, m=4, n=8, k=64, dx=5 * P, lddx=64, dw=6 * P, lddw=64, sdw=512, ws=None,
             wsb=0):
    return L.fwt_grouped_matmul_backward(x, ldx, w, ldw, sw, ends, e, dy, lddy, dtype, m, n, k,
                                         dx, lddx, dw, lddw, sdw, ws, wsb, None)


def test_backward_refusals(L):
    assert backward(L, m=0, n=0) == OK
    assert backward(L, dx=None, dw=None) == OK
    for bad in (dict(x=None), dict(w=None), dict(dy=None), dict(ends=None), dict(dtype=INT8),
                dict(dtype=F32), dict(k=0), dict(n=-1), dict(e=0), dict(dx=P), dict(dw=5 * P),
                dict(dx=4 * P), dict(dw=3 * P), dict(sdw=511), dict(lddw=63), dict(lddx=63),
                dict(sw=500), dict(m=0, ends=None)):
        assert backward(L, **bad) == EINVAL, bad
    for bad in (dict(x=P + 1), dict(dw=6 * P + 1), dict(ends=3 * P + 1)):
        assert backward(L, **bad) == EALIGN, bad
    for bad in (dict(ldx=1 << 22), dict(ldw=1 << 22, sw=1 << 27), dict(lddy=1 << 22),
                dict(e=(1 << 16) + 1), dict(m=1 << 20, k=1 << 15, ldx=1 << 15, ldw=1 << 15),
                dict(e=1 << 14, n=1 << 12, k=1 << 12, ldx=1 << 12, ldw=1 << 12, lddy=1 << 12)):
        assert backward(L, **bad) == EUNSUPPORTED, bad


def test_scratch_for_copies_is_that_of_misaligned_operands(L):
    gm, gf = L.fwt_grouped_matmul_workspace, L.fwt_grouped_matmul_workspace_for
    bm, bf = L.fwt_grouped_matmul_backward_workspace, L.fwt_grouped_matmul_backward_workspace_for
    e, m, n, k = 8, 16000, 4001, 4095
    row = lambda cols: 2 * (-(-cols // 8) * 8)                                    # noqa: E731
    pad, odd, A, O = 4096, 4095, 1 << 32, (1 << 32) + 2
    all_x, all_w, all_dy = m * row(k), e * n * row(k), m * row(n)

    def fwd(x=A, ldx=pad, w=A, ldw=pad, sw=n * pad, dtype=BF16):
        st, b = size(gf, x, ldx, w, ldw, sw, e, dtype, m, n, k)
        assert st == OK
        return b

    assert size(gm, BF16, e, m, n, k) == (OK, all_x + all_w)
    assert fwd() == 0 and fwd(x=None, w=None) == 0
    assert fwd(dtype=INT8) == 0
    assert fwd(ldx=odd) == all_x and fwd(x=O) == all_x
    assert fwd(ldw=odd, sw=n * odd) == all_w and fwd(w=O) == all_w and fwd(sw=n * pad + 1) == all_w
    assert fwd(ldx=odd, w=O) == all_x + all_w

    def bwd(x=A, ldx=pad, w=A, ldw=pad, sw=n * pad, dy=A, lddy=4008, dx=1, dw=1):
        st, b = size(bf, x, ldx, w, ldw, sw, e, dy, lddy, m, n, k, dx, dw)
        assert st == OK
        return b

    up = lambda b: -(-b // 256) * 256                                               # noqa: E731
    assert size(bm, e, m, n, k) == (OK, all_x + all_w + all_dy)
    assert bwd() == 0 and bwd(dx=0, dw=0, dy=O) == 0
    assert bwd(x=O, w=O, dy=O) == all_x + all_w + all_dy
    assert bwd(x=O) == all_x and bwd(x=O, dw=0) == 0 and bwd(w=O, dx=0) == 0
    assert bwd(dy=O) == all_dy and bwd(dy=O, x=O, dx=0) == all_dy + all_x
    # with one expert the stride between experts does not count
    assert size(gf, A, pad, A, pad, 7, 1, BF16, m, n, k) == (OK, 0)
    # never more than for any operands; sums are shared whatever lies where
    for e, m, n, k in ((2, 100, 100, 16000), (3, 3604, 1019, 3373), (1, 300, 200, 9001),
                       (4, 8000, 2001, 2001), (1, 16384, 64, 64), (32, 4000, 2001, 1501)):
        most, most_b = size(gm, BF16, e, m, n, k)[1], size(bm, e, m, n, k)[1]
        for x in (A, A + 4, O):
            for w in (A, A + 4, O):
                b = size(gf, x, k, w, k, n * k, e, BF16, m, n, k)
                assert b[0] == OK and b[1] <= most
                for dy in (A, O):
                    for want in (1, 2, 3):
                        b = size(bf, x, k, w, k, n * k, e, dy, n, m, n, k, want & 1, want & 2)
                        assert b[0] == OK and b[1] <= most_b
    # sizes past what there is
    assert size(gm, BF16, 1 << 16, 1 << 6, 1 << 20, (1 << 20) - 1)[0] == OK
    for bad in (dict(e=0), dict(m=-1), dict(k=0), dict(dtype=F32)):
        a = dict(dict(e=2, m=4, n=8, k=64, dtype=BF16), **bad)
        assert size(gf, A, 64, A, 64, 512, a["e"], a["dtype"], a["m"], a["n"], a["k"])[0] == EINVAL
        if "dtype" not in bad:
            assert size(bf, A, 64, A, 64, 512, a["e"], A, 8, a["m"], a["n"], a["k"], 1, 1)[0] == EINVAL
    assert gf(A, 64, A, 64, 512, 2, BF16, 4, 8, 64, None) == EINVAL
    assert bf(A, 64, A, 64, 512, 2, A, 8, 4, 8, 64, 1, 1, None) == EINVAL


def test_kernels_are_those_that_calls_reach(lib):
    # rows of up to 2048 elements take rotations of up to 2^11, which 32 neighbours of a
    # lane hold from the start; the layout for shorter rotations is one of long rows
    built = open(qse.library_path(), "rb").read()
    names = set(re.findall(rb"quantize8_kernelILi(\d)ELi(\d+)ELb([01])ELb([01])E", built))
    short = {int(bits) for _, bits, one, _ in names if one == b"0"}
    assert short == set(range(5, 12))
    for twice in (b"0", b"1"):
        assert {int(bits) for _, bits, one, two in names
                if one == b"1" and two == twice} == set(range(4, 15))
    assert len(names) == 3 * (7 + 11 + 11)
    # of 8-bit integers, shares of the smallest tiles alone are joined
    for kernel in (rb"\d\djoin_kernel", rb"grouped_join_kernel"):
        assert set(re.findall(kernel + rb"ILi5ELi(\d+)ELi(\d+)E", built)) == {(b"64", b"64")}


def test_host_tensors_are_refused(L):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    ends = torch.tensor([2, 4], dtype=torch.int32)
    q, s = x.to(torch.int8), torch.ones(4)
    for call in (lambda: qse.rotate_quantize_int8(x, bits=4),
                 lambda: qse.int8_matmul(q, s, q, s),
                 lambda: qse.grouped_matmul(x, w, ends),
                 lambda: qse.grouped_matmul_backward(x, w, ends, torch.zeros(4, 8))):
        with pytest.raises(ValueError):
            call()
    for bits in (-1, 15, 1 << 32, (1 << 32) + 3):     # (no wrap to a valid number)
        with pytest.raises(qse.FwtError):
            qse.rotate_quantize_int8(x, bits=bits)
    with pytest.raises(TypeError):
        qse.rotate_quantize_int8(x, bits=2.5)


def test_tangents_are_not_dropped(L):
    import torch
    from torch.autograd import forward_ad
    from quantum_state_encoding_amd import ffn
    x = torch.zeros(4, 8)
    for check in (ffn._no_graph, experts._no_graph):
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(x, torch.ones(4, 8))
            for mode in (torch.enable_grad(), torch.no_grad()):     # (both keep tangents)
                with mode, pytest.raises(ValueError, match="tangent"):
                    check("call", x, None, dual)
            check("call", x, None, dual.detach())
        check("call", x, None)
