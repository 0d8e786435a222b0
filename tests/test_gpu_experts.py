"""8-bit integer products and products grouped by expert on the GPU, against
their definitions in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32 relative to a value; half(t) of
a result type is finfo(t).eps / 2.  A sum of n terms in fp32, in any order and
with any rounding direction, is within n 2u sum |terms| of the exact one.
Integer products are compared for equality: the sum of 8-bit products is exact
in int32, and what follows are three roundings that torch makes alike.
"""
import ctypes

import pytest

import quantum_state_encoding_amd as qse
from quantum_state_encoding_amd import experts

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def say(*a):
    print("[case]", *a, flush=True)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cdiv(a, b):
    return -(-a // b)


def half(dtype):
    return torch.finfo(dtype).eps / 2


# ---- rotate_quantize_int8 ----------------------------------------------------

def hadamard_rows(x, bits):
    """x (I (x) H_bits) in the dtype of x, unnormalised."""
    m, k = x.shape
    for b in range(bits):
        x = x.reshape(-1, 2, 1 << b)
        x = torch.stack([x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]], 1)
    return x.reshape(m, k)


QUANTIZE = [  # m, k, bits
    (1, 1, 0), (3, 2, 1), (5, 31, 0), (300, 33, 0), (7, 64, 6), (1, 4096, 12), (9, 100, 2),
    (1000, 64, 5), (67, 128, 7), (130, 24, 3), (33, 1000, 3), (257, 512, 9), (5, 1024, 10),
    (6, 1280, 8), (13, 2048, 11), (4, 2048, 10), (3, 2049, 0), (17, 2112, 6), (5, 5000, 3),
    (3, 6144, 11), (2, 8192, 13), (3, 16384, 14), (2, 20480, 12), (7, 4352, 8), (9, 6656, 9),
    (2, 32768, 14), (3, 32768, 5), (2, 28672, 7),
    # rows of more than 32768 elements, with whole and partial last parts
    (2, 32769, 0), (3, 33024, 8), (2, 65536, 14), (3, 34816, 11), (2, 49152, 14), (2, 70000, 4),
    (2, 98368, 6), (1, 131071, 0),
]


@pytest.mark.parametrize("m,k,bits", QUANTIZE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_of_integers_is_the_division_rounded(m, k, bits, dtype):
    # Sums of integers up to 8 in magnitude are exact, 2^-(bits/2) is exact
    # for even bits, so y is known exactly, s is one fp32 division and a code
    # is y / s rounded to fp32 and then to an integer.
    say("quantize int", m, k, bits, dtype)
    x = torch.randint(-8, 9, (m, k), generator=gen(m + k), device="cuda").float()
    q, s = qse.rotate_quantize_int8(x.to(DT[dtype]), bits=bits)
    assert q.dtype == torch.int8 and tuple(q.shape) == (m, k) and tuple(s.shape) == (m,)
    y = hadamard_rows(x, bits)
    # (odd bits: the factor rounds, once in the library, once here)
    y = y * (2.0 ** -0.5 * 2.0 ** -(bits // 2)) if bits % 2 else y * 2.0 ** -(bits // 2)
    # (a division by a tensor: torch multiplies by a Python number's reciprocal)
    top = torch.full((), 127.0, device="cuda")
    want_s = (y.abs().amax(1) / top).clamp_min(2.0 ** -126)
    assert torch.equal(s, want_s)
    want = torch.round(y / want_s[:, None])
    assert torch.equal(q.float(), want)
    if m > 1 and q.stride(0) != k:      # the padding of a row is zeros
        ld = q.stride(0)
        assert bool((torch.as_strided(q, (m, ld), (ld, 1))[:, k:] == 0).all())


@pytest.mark.parametrize("m,k,bits", QUANTIZE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_of_activations(m, k, bits, dtype):
    say("quantize gauss", m, k, bits, dtype)
    g = gen(7 * m + k)
    x = torch.randn(m, k, generator=g, device="cuda")
    x = torch.where(torch.rand(1, k, generator=g, device="cuda") < 0.02, x * 50, x).to(DT[dtype])
    q, s = qse.rotate_quantize_int8(x, bits=bits)
    c = 2.0 ** (-bits / 2)
    y = hadamard_rows(x.double(), bits) * c
    # bits additions and the factor's rounding and product, each within u of
    # partial sums that are at most the sum of magnitudes
    mag = x.double().abs().reshape(m, k >> bits, 1 << bits).sum(2) * c
    err = ((bits + 3) * U * mag).repeat_interleave(1 << bits, 1)
    want_s = (y.abs().amax(1) / 127).clamp_min(2.0 ** -126)
    assert bool(((s.double() - want_s).abs() <= err.amax(1) / 127 + 2 * U * want_s).all())
    r = y / s.double()[:, None]
    # half a step, the division's rounding, and y's error
    tol = 0.5 + 2 * U * r.abs() + err / s.double()[:, None]
    assert bool(((q.double() - r).abs() <= tol).all())
    assert int(q.abs().amax()) <= 127


@pytest.mark.parametrize("bits", [0, 4, 6, 9, 10, 11, 13])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_of_views(bits, dtype):
    # rows that begin at any element, and a value that is not finite: its row
    # gets a NaN scale and zero codes, no other does
    say("quantize views", bits, dtype)
    for k in (1 << bits, 3 << bits, 5 << bits):
        big = torch.randn(9, k + 11, generator=gen(k), device="cuda").to(DT[dtype])
        for lo in (0, 1, 3, 8):
            view = big[:, lo:lo + k]
            q, s = qse.rotate_quantize_int8(view, bits=bits)
            q2, s2 = qse.rotate_quantize_int8(view.contiguous(), bits=bits)
            assert torch.equal(q, q2) and torch.equal(s, s2)
        for bad in (float("inf"), float("-inf"), float("nan")):
            view = big[:, 2:2 + k].clone()
            view[4, k // 2] = bad
            q2, s2 = qse.rotate_quantize_int8(view, bits=bits)
            q, s = qse.rotate_quantize_int8(big[:, 2:2 + k], bits=bits)
            other = torch.arange(9, device="cuda") != 4
            assert torch.equal(q[other], q2[other]) and torch.equal(s[other], s2[other])
            assert bool(torch.isnan(s2[4])) and bool((q2[4] == 0).all())


def test_quantize_extremes():
    say("quantize extremes")
    for k in (512, 4096, 40960):
        x = torch.zeros(5, k, device="cuda")
        x[1] = 3.0e38                   # the largest magnitudes
        x[2, :128] = 1e-42              # subnormal: the scale stays normal
        x[3, 3] = -1.0
        x[4, k - 1] = float("nan")
        q, s = qse.rotate_quantize_int8(x)
        assert bool((q[0] == 0).all()) and float(s[0]) == 2.0 ** -126
        assert bool((q[1] == 127).all()) and abs(float(s[1]) - 3.0e38 / 127) < 1e30
        assert bool((q[2] == 0).all()) and float(s[2]) == 2.0 ** -126
        assert int(q[3, 3]) == -127 and int(q[3].abs().sum()) == 127
        assert bool(torch.isnan(s[4])) and bool((q[4] == 0).all())
        # 512 times 3e38 passes the fp32 range, in its row alone
        q, s = qse.rotate_quantize_int8(x, bits=9)
        assert torch.isnan(s).tolist() == [False, True, False, False, True]
        assert bool((q[1] == 0).all()) and bool((q[3, :512].abs() == 127).all())
        assert bool((q[3, 512:] == 0).all())


# ---- int8_matmul -------------------------------------------------------------

def padded(q):
    """Codes in rows padded to 16 bytes, the padding -128: it is not read."""
    k = q.shape[-1]
    full = torch.full(q.shape[:-1] + (cdiv(k, 16) * 16,), -128, dtype=torch.int8, device="cuda")
    full[..., :k] = q
    return full[..., :k]


def codes(g, *shape):
    return padded(torch.randint(-128, 128, shape, generator=g, device="cuda").to(torch.int8))


def some_scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 1e-2 + 1e-4


def int8_result(a, sa, b, sb, dtype):
    """(exact sum rounded to fp32) sa sb, rounded after each product, then to dtype."""
    return (exact_product(a, b).float() * sa[:, None] * sb).to(dtype)


def exact_product(a, b):
    """Sums below 2^53: exact in 64-bit floats."""
    return a.double() @ b.double().t()


MATMUL = [  # m, n, k
    (1, 1, 1), (1, 16, 128), (1, 300, 4096), (2, 17, 129), (16, 256, 384), (17, 129, 255),
    (33, 64, 100), (64, 500, 1000), (65, 128, 128), (128, 130, 2000), (130, 1, 16),
    (257, 255, 640), (300, 1025, 144), (1000, 700, 15), (100, 2100, 513),
    (3600, 3400, 272), (3601, 3399, 1007),
    # ragged edges in every tile
    (700, 4001, 400), (1900, 4000, 260), (500, 3970, 130), (200, 1030, 2100), (20, 16400, 300),
    (9, 16390, 1111), (31, 777, 8193), (2, 100, 9000), (1, 16385, 500),
    # few results of a long contraction, which several workgroups share
    (300, 200, 16001), (65, 70, 9100), (33, 129, 30000),
    # the longest contraction
    (40, 30, 131071), (3, 20, 131071),
]


@pytest.mark.parametrize("m,n,k", MATMUL)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_int8_matmul_is_exact(m, n, k, out):
    say("int8", m, n, k, out)
    g = gen(m + 3 * n + k)
    a, b = codes(g, m, k), codes(g, n, k)
    sa, sb = some_scales(g, m), some_scales(g, n)
    c = qse.int8_matmul(a, sa, b, sb, out_dtype=DT[out])
    assert c.dtype == DT[out] and tuple(c.shape) == (m, n)
    assert torch.equal(c, int8_result(a, sa, b, sb, DT[out]))


@pytest.mark.parametrize("k", [131071, 130000])
def test_int8_sums_reach_the_ends_of_32_bits(k):
    # all products 128^2, or -128 * 127: sums next to 2^31
    say("int8 ends", k)
    a = padded(torch.full((40, k), -128, dtype=torch.int8, device="cuda"))
    b = padded(torch.full((70, k), -128, dtype=torch.int8, device="cuda"))
    b[1::2] = 127
    one = torch.ones(70, device="cuda")
    c = qse.int8_matmul(a, one[:40], b, one, out_dtype=torch.float32)
    assert torch.equal(c, exact_product(a, b).float())
    assert float(c.max()) == float(torch.tensor(128.0 * 128 * k, dtype=torch.float32))


def test_int8_scales_one_after_the_other():
    # products of scales that leave fp32's range where the results do not
    say("int8 scales")
    g = gen(8)
    for m in (3, 100):
        a, b = codes(g, m, 64), codes(g, 50, 64)
        sa = torch.full((m,), 2.0 ** -120, device="cuda")
        sb = torch.full((50,), 2.0 ** -20, device="cuda")
        c = qse.int8_matmul(a, sa, b, sb, out_dtype=torch.float32)
        want = (exact_product(a, b) * 2.0 ** -140).float()       # subnormal, exact sums
        assert torch.equal(c, want) and bool((c != 0).any())


def test_int8_into_a_view_leaves_the_rest():
    say("int8 out view")
    g = gen(3)
    for m, n, k in ((5, 33, 200), (150, 131, 300)):
        a, b = codes(g, m, k), codes(g, n, k)
        sa, sb = some_scales(g, m), some_scales(g, n)
        for dt in DT.values():
            big = torch.full((m + 2, n + 9), 7.0, dtype=dt, device="cuda")
            view = big[1:m + 1, 4:n + 4]
            assert qse.int8_matmul(a, sa, b, sb, out=view) is view
            assert torch.equal(view, qse.int8_matmul(a, sa, b, sb, out_dtype=dt))
            big[1:m + 1, 4:n + 4] = 7.0
            assert bool((big == 7.0).all())


def test_int8_nan_scales_reach_their_rows_and_columns():
    say("int8 nan")
    g = gen(4)
    for m in (3, 20, 200):
        a, b = codes(g, m, 256), codes(g, 40, 256)
        sa, sb = some_scales(g, m), some_scales(g, 40)
        clean = qse.int8_matmul(a, sa, b, sb)
        sa[1] = float("nan")
        sb[7] = float("inf")
        c = qse.int8_matmul(a, sa, b, sb)
        assert bool(torch.isnan(c[1]).all())
        assert not bool(torch.isfinite(c[:, 7]).any())
        keep = torch.ones_like(c, dtype=torch.bool)
        keep[1], keep[:, 7] = False, False
        assert torch.equal(c[keep], clean[keep])


def test_int8_without_scratch_is_the_same():
    say("int8 no scratch")
    L = experts._load()
    g = gen(6)
    for m, n, k in ((300, 200, 16000), (64, 64, 9104)):
        a, b = codes(g, m, k), codes(g, n, k)
        sa, sb = some_scales(g, m), some_scales(g, n)
        c = torch.empty(m, n, device="cuda")
        st = L.fwt_int8_matmul(a.data_ptr(), a.stride(0), sa.data_ptr(), b.data_ptr(),
                               b.stride(0), sb.data_ptr(), m, n, k, c.data_ptr(), 2, n, None, 0,
                               torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(c, qse.int8_matmul(a, sa, b, sb, out_dtype=torch.float32))


# ---- grouped_matmul ----------------------------------------------------------

def ends_of(counts):
    t = torch.tensor(counts, dtype=torch.int64).cumsum(0)
    return t.to(torch.int32).cuda()


def spread_counts(m, e, seed):
    """m rows over e experts, unevenly; some get none."""
    g = torch.Generator()
    g.manual_seed(seed)
    p = torch.rand(e, generator=g) ** 3 + 1e-6
    pick = torch.multinomial(p, max(m, 1), replacement=True, generator=g)[:m]
    return torch.bincount(pick, minlength=e).tolist()


GROUPED = [  # counts, rest, n, k
    ([1], 0, 1, 1), ([1], 0, 16, 64), ([0, 1, 0], 0, 33, 100), ([0], 3, 20, 40),
    ([0, 0, 0], 70, 300, 130), ([3, 0, 5, 1], 2, 70, 257), ([16, 17, 15, 1], 0, 130, 512),
    ([40, 1, 0, 33], 9, 129, 1000), ([200, 0, 56], 0, 256, 64), ([1, 255, 257], 1, 255, 330),
    ([130, 129, 0, 1, 300], 77, 500, 72), ([700], 0, 1000, 200), ([600, 500], 0, 2050, 136),
    ([64] * 8, 0, 192, 320), ([2] * 70, 1, 48, 96), ([0] * 64 + [5] + [0] * 64 + [7], 0, 40, 128),
    ([1] * 130, 0, 65, 60), ([3000, 10, 1500, 0, 2000], 100, 3000, 264),
    ([900, 1100, 0, 2000], 0, 4100, 520), ([257] * 9, 30, 4000, 130), ([5, 7], 0, 100, 16001),
    ([300], 0, 200, 16008), ([33, 60], 7, 130, 9104), ([128] * 32, 0, 512, 640),
    ([4, 0, 1], 0, 7, 3), ([50, 100], 0, 5, 2000), ([50, 100], 0, 2000, 5), ([9, 8], 1, 15, 7),
]


def group_bounds(counts):
    lo = 0
    for e, c in enumerate(counts):
        yield e, lo, lo + c
        lo += c


def grouped_reference(x, w, counts, total, scale=None):
    """y and the sums of magnitudes in 64 bits; zeros behind the last group."""
    y = torch.zeros(total, w.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for e, lo, hi in group_bounds(counts):
        if hi > lo:
            a, b = x[lo:hi].double(), w[e].double()
            y[lo:hi] = a @ b.t()
            mag[lo:hi] = a.abs() @ b.abs().t()
    return y, mag


def check_sums(got, want, mag, terms, dtype):
    e = (terms + 2) * 2 * U * mag
    tol = e + half(dtype) * (want.abs() + e)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25          # half a step of its subnormals
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("odd", [0, 1])
def test_grouped(case, dtype, odd):
    # odd: rows and experts that begin at any element, inside NaN
    counts, rest, n, k = GROUPED[case]
    say("grouped", case, counts[:8], rest, n, k, dtype, odd)
    g, dt = gen(case), DT[dtype]
    m, e = sum(counts) + rest, len(counts)
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(e, n, k, generator=g, device="cuda") * k ** -0.5).to(dt)
    if odd:
        bx = torch.full((m, k + 5), float("nan"), dtype=dt, device="cuda")
        bx[:, 3:3 + k] = x
        bw = torch.full((e, n + 1, k + 3), float("nan"), dtype=dt, device="cuda")
        bw[:, :n, 1:1 + k] = w
        xs, ws = bx[:, 3:3 + k], bw[:, :n, 1:1 + k]
    else:
        xs, ws = x, w
    if rest:
        xs[m - rest:] = float("nan")    # not read
    for i, c in enumerate(counts):
        if c == 0:
            ws[i] = float("nan")        # nor these
    y = qse.grouped_matmul(xs, ws, ends_of(counts))
    assert y.dtype == dt and tuple(y.shape) == (m, n)
    want, mag = grouped_reference(x, w, counts, m)
    check_sums(y, want, mag, k, dt)


@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_grouped_int8_is_exact(case, out):
    counts, rest, n, k = GROUPED[case]
    say("grouped int8", case, counts[:8], rest, n, k, out)
    g = gen(case)
    m, e = sum(counts) + rest, len(counts)
    x, w = codes(g, m, k), codes(g, e, n, k)
    sx, sw = some_scales(g, m), some_scales(g, e, n)
    for i, c in enumerate(counts):
        if c == 0:
            sw[i] = float("nan")
    sx[m - rest:] = float("nan") if rest else 1.0
    y = qse.grouped_matmul(x, w, ends_of(counts), x_scales=sx, w_scales=sw, out_dtype=DT[out])
    assert y.dtype == DT[out] and tuple(y.shape) == (m, n)
    want = torch.zeros(m, n, dtype=DT[out], device="cuda")
    for i, lo, hi in group_bounds(counts):
        want[lo:hi] = int8_result(x[lo:hi], sx[lo:hi], w[i], sw[i], DT[out])
    assert torch.equal(y, want)


@pytest.mark.parametrize("m,e,n,k", [(5, 64, 256, 512), (300, 40, 200, 264), (2000, 6, 1100, 72),
                                     (9000, 12, 600, 128), (1000, 200, 32, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_grouped_of_uneven_groups_into_a_view(m, e, n, k, dtype):
    # rows of no expert, and what surrounds the view, are left as they were
    say("grouped view", m, e, n, k, dtype)
    g = gen(m)
    counts = spread_counts(m, e, m)
    rest = 37
    big = torch.full((m + rest + 2, n + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    view = big[1:-1, 4:n + 4]
    if dtype == "int8":
        x, w = codes(g, m + rest, k), codes(g, e, n, k)
        kw = dict(x_scales=some_scales(g, m + rest), w_scales=some_scales(g, e, n))
    else:
        x = torch.randn(m + rest, k, generator=g, device="cuda").bfloat16()
        w = torch.randn(e, n, k, generator=g, device="cuda").bfloat16()
        kw = {}
    ends = ends_of(counts)
    fresh = qse.grouped_matmul(x, w, ends, **kw)
    assert bool((fresh[m:] == 0).all())
    assert qse.grouped_matmul(x, w, ends, out=view, **kw) is view
    assert torch.equal(view[:m], fresh[:m]) and bool((view[m:] == 7.0).all())
    big[1:m + 1, 4:n + 4] = 7.0
    assert bool((big == 7.0).all())
    if dtype == "bf16":
        want, mag = grouped_reference(x, w, counts, m + rest)
        check_sums(fresh, want, mag, k, torch.bfloat16)
    else:
        for i, lo, hi in group_bounds(counts):
            assert torch.equal(fresh[lo:hi], int8_result(x[lo:hi], kw["x_scales"][lo:hi], w[i],
                                                         kw["w_scales"][i], torch.bfloat16))


def test_grouped_ends_outside_the_rows_are_cut():
    # nothing outside the arrays is read or written; groups that do not
    # contradict each other are computed
    say("grouped ends")
    g = gen(2)
    m, n, k = 100, 70, 64
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(4, n, k, generator=g, device="cuda").bfloat16()
    for ends, counts in (([-5, 20, 2 ** 31 - 1, 2 ** 31 - 1], [0, 20, 80, 0]),
                         ([30, 30, 200, 300], [30, 0, 70, 0]),
                         ([-2 ** 31, -1, 0, 60], [0, 0, 0, 60])):
        big = torch.full((m + 40, n), 7.0, dtype=torch.bfloat16, device="cuda")
        view = big[20:20 + m]
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        qse.grouped_matmul(x, w, e, out=view)
        want, mag = grouped_reference(x, w, counts, m)
        done = sum(counts)
        check_sums(view[:done], want[:done], mag[:done], k, torch.bfloat16)
        view[:done] = 7.0
        assert bool((big == 7.0).all())
    # falling ends: unspecified rows, but nothing around them
    for ends in ([60, 10, 90, 20], [100, 0, 100, 0], [90, 80, 70, 60]):
        big = torch.full((m + 40, n), 7.0, dtype=torch.bfloat16, device="cuda")
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        qse.grouped_matmul(x, w, e, out=big[20:20 + m])
        big[20:20 + m] = 7.0
        assert bool((big == 7.0).all())
        dx, dw = qse.grouped_matmul_backward(x, w, e, big[:m])
        assert bool(torch.isfinite(dw.float()).all())


# ---- grouped_matmul_backward -------------------------------------------------

@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("odd", [0, 1])
def test_grouped_backward(case, dtype, odd):
    counts, rest, n, k = GROUPED[case]
    say("grouped backward", case, counts[:8], rest, n, k, dtype, odd)
    g, dt = gen(100 + case), DT[dtype]
    m, e = sum(counts) + rest, len(counts)
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(e, n, k, generator=g, device="cuda") * n ** -0.5).to(dt)
    dy = (torch.randn(m, n, generator=g, device="cuda") * 0.1).to(dt)
    if odd:
        bx = torch.full((m, k + 5), float("nan"), dtype=dt, device="cuda")
        bx[:, 3:3 + k] = x
        bw = torch.full((e, n + 1, k + 3), float("nan"), dtype=dt, device="cuda")
        bw[:, :n, 1:1 + k] = w
        bd = torch.full((m, n + 7), float("nan"), dtype=dt, device="cuda")
        bd[:, 5:5 + n] = dy
        xs, ws, ds = bx[:, 3:3 + k], bw[:, :n, 1:1 + k], bd[:, 5:5 + n]
    else:
        xs, ws, ds = x, w, dy
    if rest:
        xs[m - rest:] = float("nan")
        ds[m - rest:] = float("nan")
    for i, c in enumerate(counts):
        if c == 0:
            ws[i] = float("nan")
    dx, dw = qse.grouped_matmul_backward(xs, ws, ends_of(counts), ds)
    assert dx.dtype == dt and tuple(dx.shape) == (m, k)
    assert dw.dtype == dt and tuple(dw.shape) == (e, n, k)
    used = sum(counts)
    assert bool((dx[used:] == 0).all())
    for i, lo, hi in group_bounds(counts):
        if hi == lo:
            assert bool((dw[i] == 0).all())
            continue
        gr, a, b = dy[lo:hi].double(), x[lo:hi].double(), w[i].double()
        check_sums(dx[lo:hi], gr @ b, gr.abs() @ b.abs(), n, dt)
        check_sums(dw[i], gr.t() @ a, gr.abs().t() @ a.abs(), hi - lo, dt)


@pytest.mark.parametrize("counts,n,k", [([2500], 64, 64), ([9000, 0, 4000], 130, 70),
                                        ([16384], 256, 200), ([4000] * 4, 100, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_backward_of_few_results_of_many_rows(counts, n, k, dtype):
    # contractions that several workgroups share, with and without scratch
    say("grouped backward shares", counts, n, k, dtype)
    L = experts._load()
    g, dt = gen(5), DT[dtype]
    m, e = sum(counts), len(counts)
    k8 = cdiv(k, 8) * 8
    for kk in (k8, k):
        x = torch.randn(m, kk, generator=g, device="cuda").to(dt)
        w = torch.randn(e, n, kk, generator=g, device="cuda").to(dt)
        dy = (torch.randn(m, n, generator=g, device="cuda") * 0.1).to(dt)
        ends = ends_of(counts)
        dx, dw = qse.grouped_matmul_backward(x, w, ends, dy)
        dw2 = torch.empty_like(dw)
        st = L.fwt_grouped_matmul_backward(
            x.data_ptr(), kk, w.data_ptr(), kk, n * kk, ends.data_ptr(), e, dy.data_ptr(), n,
            0 if dtype == "bf16" else 1, m, n, kk, None, 0, dw2.data_ptr(), kk, n * kk, None, 0,
            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for i, lo, hi in group_bounds(counts):
            gr, a = dy[lo:hi].double(), x[lo:hi].double()
            for d in (dw, dw2):
                check_sums(d[i], gr.t() @ a, gr.abs().t() @ a.abs(), hi - lo, dt)
            check_sums(dx[lo:hi], gr @ w[i].double(), gr.abs() @ w[i].double().abs(), n, dt)


def test_gradients_are_the_differences():
    # small integers: the product and both gradients are exact in fp32, so
    # the change of sum(dy * y) by a step in one operand is its gradient times it
    say("grouped differences")
    g = gen(11)
    counts, n, k = [5, 0, 20, 40], 24, 40
    m = sum(counts) + 3
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, dy, ends = ints(m, k), ints(4, n, k), ints(m, n), ends_of(counts)
    dx, dw = qse.grouped_matmul_backward(x, w, ends, dy)

    def loss(x, w):
        # (in fp32, from the library's products of operands of one column's step)
        y = qse.grouped_matmul(x, w, ends).double()
        return float((dy.double()[:sum(counts)] * y[:sum(counts)]).sum())

    base_y = qse.grouped_matmul(x, w, ends).float()
    assert float(base_y.abs().max()) <= 256          # integers that bf16 holds
    base = loss(x, w)
    r = torch.Generator()
    r.manual_seed(1)
    for _ in range(12):
        i, c = int(torch.randint(m, (1,), generator=r)), int(torch.randint(k, (1,), generator=r))
        x2 = x.clone()
        x2[i, c] += 1
        assert float(qse.grouped_matmul(x2, w, ends).float().abs().max()) <= 256
        assert loss(x2, w) - base == float(dx[i, c])
        e, j = int(torch.randint(4, (1,), generator=r)), int(torch.randint(n, (1,), generator=r))
        w2 = w.clone()
        w2[e, j, c] += 1
        assert float(qse.grouped_matmul(x, w2, ends).float().abs().max()) <= 256
        want = loss(x, w2) - base
        # (dw is rounded to bf16: an integer below 2^12, within half a step)
        assert abs(want - float(dw[e, j, c])) <= half(torch.bfloat16) * abs(want)


# ---- as they are used ----------------------------------------------------------

def test_together_in_an_expert_block():
    # 8-bit experts after a rotation give what 16-bit ones give, up to the
    # codes' steps: |y8 - y| <= sum |x| |dw| + |dx| |w| with every element off by
    # half a step of its row's scale
    say("expert block")
    g = gen(21)
    counts, n, k, bits = [60, 0, 7, 130], 200, 512, 7
    m, e = sum(counts), len(counts)
    x = torch.randn(m, k, generator=g, device="cuda")
    x[:, ::64] *= 30
    x = x.bfloat16()
    w = (torch.randn(e, n, k, generator=g, device="cuda") * k ** -0.5).bfloat16()
    ends = ends_of(counts)
    xq, xs = qse.rotate_quantize_int8(x, bits=bits)
    wq, ws = qse.rotate_quantize_int8(w.view(e * n, k), bits=bits)
    y8 = qse.grouped_matmul(xq, wq.view(e, n, k), ends, x_scales=xs, w_scales=ws.view(e, n),
                            out_dtype=torch.float32)
    want, _ = grouped_reference(x, w, counts, m)
    for i, lo, hi in group_bounds(counts):
        xr = hadamard_rows(x[lo:hi].double(), bits) * 2.0 ** (-bits / 2)
        wr = hadamard_rows(w[i].double(), bits) * 2.0 ** (-bits / 2)
        hx, hw = xs[lo:hi].double()[:, None] * 0.5001, ws.view(e, n)[i].double() * 0.5001
        tol = hx * wr.abs().sum(1) + xr.abs().sum(1)[:, None] * hw + hx * hw * k
        assert bool(((y8[lo:hi].double() - want[lo:hi]).abs() <= tol + 1e-6).all())
    # the dense product of one expert's rows is the grouped one's
    lo, hi = 67, 197
    assert torch.equal(y8[lo:hi], qse.int8_matmul(xq[lo:hi], xs[lo:hi], wq.view(e, n, k)[3],
                                                  ws.view(e, n)[3], out_dtype=torch.float32))


def test_captured_calls_follow_the_ends():
    # one graph, replayed with other inputs and other groups, between eager
    # calls; every replay against the eager results
    say("expert graph")
    g = gen(31)
    m, e, n, k = 300, 6, 264, 1024
    x = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(e, n, k, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    ends = torch.zeros(e, dtype=torch.int32, device="cuda")

    def step():
        y = qse.grouped_matmul(x, w, ends)
        dx, dw = qse.grouped_matmul_backward(x, w, ends, dy)
        q, s = qse.rotate_quantize_int8(x, bits=9)
        wq, ws = qse.rotate_quantize_int8(w.view(e * n, k), bits=9)
        y8 = qse.grouped_matmul(q, wq.view(e, n, k), ends, x_scales=s, w_scales=ws.view(e, n))
        z = qse.int8_matmul(q, s, wq[:n], ws[:n])
        return y, dx, dw, q, s, y8, z

    def fill(seed):
        gg = gen(seed)
        x.copy_(torch.randn(m, k, generator=gg, device="cuda"))
        w.copy_(torch.randn(e, n, k, generator=gg, device="cuda"))
        dy.copy_(torch.randn(m, n, generator=gg, device="cuda"))
        ends.copy_(ends_of(spread_counts(m - seed, e, seed)))

    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (2, 3, 50, 299, 2):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_a_given_stream():
    say("expert stream")
    g = gen(41)
    x = torch.randn(200, 512, generator=g, device="cuda").bfloat16()
    w = torch.randn(5, 128, 512, generator=g, device="cuda").bfloat16()
    dy = torch.randn(200, 128, generator=g, device="cuda").bfloat16()
    ends = ends_of([50, 0, 100, 1, 30])
    q, s = qse.rotate_quantize_int8(x)
    want = [qse.grouped_matmul(x, w, ends), *qse.grouped_matmul_backward(x, w, ends, dy), q, s,
            qse.int8_matmul(q, s, q, s)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = [qse.grouped_matmul(x, w, ends, stream=st),
           *qse.grouped_matmul_backward(x, w, ends, dy, stream=st)]
    got += [*qse.rotate_quantize_int8(x, stream=st), qse.int8_matmul(q, s, q, s, stream=st)]
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    say("expert refusals")
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 16, 64, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    ends = torch.tensor([3, 8], dtype=torch.int32, device="cuda")
    q, s = x.to(torch.int8), torch.ones(8, device="cuda")
    wq, ws = w.to(torch.int8), torch.ones(2, 16, device="cuda")
    gm, gb, im = qse.grouped_matmul, qse.grouped_matmul_backward, qse.int8_matmul
    calls = [
        lambda: gm(x.float(), w.float(), ends), lambda: gm(x, w.half(), ends),
        lambda: gm(x, w[0], ends), lambda: gm(x, w[:, :, :32], ends), lambda: gm(x[0], w, ends),
        lambda: gm(x, w[:0], ends[:0]),
        lambda: gm(x, w, ends.long()), lambda: gm(x, w, ends[:1]), lambda: gm(x, w, ends.cpu()),
        lambda: gm(x, w, ends[None]), lambda: gm(x, w, ends.repeat(2)[::2]),
        lambda: gm(x, w, ends, x_scales=s), lambda: gm(x, w, ends, out_dtype=torch.float32),
        lambda: gm(x, w, ends, out=dy.float()), lambda: gm(x, w, ends, out=dy[:4]),
        lambda: gm(x, w.transpose(1, 2).contiguous().transpose(1, 2), ends),
        lambda: gm(x, w[:1].expand(2, 16, 64), ends),
        lambda: gm(q, wq, ends), lambda: gm(q, wq, ends, x_scales=s),
        lambda: gm(q, wq, ends, x_scales=s, w_scales=ws[0]),
        lambda: gm(q, wq, ends, x_scales=s.half(), w_scales=ws),
        lambda: gm(q, wq, ends, x_scales=s, w_scales=ws, out_dtype=torch.int8),
        lambda: gm(q, w, ends, x_scales=s, w_scales=ws),
        lambda: gb(x, w, ends, dy[:4]), lambda: gb(x, w, ends, dy.half()),
        lambda: gb(q, wq, ends, dy),
        lambda: im(q, s, q, s[:4]), lambda: im(q, s, q[:, :32], s), lambda: im(x, s, x, s),
        lambda: im(q, s, q, s, out_dtype=torch.int32),
        lambda: im(q, s.cpu(), q, s), lambda: qse.rotate_quantize_int8(q),
        lambda: qse.rotate_quantize_int8(x[0]),
        lambda: qse.rotate_quantize_int8(x.float().requires_grad_()),
        lambda: gm(x.clone().requires_grad_(), w, ends),
        lambda: gm(x, w.clone().requires_grad_(), ends),
        lambda: im(q, s.clone().requires_grad_(), q, s),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    with torch.no_grad():
        gm(x.clone().requires_grad_(), w, ends)
    # rows that are not 16-byte aligned, outputs across operands
    big = torch.zeros(8, 70, dtype=torch.int8, device="cuda")
    for call in (lambda: im(big[:, 1:65], s, q, s), lambda: im(q, s, big[:, :64], s),
                 lambda: qse.rotate_quantize_int8(x[:, :63], bits=1),
                 lambda: gm(x, x[:, None, :16].expand(8, 4, 16)[:2].contiguous().repeat(1, 1, 4),
                            ends, out=x[:, :4])):
        with pytest.raises((qse.FwtError, ValueError)):
            call()


def test_empty_sizes():
    say("expert empty")
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    ends = torch.zeros(2, dtype=torch.int32, device="cuda")
    w = z(2, 16, 64)
    assert tuple(qse.grouped_matmul(z(0, 64), w, ends).shape) == (0, 16)
    assert tuple(qse.grouped_matmul(z(5, 64), z(2, 0, 64), ends).shape) == (5, 0)
    dx, dw = qse.grouped_matmul_backward(z(0, 64), w, ends, z(0, 16))
    assert tuple(dx.shape) == (0, 64) and bool((dw == 0).all())
    dx, dw = qse.grouped_matmul_backward(z(5, 64), z(2, 0, 64), ends, z(5, 0))
    assert bool((dx == 0).all()) and tuple(dw.shape) == (2, 0, 64)
    q, s = qse.rotate_quantize_int8(z(0, 64))
    assert tuple(q.shape) == (0, 64) and tuple(s.shape) == (0,)
    assert tuple(qse.int8_matmul(q, s, z(3, 64, d=torch.int8), s.new_ones(3)).shape) == (0, 3)


def test_operands_past_4_gib():
    say("expert 4 GiB")
    g = gen(51)
    # experts 2 GiB apart, rows 4 MiB apart
    n, k, e = 64, 256, 4
    store = torch.empty(e << 30, dtype=torch.bfloat16, device="cuda")
    w = store.as_strided((e, n, k), (1 << 30, 1 << 21, 1))
    w.copy_(torch.randn(e, n, k, generator=g, device="cuda"))
    far = torch.empty(1100 << 21, dtype=torch.bfloat16, device="cuda")
    x = far.as_strided((1100, k), (1 << 21, 1))
    x.copy_(torch.randn(1100, k, generator=g, device="cuda"))
    dy = torch.randn(1100, n, generator=g, device="cuda").bfloat16()
    for counts in ([20, 500, 30, 550], [3, 0, 4, 5]):
        m = sum(counts)
        ends = ends_of(counts)
        y = qse.grouped_matmul(x[1100 - m:], w, ends)
        assert torch.equal(y, qse.grouped_matmul(x[1100 - m:].contiguous(), w.contiguous(), ends))
        got = qse.grouped_matmul_backward(x[1100 - m:], w, ends, dy[:m])
        want = qse.grouped_matmul_backward(x[1100 - m:].contiguous(), w.contiguous(), ends, dy[:m])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        out = far.as_strided((m, n), (1 << 21, 1), 1 << 20)
        qse.grouped_matmul(x[1100 - m:].contiguous(), w, ends, out=out)
        assert torch.equal(out, y)
    q, s = qse.rotate_quantize_int8(x, bits=8)
    q2, s2 = qse.rotate_quantize_int8(x.contiguous(), bits=8)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    qf = far.view(torch.int8).as_strided((1000, k), (1 << 22, 1))
    qf.copy_(q[:1000])
    c = qse.int8_matmul(qf, s[:1000], qf[300:700], s[300:700])
    assert torch.equal(c, qse.int8_matmul(q[:1000], s[:1000], q[300:700], s[300:700]))


def test_many_rows_and_wide_results():
    # results past 4 GiB and many tiles
    say("expert wide")
    g = gen(61)
    m, n, k = 70000, 40000, 64
    a, b = codes(g, m, k), codes(g, n, k)
    sa, sb = some_scales(g, m), some_scales(g, n)
    c = qse.int8_matmul(a, sa, b, sb)
    for lo in (0, 33333, m - 300):
        assert torch.equal(c[lo:lo + 300], int8_result(a[lo:lo + 300], sa[lo:lo + 300], b, sb,
                                                       torch.bfloat16))
    del c
    counts = [30000, 1, 0, 39000]
    w = codes(g, 4, n // 2, k)
    sw = some_scales(g, 4, n // 2)
    y = qse.grouped_matmul(a, w, ends_of(counts), x_scales=sa, w_scales=sw, out_dtype=torch.float32)
    for e, lo, hi in group_bounds(counts):
        part = slice(max(lo, hi - 200), hi)
        assert torch.equal(y[part], int8_result(a[part], sa[part], w[e], sw[e], torch.float32))
    assert bool((y[sum(counts):] == 0).all())
