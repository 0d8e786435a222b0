"""Edges of the 8-bit integer products and of the products grouped by expert:
padding that is not a number, many experts, tiles shared by two workgroups,
strided gradients, two threads.  References and tolerances as in
test_gpu_experts.py."""
import ctypes
import threading

import pytest

import quantum_state_encoding_amd as qse
from quantum_state_encoding_amd import experts

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_experts import (DT, cdiv, check_sums, codes, ends_of, gen, group_bounds,  # noqa: E402
                              grouped_reference, int8_result, say, some_scales,
                              spread_counts)


def in_padding(t, rows=0):
    """t in rows padded to 16 bytes, NaN around it (no row behind the last)."""
    k = t.shape[-1]
    pad = cdiv(k, 8) * 8 + 8
    big = torch.full(t.shape[:-1] + (pad,), float("nan"), dtype=t.dtype, device="cuda")
    view = big[..., :k]
    view.copy_(t)
    return view


@pytest.mark.parametrize("counts,rest,n,k", [
    ([3, 0, 5, 1], 2, 70, 257), ([40, 1, 0, 33], 9, 129, 999), ([200, 0, 56], 0, 251, 61),
    ([130, 129, 0, 1, 300], 77, 500, 71), ([700], 0, 1003, 205), ([600, 500], 0, 2051, 139),
    ([1], 0, 5, 3), ([3000, 10, 1500, 0, 2000], 100, 3001, 267), ([300, 21], 5, 203, 9001),
])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_aligned_rows_with_padding_that_is_not_a_number(counts, rest, n, k, dtype):
    say("padding", counts, rest, n, k, dtype)
    g, dt = gen(n), DT[dtype]
    m, e = sum(counts) + rest, len(counts)
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(e, n, k, generator=g, device="cuda") * k ** -0.5).to(dt)
    dy = (torch.randn(m, n, generator=g, device="cuda") * 0.1).to(dt)
    xs, ws, ds, ends = in_padding(x), in_padding(w), in_padding(dy), ends_of(counts)
    used = m - rest
    xs[used:] = float("nan")
    ds[used:] = float("nan")
    y = qse.grouped_matmul(xs, ws, ends)
    want, mag = grouped_reference(x, w, counts, m)
    check_sums(y, want, mag, k, dt)
    dx, dw = qse.grouped_matmul_backward(xs, ws, ends, ds)
    assert bool((dx[used:] == 0).all())
    for i, lo, hi in group_bounds(counts):
        if hi == lo:
            assert bool((dw[i] == 0).all())
            continue
        gr, a, b = dy[lo:hi].double(), x[lo:hi].double(), w[i].double()
        check_sums(dx[lo:hi], gr @ b, gr.abs() @ b.abs(), n, dt)
        check_sums(dw[i], gr.t() @ a, gr.abs().t() @ a.abs(), hi - lo, dt)


def at_four_bytes(t):
    """t inside NaN, rows at multiples of 4 bytes, not all of 16."""
    k = t.shape[-1]
    ld = cdiv(k, 2) * 2 + 4
    ld += 2 if ld % 8 == 0 else 0
    big = torch.full(t.shape[:-1] + (ld,), float("nan"), dtype=t.dtype, device="cuda")
    view = big[..., 2:2 + k]
    view.copy_(t)
    return view


@pytest.mark.parametrize("counts,rest,n,k", [
    ([1], 0, 1, 1), ([2, 1], 1, 3, 2), ([3, 0, 5, 1], 2, 70, 257), ([9, 8], 1, 15, 7),
    ([40, 1, 0, 33], 9, 129, 998), ([200, 0, 56], 0, 250, 61), ([130, 129, 0, 1, 300], 77, 500, 70),
    ([700], 0, 1003, 206), ([600, 500], 0, 2050, 138), ([3000, 10, 1500, 0, 2000], 100, 3001, 266),
    ([300, 21], 5, 202, 9002), ([1] * 70, 3, 34, 130), ([257, 255, 2049], 3, 2046, 126),
    ([50, 100], 0, 6, 2002), ([50, 100], 0, 2002, 6), ([64], 0, 100, 16002), ([2600], 0, 66, 62),
])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_at_multiples_of_four_bytes(counts, rest, n, k, dtype):
    say("four bytes", counts[:5], rest, n, k, dtype)
    g, dt = gen(n + k), DT[dtype]
    m, e = sum(counts) + rest, len(counts)
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(e, n, k, generator=g, device="cuda") * k ** -0.5).to(dt)
    dy = (torch.randn(m, n, generator=g, device="cuda") * 0.1).to(dt)
    xs, ws, ds, ends = at_four_bytes(x), at_four_bytes(w), at_four_bytes(dy), ends_of(counts)
    for t in (xs, ws, ds):
        assert t.data_ptr() % 4 == 0 and all(s % 2 == 0 for s in t.stride()[:-1])
    used = m - rest
    xs[used:] = float("nan")
    ds[used:] = float("nan")
    y = qse.grouped_matmul(xs, ws, ends)
    want, mag = grouped_reference(x, w, counts, m)
    check_sums(y, want, mag, k, dt)
    dx, dw = qse.grouped_matmul_backward(xs, ws, ends, ds)
    assert bool((dx[used:] == 0).all())
    for i, lo, hi in group_bounds(counts):
        if hi == lo:
            assert bool((dw[i] == 0).all())
            continue
        gr, a, b = dy[lo:hi].double(), x[lo:hi].double(), w[i].double()
        check_sums(dx[lo:hi], gr @ b, gr.abs() @ b.abs(), n, dt)
        check_sums(dw[i], gr.t() @ a, gr.abs().t() @ a.abs(), hi - lo, dt)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("where", ["x", "w"])
def test_values_that_are_not_finite_stay_in_their_rows_and_columns(kind, where):
    say("not finite", kind, where)
    g = gen(7)
    for counts, n, k in (([3, 2, 0, 4], 40, 130), ([300, 70, 0, 600], 520, 328)):
        m, e = sum(counts), len(counts)
        if kind == "int8":
            x, w = codes(g, m, k), codes(g, e, n, k)
            kw = dict(x_scales=some_scales(g, m), w_scales=some_scales(g, e, n))
        else:
            x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
            w = torch.randn(e, n, k, generator=g, device="cuda").bfloat16()
            kw = {}
        ends = ends_of(counts)
        clean = qse.grouped_matmul(x, w, ends, **kw)
        keep = torch.ones_like(clean, dtype=torch.bool)
        if where == "x":
            keep[counts[0]] = False                  # a row of the second expert
            if kind == "int8":
                kw["x_scales"][counts[0]] = float("nan")
            else:
                x[counts[0], k - 1] = float("inf")
        else:
            keep[sum(counts[:3]):, n - 1] = False    # the last expert's last column
            if kind == "int8":
                kw["w_scales"][3, n - 1] = float("inf")
            else:
                w[3, n - 1, 0] = float("nan")
        y = qse.grouped_matmul(x, w, ends, **kw)
        assert torch.equal(y[keep], clean[keep])
        assert not bool(torch.isfinite(y[~keep]).any())


@pytest.mark.parametrize("e", [63, 64, 65, 127, 128, 129, 1000, 5000])
@pytest.mark.parametrize("m", [1, 50, 3000])
def test_many_experts(e, m):
    say("many experts", e, m)
    g = gen(e + m)
    n, k = 24, 32
    counts = spread_counts(m, e, e)
    x, w = codes(g, m + 3, k), codes(g, e, n, k)
    sx, sw = some_scales(g, m + 3), some_scales(g, e, n)
    y = qse.grouped_matmul(x, w, ends_of(counts), x_scales=sx, w_scales=sw)
    owner = torch.repeat_interleave(torch.arange(e), torch.tensor(counts)).cuda()
    sums = (x[:m].double()[:, None] * w[owner].double()).sum(2).float()
    assert torch.equal(y[:m], (sums * sx[:m, None] * sw[owner]).bfloat16())
    assert bool((y[m:] == 0).all())
    xh = torch.randn(m + 3, k, generator=g, device="cuda").half()
    wh = torch.randn(e, n, k, generator=g, device="cuda").half()
    dy = torch.randn(m + 3, n, generator=g, device="cuda").half()
    dx, dw = qse.grouped_matmul_backward(xh, wh, ends_of(counts), dy)
    want = (dy[:m].double()[:, :, None] * wh[owner].double()).sum(1)
    mag = (dy[:m].double()[:, :, None] * wh[owner].double()).abs().sum(1)
    check_sums(dx[:m], want, mag, n, torch.float16)
    assert bool((dx[m:] == 0).all())
    each = dy[:m].double()[:, :, None] * xh[:m].double()[:, None]
    want = torch.zeros(e, n, k, dtype=torch.float64, device="cuda").index_add_(0, owner, each)
    mag = torch.zeros(e, n, k, dtype=torch.float64, device="cuda").index_add_(0, owner, each.abs())
    check_sums(dw, want, mag, max(counts), torch.float16)


# sizes whose misaligned operands are copied into aligned rows first
COPIED = [([3089, 0, 415], 100, 1019, 3373), ([2500, 2200, 1], 0, 1510, 1001),
          ([1200] * 4, 7, 2001, 2004), ([4000], 333, 1999, 2000)]


def copied_operands(case, dt):
    counts, rest, n, k = COPIED[case]
    g = gen(case)
    m, e = sum(counts) + rest, len(counts)
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(e, n, k, generator=g, device="cuda") * k ** -0.5).to(dt)
    dy = (torch.randn(m, n, generator=g, device="cuda") * 0.1).to(dt)
    x[m - rest:] = float("nan")
    dy[m - rest:] = float("nan")
    for i, c in enumerate(counts):
        if c == 0:
            w[i] = float("nan")
    return counts, rest, n, k, x, w, dy


def check_copied(counts, rest, n, k, x, w, dy, y, dx, dw):
    dt, used = x.dtype, x.shape[0] - rest
    assert bool((y[used:] == 0).all()) and bool((dx[used:] == 0).all())
    for i, lo, hi in group_bounds(counts):
        if hi == lo:
            assert bool((dw[i] == 0).all())
            continue
        a, b, gr = x[lo:hi].double(), w[i].double(), dy[lo:hi].double()
        check_sums(y[lo:hi], a @ b.t(), a.abs() @ b.abs().t(), k, dt)
        check_sums(dx[lo:hi], gr @ b, gr.abs() @ b.abs(), n, dt)
        check_sums(dw[i], gr.t() @ a, gr.abs().t() @ a.abs(), hi - lo, dt)


@pytest.mark.parametrize("case", range(len(COPIED)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("strided", [0, 1])
def test_copied_operands(case, dtype, strided):
    say("copied", case, dtype, strided)
    counts, rest, n, k, x, w, dy = copied_operands(case, DT[dtype])
    ends = ends_of(counts)

    def lay(t):      # rows of an odd stride from an odd place, NaN around them
        if not strided:
            return t
        big = torch.full(t.shape[:-1] + (t.shape[-1] + 3 + t.shape[-1] % 2,), float("nan"),
                         dtype=t.dtype, device="cuda")
        view = big[..., 1:1 + t.shape[-1]]
        view.copy_(t)
        return view

    xs, ws, ds = lay(x), lay(w), lay(dy)
    y = qse.grouped_matmul(xs, ws, ends)
    dx, dw = qse.grouped_matmul_backward(xs, ws, ends, ds)
    check_copied(counts, rest, n, k, x, w, dy, y, dx, dw)
    assert torch.equal(qse.grouped_matmul(xs, ws, ends), y)
    again = qse.grouped_matmul_backward(xs, ws, ends, ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_copied_operands_scratch_and_parts():
    # scratch of the size that is asked for holds the sums and the copies; dx or dw
    # alone; no scratch
    L = experts._load()
    stream = torch.cuda.current_stream().cuda_stream
    asked = 0
    for case in range(len(COPIED)):
        say("copied scratch", case)
        counts, rest, n, k, x, w, dy = copied_operands(case, torch.bfloat16)
        m, e, ends = x.shape[0], len(counts), ends_of(counts)
        size = ctypes.c_size_t()
        for parts in (3, 1, 2, 0):
            assert L.fwt_grouped_matmul_workspace(0, e, m, n, k, ctypes.byref(size)) == 0
            need = size.value
            assert L.fwt_grouped_matmul_backward_workspace(e, m, n, k, ctypes.byref(size)) == 0
            need = max(need, size.value)
            asked = max(asked, need)
            ws = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
            at, room = (ws.data_ptr(), need) if parts else (None, 0)
            y = torch.empty(m, n, dtype=x.dtype, device="cuda")
            dx, dw = torch.full_like(x, 3.0), torch.full_like(w, 3.0)
            assert L.fwt_grouped_matmul(x.data_ptr(), k, None, w.data_ptr(), k, n * k, None,
                                        ends.data_ptr(), e, 0, m, n, k, y.data_ptr(), 0, n, 1,
                                        at, room, stream) == 0
            for which in ((3,) if parts in (0, 3) else (parts, 3 - parts)):
                assert L.fwt_grouped_matmul_backward(
                    x.data_ptr(), k, w.data_ptr(), k, n * k, ends.data_ptr(), e, dy.data_ptr(),
                    n, 0, m, n, k, dx.data_ptr() if which & 1 else None, k,
                    dw.data_ptr() if which & 2 else None, k, n * k, at, room, stream) == 0
            check_copied(counts, rest, n, k, x, w, dy, y, dx, dw)
            assert bool((ws[need:] == 0x5a).all())
    assert asked > 16 << 20          # (copies are among them)


def test_aligned_rows_take_no_scratch_for_copies():
    # sizes whose misaligned operands are copied, here in rows of multiples of 16 bytes:
    # a call allocates its results; one misaligned operand, room for that one more
    say("no scratch for copies")
    counts, rest, n, k = COPIED[0]
    m, e = sum(counts) + rest, len(counts)
    x, w = torch.randn(m, k, device="cuda").bfloat16(), torch.randn(e, n, k, device="cuda").bfloat16()
    dy = torch.randn(m, n, device="cuda").bfloat16()
    xs, ws, ds, ends = in_padding(x), in_padding(w), in_padding(dy), ends_of(counts)

    def peak(call):
        call()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        out = call()
        del out
        return torch.cuda.max_memory_allocated() - before

    results = 2 * m * n
    some = 1 << 20                    # (of the allocator's)
    assert peak(lambda: qse.grouped_matmul(xs, ws, ends)) <= results + some
    with_x = peak(lambda: qse.grouped_matmul(x, ws, ends))
    with_both = peak(lambda: qse.grouped_matmul(x, w, ends))
    copy = 2 * m * cdiv(k, 8) * 8
    assert with_x <= results + copy + some and with_both > results + copy + some
    grads = 2 * (m + e * n) * k
    assert peak(lambda: qse.grouped_matmul_backward(xs, ws, ends, ds)) <= grads + 2 * some


def test_copied_operands_that_begin_at_one_place():
    # x and grad are views of one buffer, of different widths
    say("copied, one place")
    counts, rest, n, k, _, w, _ = copied_operands(1, torch.bfloat16)
    big = torch.randn(sum(counts), 1511, generator=gen(9), device="cuda").bfloat16()
    x, dy = big[:, :k], big[:, :n]
    y = qse.grouped_matmul(x, w, ends_of(counts))
    dx, dw = qse.grouped_matmul_backward(x, w, ends_of(counts), dy)
    check_copied(counts, rest, n, k, x, w, dy, y, dx, dw)


def test_copied_operands_replayed():
    say("copied, replayed")
    counts, rest, n, k, x, w, dy = copied_operands(2, torch.float16)
    x[sum(counts):], dy[sum(counts):] = 1.0, 1.0
    ends = ends_of(counts)
    call = lambda: ((qse.grouped_matmul(x, w, ends),)                     # noqa: E731
                    + qse.grouped_matmul_backward(x, w, ends, dy))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for turn in range(4):
        x.copy_(torch.randn(x.shape, generator=gen(turn), device="cuda"))
        new = ends_of([[1200, 1200, 1200, 1200], [0, 4000, 10, 0], [4807, 0, 0, 0],
                       [1, 1, 1, 1]][turn])
        ends.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_falling_ends_of_very_many_experts():
    # every second of 2^16 experts claims all rows: 2^15 times 2^16 tiles of 128 x 128
    # and more, which 32 bits do not hold.  The rows are unspecified; nothing around
    # them is written, and rows of the weights that all experts share are what is read.
    e, m, n, k = 1 << 16, 1 << 20, 1040, 8
    tiles = (m // 128) * cdiv(n, 128)
    assert e // 2 * tiles > 2 ** 31
    say("falling ends", e, m, n, k)
    ends = torch.zeros(e, dtype=torch.int32, device="cuda")
    ends[::2] = m
    x = torch.ones(m, k, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(e, n, k, dtype=torch.bfloat16, device="cuda")
    around = torch.full((m + 16, n), -1.0, dtype=torch.bfloat16, device="cuda")
    qse.grouped_matmul(x, w, ends, out=around[8:m + 8])
    torch.cuda.synchronize()
    assert bool((around[:8] == -1).all()) and bool((around[m + 8:] == -1).all())
    rows = around[8:m + 8]
    assert bool(((rows == -1) | (rows == k)).all())
    # and the next call is right
    y = qse.grouped_matmul(x[:100], w[:3], ends_of([40, 0, 60]))
    assert bool((y == k).all())


def falling_ends(m, kind):
    """Ends that fall, and for each row the experts that claim it."""
    half = m // 2
    if kind == "last":          # the rows of the second half are the last expert's alone
        ends = [half, 0] * 40 + [half, m]
    elif kind == "none":        # ... are no expert's
        ends = [half, 0] * 40
    elif kind == "middle":      # a part is a middle expert's alone, of the second 64
        ends = [half - 5, 0] * 45 + [half - 5, half + 7] + [half + 7] * 3 + [m, half + 9] * 3 + [m]
    else:
        g = torch.Generator()
        g.manual_seed(kind)
        ends = (torch.randint(-m // 8, m * 9 // 8, (7 + 30 * kind,), generator=g)).tolist()
        ends[3:3] = [m // 3] * 2
    cut = [0] + [min(max(v, 0), m) for v in ends]
    claims = [[] for _ in range(m)]
    for e, (lo, hi) in enumerate(zip(cut, cut[1:])):
        for r in range(lo, hi):
            claims[r].append(e)
    return ends, claims, cut[-1]


@pytest.mark.parametrize("m,n,k", [(40, 64, 64), (300, 200, 512), (1000, 200, 60), (2000, 1000, 61),
                                   (4096, 2048, 64), (300, 130, 4096)])
@pytest.mark.parametrize("kind", ["last", "none", "middle", 1, 2, 3])
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_falling_ends_leave_the_other_rows(m, n, k, kind, dtype):
    # rows that one expert alone claims are that expert's, rows that none does are
    # zeros, however often the other ends fall.  Small integers: sums are exact.
    if dtype == "int8" and k % 16:
        k = cdiv(k, 16) * 16
    say("falling ends, other rows", m, n, k, kind, dtype)
    L = experts._load()
    g = gen(n)
    stream = torch.cuda.current_stream().cuda_stream
    ends, claims, last = falling_ends(m, kind)
    e = len(ends)
    one = [r for r in range(m) if len(claims[r]) == 1 and r < last]
    none = [r for r in range(m) if not claims[r]]
    assert one or none or isinstance(kind, int)
    sparse = lambda *shape: (torch.rand(*shape, generator=g, device="cuda") < 32 / shape[-1]).float() \
        * torch.randint(-1, 2, shape, generator=g, device="cuda")                    # noqa: E731
    dt = torch.int8 if dtype == "int8" else torch.bfloat16
    x, w, dy = sparse(m, k), sparse(e, n, k), sparse(m, n)
    dev = torch.tensor(ends, dtype=torch.int32, device="cuda")
    rows = torch.tensor(one, dtype=torch.int64, device="cuda")
    whose = torch.tensor([claims[r][0] for r in one], dtype=torch.int64, device="cuda")
    empty = torch.tensor(none, dtype=torch.int64, device="cuda")
    x8, w8 = x.to(dt), w.to(dt)
    sx, sw = torch.ones(m, device="cuda"), torch.ones(e, n, device="cuda")
    y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert L.fwt_grouped_matmul(
        x8.data_ptr(), k, sx.data_ptr() if dtype == "int8" else None, w8.data_ptr(), k, n * k,
        sw.data_ptr() if dtype == "int8" else None, dev.data_ptr(), e, 5 if dtype == "int8" else 0,
        m, n, k, y.data_ptr(), 0, n, 1, None, 0, stream) == 0

    def check(got, a, b):
        assert bool((got[empty] == 0).all())
        for i in whose.unique().tolist():
            mine = rows[whose == i]
            assert torch.equal(got[mine].float(), a[mine] @ b(i))
        assert not bool(torch.isnan(got.float()).any())       # every row is written

    check(y, x, lambda i: w[i].t().contiguous())
    if dtype == "int8":
        return
    dx = torch.full((m, k), float("nan"), dtype=torch.bfloat16, device="cuda")
    d8 = dy.to(dt)
    dw = torch.full((e, n, k), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert L.fwt_grouped_matmul_backward(
        x8.data_ptr(), k, w8.data_ptr(), k, n * k, dev.data_ptr(), e, d8.data_ptr(), n, 0, m, n, k,
        dx.data_ptr(), k, dw.data_ptr(), k, n * k, None, 0, stream) == 0
    check(dx, dy, lambda i: w[i])
    assert not bool(torch.isnan(dw.float()).any())


def test_falling_ends_with_copied_operands():
    # the last expert's rows are its own, in sizes whose operands are copied first
    say("falling ends, copied")
    counts, rest, n, k, x, w, dy = copied_operands(0, torch.bfloat16)
    used = sum(counts)
    ends = torch.tensor([1500, 0, used], dtype=torch.int32, device="cuda")
    y = qse.grouped_matmul(x, w, ends)
    dx, dw = qse.grouped_matmul_backward(x, w, ends, dy)
    assert bool((y[used:] == 0).all()) and bool((dx[used:] == 0).all())
    a, b, gr = x[1500:used].double(), w[2].double(), dy[1500:used].double()
    check_sums(y[1500:used], a @ b.t(), a.abs() @ b.abs().t(), k, torch.bfloat16)
    check_sums(dx[1500:used], gr @ b, gr.abs() @ b.abs(), n, torch.bfloat16)
    assert bool(torch.isfinite(y.float()).all()) and bool(torch.isfinite(dx.float()).all())


@pytest.mark.parametrize("counts,n", [
    # whole rounds of 256 tiles and a few more, which two workgroups share each:
    # of more and of fewer than half a tile's rows, with rows of no expert
    ([2049] * 4, 4096), ([2048 + 128] * 4, 4096), ([2048 + 129] * 4, 4096),
    ([8192 + 1], 2048), ([2300, 1700, 4196], 2050), ([256] * 33, 2048), ([100] * 80, 2048),
    ([4096 + 256], 4096),
])
@pytest.mark.parametrize("rest", [0, 700])
def test_last_tiles_shared_by_two(counts, n, rest):
    say("halves", counts[:4], len(counts), n, rest)
    g = gen(len(counts) + n)
    m, e, k = sum(counts) + rest, len(counts), 320
    x, w = codes(g, m, k), codes(g, e, n, k)
    sx, sw = some_scales(g, m), some_scales(g, e, n)
    ends = ends_of(counts)
    y = qse.grouped_matmul(x, w, ends, x_scales=sx, w_scales=sw)
    for i, lo, hi in group_bounds(counts):
        assert torch.equal(y[lo:hi], int8_result(x[lo:hi], sx[lo:hi], w[i], sw[i], torch.bfloat16))
    assert bool((y[m - rest:] == 0).all())
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    qse.grouped_matmul(x, w, ends, x_scales=sx, w_scales=sw, out=out)
    assert torch.equal(out[:m - rest], y[:m - rest]) and bool((out[m - rest:] == 7.0).all())
    xh = x.bfloat16()
    wh = (w[:, :, :64] // 16).bfloat16()
    z = qse.grouped_matmul(xh[:, :64], wh, ends)
    for i, lo, hi in list(group_bounds(counts))[::7]:
        a, b = xh[lo:hi, :64].double(), wh[i].double()
        check_sums(z[lo:hi], a @ b.t(), a.abs() @ b.abs().t(), 64, torch.bfloat16)
    assert bool((z[m - rest:] == 0).all())


def test_strided_gradients_through_the_entry_point():
    say("strided gradients")
    L = experts._load()
    g = gen(3)
    stream = torch.cuda.current_stream().cuda_stream
    for counts, rest, n, k in (([50, 0, 70], 9, 40, 72), ([600, 300, 0, 500], 30, 520, 264),
                               ([50, 0, 70], 9, 41, 73)):
        m, e = sum(counts) + rest, len(counts)
        x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
        w = torch.randn(e, n, k, generator=g, device="cuda").bfloat16()
        dy = torch.randn(m, n, generator=g, device="cuda").bfloat16()
        ends = ends_of(counts)
        want = qse.grouped_matmul_backward(x, w, ends, dy)
        bx = torch.full((m, k + 13), 7.0, dtype=torch.bfloat16, device="cuda")
        bw = torch.full((e, n + 2, k + 5), 7.0, dtype=torch.bfloat16, device="cuda")
        dx, dw = bx[:, 5:5 + k], bw[:, 1:1 + n, 3:3 + k]

        def call(dxp, dwp):
            return L.fwt_grouped_matmul_backward(
                x.data_ptr(), k, w.data_ptr(), k, n * k, ends.data_ptr(), e, dy.data_ptr(), n, 0,
                m, n, k, dxp, k + 13, dwp, k + 5, (n + 2) * (k + 5), None, 0, stream)

        assert call(dx.data_ptr(), None) == 0
        check = torch.full_like(bw, 7.0)
        assert torch.equal(bw, check)            # dw was not asked for
        assert call(None, dw.data_ptr()) == 0
        assert torch.equal(dx, want[0])
        gr, a = dy.double(), x.double()
        for i, lo, hi in group_bounds(counts):
            check_sums(dw[i], gr[lo:hi].t() @ a[lo:hi], gr[lo:hi].abs().t() @ a[lo:hi].abs(),
                       max(hi - lo, 1), torch.bfloat16)
        dx.fill_(7.0)
        dw.fill_(7.0)
        assert bool((bx == 7.0).all()) and bool((bw == 7.0).all())


def test_rows_of_no_expert_through_the_entry_point():
    say("zero_rest")
    L = experts._load()
    g = gen(4)
    m, n, k = 90, 33, 64
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(2, n, k, generator=g, device="cuda").bfloat16()
    ends = ends_of([20, 30])
    for zero in (0, 1):
        y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
        assert L.fwt_grouped_matmul(x.data_ptr(), k, None, w.data_ptr(), k, n * k, None,
                                    ends.data_ptr(), 2, 0, m, n, k, y.data_ptr(), 0, n, zero, None,
                                    0, torch.cuda.current_stream().cuda_stream) == 0
        assert bool((y[50:] == (0.0 if zero else 7.0)).all())


def test_results_do_not_depend_on_where_a_group_lies():
    # an expert's rows give the same bits in any group of the same call's sizes
    say("place")
    g = gen(9)
    n, k = 300, 520
    x = torch.randn(400, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(1, n, k, generator=g, device="cuda").bfloat16().expand(4, n, k).contiguous()
    first = qse.grouped_matmul(x, w, ends_of([400, 0, 0, 0]))
    for counts in ([0, 400, 0, 0], [100, 100, 100, 100], [1, 398, 0, 1], [33, 0, 367, 0]):
        assert torch.equal(qse.grouped_matmul(x, w, ends_of(counts)), first)


def test_two_threads_on_streams_of_their_own():
    say("threads")
    g = gen(5)
    counts = [100, 0, 350, 50]
    x = torch.randn(500, 2048, generator=g, device="cuda").bfloat16()
    w = torch.randn(4, 256, 2048, generator=g, device="cuda").bfloat16()
    dy = torch.randn(500, 256, generator=g, device="cuda").bfloat16()
    ends = ends_of(counts)

    def calls():
        q, s = qse.rotate_quantize_int8(x, bits=11)
        wq, ws = qse.rotate_quantize_int8(w.view(-1, 2048), bits=11)
        return [qse.grouped_matmul(x, w, ends), *qse.grouped_matmul_backward(x, w, ends, dy), q, s,
                qse.grouped_matmul(q, wq.view(4, 256, 2048), ends, x_scales=s,
                                   w_scales=ws.view(4, 256)),
                qse.int8_matmul(q[:300], s[:300], wq[:200], ws[:200])]

    want = calls()
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = calls()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_a_given_stream_keeps_the_operands():
    # the operands' memory is not handed out again before the stream has passed
    say("kept operands")
    g = gen(6)
    side = torch.cuda.Stream()
    base = torch.randn(512, 4096, generator=g, device="cuda").bfloat16()
    w = torch.randn(4, 512, 4096, generator=g, device="cuda").bfloat16()
    ends = ends_of([100, 200, 12, 200])
    want = qse.grouped_matmul(base, w, ends)
    torch.cuda.synchronize()
    for _ in range(10):
        x = base.clone()
        torch.cuda.synchronize()
        for _ in range(20):
            got = qse.grouped_matmul(x, w, ends, stream=side)
        del x
        junk = torch.full((512, 4096), 9.0, dtype=torch.bfloat16, device="cuda")
        side.synchronize()
        assert torch.equal(got, want)
        del junk


def test_outputs_count_as_written():
    say("written")
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, 8, 16, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    before = out._version
    qse.grouped_matmul(x, w, ends_of([4]), out=out)
    assert out._version > before
    before = out._version
    q, s = x.to(torch.int8), torch.ones(4, device="cuda")
    qse.int8_matmul(q, s, q[:1].expand(8, 16).contiguous(), torch.ones(8, device="cuda"), out=out)
    assert out._version > before


@pytest.mark.parametrize("dtype,counts,n,k", [
    ("bf16", [8], 512, 16384), ("f16", [16], 128, 16384), ("bf16", [3, 0, 6, 1], 48, 18448),
    ("bf16", [1], 40, 30000), ("int8", [12], 213, 32608), ("int8", [4, 0, 9], 92, 28672),
    ("bf16", [2, 3], 100, 12345),
])
def test_few_rows_share_a_long_contraction(dtype, counts, n, k):
    # the binding offers the scratch that the library wants for up to 16 rows too, so its
    # results are the bits of a call through the entry point that has it
    say("few rows, long contraction", dtype, counts, n, k)
    L = experts._load()
    m, e, g = sum(counts), len(counts), gen(n)
    kw = {}
    if dtype == "int8":
        x, w = codes(g, m, k), codes(g, e, n, k)
        kw = dict(x_scales=some_scales(g, m), w_scales=some_scales(g, e, n))
    else:
        x = torch.randn(m, k, generator=g, device="cuda").to(DT[dtype])
        w = (torch.randn(e, n, k, generator=g, device="cuda") * k ** -0.5).to(DT[dtype])
    ends, size, code = ends_of(counts), ctypes.c_size_t(), {"bf16": 0, "f16": 1, "int8": 5}[dtype]
    assert L.fwt_grouped_matmul_workspace(code, e, m, n, k, ctypes.byref(size)) == 0
    assert size.value > 1 << 19
    ws = torch.empty(size.value, dtype=torch.uint8, device="cuda")
    out = 1 if dtype == "f16" else 0
    want = torch.empty(m, n, dtype=DT["f16" if out else "bf16"], device="cuda")
    ptr = lambda t: None if t is None else t.data_ptr()                             # noqa: E731
    assert L.fwt_grouped_matmul(
        x.data_ptr(), k, ptr(kw.get("x_scales")), w.data_ptr(), k, n * k, ptr(kw.get("w_scales")),
        ends.data_ptr(), e, code, m, n, k, want.data_ptr(), out, n, 1, ws.data_ptr(), size.value,
        torch.cuda.current_stream().cuda_stream) == 0
    del ws
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    y = qse.grouped_matmul(x, w, ends, **kw)
    assert torch.cuda.max_memory_allocated() - before >= size.value
    assert torch.equal(y, want)
    for i, lo, hi in group_bounds(counts):
        if hi > lo and dtype == "int8":
            assert torch.equal(y[lo:hi], int8_result(x[lo:hi], kw["x_scales"][lo:hi], w[i],
                                                     kw["w_scales"][i], torch.bfloat16))
        elif hi > lo:
            a, b = x[lo:hi].double(), w[i].double()
            check_sums(y[lo:hi], a @ b.t(), a.abs() @ b.abs().t(), k, x.dtype)


def test_operands_with_tangents_are_refused():
    say("tangents")
    from torch.autograd import forward_ad
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, 8, 16, dtype=torch.bfloat16, device="cuda")
    q, s, ws = x.to(torch.int8), torch.ones(4, device="cuda"), torch.ones(1, 8, device="cuda")
    ends = ends_of([4])
    wq, e4, es = w.to(torch.int8), x.to(torch.float8_e4m3fn), torch.ones(1, 4, device="cuda")
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))               # noqa: E731
        for call in (lambda: qse.rotate_quantize_int8(dual(x)), lambda: qse.rotate_quantize(dual(x)),
                     lambda: qse.grouped_matmul(dual(x), w, ends),
                     lambda: qse.grouped_matmul(x, dual(w), ends),
                     lambda: qse.grouped_matmul(x, w, ends, out=dual(x[:, :8].clone())),
                     lambda: qse.grouped_matmul(q, wq, ends, x_scales=dual(s), w_scales=ws),
                     lambda: qse.int8_matmul(q, dual(s), q, s),
                     lambda: qse.scaled_matmul(e4, dual(es), e4, es),
                     lambda: qse.gated_ffn(x, dual(w[0]), w[0])):
            with pytest.raises(ValueError, match="tangent"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                call()
        qse.grouped_matmul(dual(x).detach(), w, ends)


def test_workspaces_are_enough_for_every_number_of_groups():
    # the scratch that is asked for holds the sums whatever zero_rest is: what
    # lies behind it stays as it was
    say("workspace")
    L = experts._load()
    stream = torch.cuda.current_stream().cuda_stream
    for e, m, n, k in ((1, 17, 64, 4096), (2, 100, 100, 16000), (7, 921, 300, 2048), (3, 400, 500, 3000),
                       (5, 64, 128, 8192), (85, 85, 64, 2048), (1, 2000, 1000, 1000)):
        size = ctypes.c_size_t()
        for dtype, tdt in ((0, torch.bfloat16), (5, torch.int8)):
            if dtype == 5 and k % 16:
                continue
            assert L.fwt_grouped_matmul_workspace(dtype, e, m, n, k, ctypes.byref(size)) == 0
            ws = torch.full((size.value + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
            counts = spread_counts(m, e, m)
            g = gen(m)
            ends = ends_of(counts)
            if dtype == 5:
                x, w = codes(g, m, k), codes(g, e, n, k)
                sx, sw = some_scales(g, m), some_scales(g, e, n)
            else:
                x = torch.randn(m, k, generator=g, device="cuda").to(tdt)
                w = torch.randn(e, n, k, generator=g, device="cuda").to(tdt)
                sx = sw = None
            ys = []
            for zero in (0, 1):
                y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
                assert L.fwt_grouped_matmul(
                    x.data_ptr(), k, sx.data_ptr() if dtype else None, w.data_ptr(), k, n * k,
                    sw.data_ptr() if dtype else None, ends.data_ptr(), e, dtype, m, n, k,
                    y.data_ptr(), 0, n, zero, ws.data_ptr() if size.value else None, size.value,
                    stream) == 0
                ys.append(y)
            assert bool((ws[size.value:] == 0x5a).all())
            assert torch.equal(ys[0], ys[1])
            want, mag = (None, None) if dtype else grouped_reference(x, w, counts, m)
            if not dtype:
                check_sums(ys[0], want, mag, k, torch.bfloat16)
            else:
                for i, lo, hi in group_bounds(counts):
                    assert torch.equal(ys[0][lo:hi], int8_result(x[lo:hi], sx[lo:hi], w[i], sw[i],
                                                                 torch.bfloat16))
