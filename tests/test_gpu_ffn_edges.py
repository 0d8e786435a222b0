"""The feed-forward operators on the GPU where a size, a stride, a type's range
or a value that is not finite is at its border.

Tolerances as in test_gpu_ffn.py: half(t) = finfo(t).eps / 2 for a rounding,
2 U a term for fp32 sums.
"""
import math

import pytest

import quantum_state_encoding_amd as qse

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BLOCK = 128
U = 2.0 ** -24
F8 = torch.float8_e4m3fn
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


def integers(g, rows, cols, dtype):
    return torch.randint(-4, 5, (rows, cols), generator=g, device="cuda").float().to(dtype)


# ---- rows past an operand's last -------------------------------------------

def before_nan(t, ld, rows):
    """t in rows of ld elements, with `rows` rows of NaN behind its last."""
    big = torch.full((t.shape[0] + rows, ld), float("nan"), device="cuda").to(t.dtype)
    big[:t.shape[0], :t.shape[1]] = t
    return big[:t.shape[0], :t.shape[1]]


# few rows in the last tile of each size (64, 128 and 256 rows), so that most
# of its rows lie behind the operand
@pytest.mark.parametrize("m,n,k", [(33, 17, 96), (65, 130, 144), (129, 257, 272), (257, 129, 80),
                                   (2049, 4097, 96), (1025, 8193, 64), (66, 70, 4096)])
def test_rows_behind_an_operand_are_not_used(m, n, k):
    # integers: every sum is exact, whatever tile takes it
    say("rows behind", m, n, k)
    g = gen(m + n + k)
    a, b = integers(g, m, k, F8), integers(g, n, k, F8)
    ones = [torch.ones(cdiv(k, BLOCK), r, device="cuda") for r in (m, n)]
    want = a.float() @ b.float().t()
    for ld in (k + 16, 1 << 13):
        fa, fb = before_nan(a, ld, 300), before_nan(b, ld, 300)
        for out in (torch.float32, torch.bfloat16):
            c = qse.scaled_matmul(fa, ones[0], fb, ones[1], out_dtype=out)
            assert torch.equal(c, want.to(out))
    x, wg, wu, dh = (integers(g, r, c, torch.bfloat16) * 0.0625
                     for r, c in ((m, k), (n, k), (n, k), (m, n)))
    h = qse.gated_ffn(x, wg, wu)
    grads = qse.gated_ffn_backward(x, wg, wu, dh)
    for ld in (k + 8, 1 << 13):
        fx, fg, fu = (before_nan(t, ld, 300) for t in (x, wg, wu))
        assert torch.equal(qse.gated_ffn(fx, fg, fu), h)
        got = qse.gated_ffn_backward(fx, fg, fu, before_nan(dh, n + 3, 2))
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
