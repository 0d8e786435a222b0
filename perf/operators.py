"""Cases of the feed-forward operators around the Walsh-Hadamard rotation,
for timing and for comparing the library's kernels with a plain form.

Four operators, used one after another in an 8-bit feed-forward block:

* ``rotate_quantize``: x times I (x) H_b along the contraction axis (H_b the
  normalised Walsh-Hadamard matrix of 2^b), then e4m3 codes with one fp32
  scale for each block of 128 (of a row, or of a 128 x 128 tile);
* ``scaled_matmul``: the product of two such operands, scales[k block] per
  row of the left one, per row or per tile of the right one;
* ``gated_ffn``: act(x Wg^T) * (x Wu^T), on 16-bit or on e4m3 operands;
* ``gated_ffn_backward``: its gradients for x, Wg and Wu.

``run`` computes the plain form in 32 bits with elementary torch operations,
or, with ``own`` set, calls the library.
"""
import math

import torch

own = False

BLOCK = 128      # contraction elements that share a scale
TOP = 448.0      # largest e4m3 value
TINY = 2.0 ** -126

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token's activations before an 8-bit projection: latency
        dict(name="rotate_token", op="rotate_quantize", m=1, k=4096, bits=12, dtype="bf16",
             scales="row", transpose=False),
        # the hidden activations of a long prompt, rotated over the whole row
        dict(name="rotate_prompt", op="rotate_quantize", m=8192, k=16384, bits=14, dtype="bf16",
             scales="row", transpose=False),
        # a weight matrix prepared for serving: one scale for a 128 x 128 tile
        dict(name="rotate_weight", op="rotate_quantize", m=4096, k=16384, bits=10, dtype="f32",
             scales="tile", transpose=False),
        # an output gradient for the weight gradient's product: blocks of 128
        # tokens, the codes transposed, a ragged number of tokens
        dict(name="rotate_grad_t", op="rotate_quantize", m=8192, k=4000, bits=5, dtype="bf16",
             scales="row", transpose=True),
        # one token through a down projection: the weights' bytes
        dict(name="matmul_token", op="scaled_matmul", m=1, n=4096, k=16384, right="tile",
             out="bf16"),
        # a short ragged prompt
        dict(name="matmul_ragged", op="scaled_matmul", m=333, n=4100, k=2056, right="tile",
             out="f16"),
        # a long prompt through a down projection
        dict(name="matmul_prompt", op="scaled_matmul", m=8192, n=4096, k=16384, right="tile",
             out="bf16"),
        # a weight gradient: both operands in blocks along the tokens, fp32 out
        dict(name="matmul_wgrad", op="scaled_matmul", m=4096, n=4096, k=8192, right="row",
             out="f32"),
        # eight sequences' next tokens through a 16-bit gated block
        dict(name="gated_decode", op="gated_ffn", m=8, n=16384, k=4096, dtype="bf16",
             act="silu"),
        # sizes that are multiples of nothing
        dict(name="gated_odd", op="gated_ffn", m=1021, n=5501, k=2047, dtype="f16",
             act="gelu"),
        # a training step's gradients
        dict(name="gated_backward", op="gated_ffn_backward", m=4096, n=8192, k=4096,
             dtype="bf16", act="silu"),
        # a long prompt through an 8-bit gated block
        dict(name="gated_fp8_prompt", op="gated_ffn", m=8192, n=16384, k=4096, dtype="e4m3",
             act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the logarithm of their ranges, half of the
    contraction lengths odd or ragged."""
    op = rng.choice(["rotate_quantize", "scaled_matmul", "gated_ffn", "gated_ffn_backward"])
    while True:
        if op == "rotate_quantize":
            transpose = rng.random() < 0.4
            bits = rng.randint(0, 7 if transpose else 14)
            m, k = _log(rng, 1, 8192), _log(rng, 64, 16384)
            k = max(1, k >> bits) << bits
            c = dict(op=op, m=m, k=k, bits=bits, dtype=rng.choice(["bf16", "f16", "f32"]),
                     scales=rng.choice(["row", "tile"]), transpose=transpose)
            if m * k <= 8192 * 16384:
                return c
            continue
        m = _log(rng, 1, 8192)
        n, k = _log(rng, 64, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.5:
            n, k = max(16, n // 16 * 16), max(16, k // 16 * 16)
        if op == "scaled_matmul":
            c = dict(op=op, m=m, n=n, k=k, right=rng.choice(["row", "tile"]),
                     out=rng.choice(["bf16", "f16", "f32"]))
            most = 2 * 8192 * 4096 * 16384
        elif op == "gated_ffn":
            c = dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "f16", "e4m3"]),
                     act=rng.choice(["silu", "gelu"]))
            most = 4 * 8192 * 16384 * 4096
        else:
            m = max(m, 16)
            c = dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "f16"]),
                     act=rng.choice(["silu", "gelu"]))
            most = 12 * 4096 * 8192 * 4096
        if work(c)["flops"] <= most:
            return c


def _ceil(a, b):
    return -(-a // b)


def work(case):
    """Each input read once, each output written once; the products'
    operations, and one addition for each element and rotation stage."""
    m, k = case["m"], case["k"]
    kb = _ceil(k, BLOCK)
    if case["op"] == "rotate_quantize":
        size = 4 if case["dtype"] == "f32" else 2
        ns = kb * (m if case["scales"] == "row" else _ceil(m, BLOCK))
        return {"bytes": m * k * (size + 1) + 4 * ns, "flops": m * k * (case["bits"] + 2)}
    n = case["n"]
    if case["op"] == "scaled_matmul":
        nb = n if case["right"] == "row" else _ceil(n, BLOCK)
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": (m + n) * k + 4 * kb * (m + nb) + m * n * out, "flops": 2 * m * n * k}
    if case["op"] == "gated_ffn":
        if case["dtype"] == "e4m3":
            ops = (m + 2 * n) * k + 4 * kb * (m + 2 * _ceil(n, BLOCK))
        else:
            ops = 2 * (m + 2 * n) * k
        return {"bytes": ops + 2 * m * n, "flops": 4 * m * n * k}
    return {"bytes": 2 * (2 * (m + 2 * n) * k + m * n), "flops": 12 * m * n * k}


# ---- inputs ---------------------------------------------------------------

def _activations(g, rows, cols, dtype):
    """N(0, 1) with about one channel in 64 thirty times as large, as the
    activations that a rotation is used for have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.rand(cols, generator=g, device="cuda") < 1.0 / 64
    return x.mul_(torch.where(loud, 30.0, 1.0)).to(dtype)


def _weights(g, rows, cols, dtype):
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return x.mul_(cols ** -0.5).to(dtype)


def _codes(x, scales):
    """e4m3 codes of x (rows padded to a multiple of 16 bytes) and scales."""
    m, k = x.shape
    kb, mb = _ceil(k, BLOCK), _ceil(m, BLOCK)
    full = torch.zeros(mb * BLOCK, kb * BLOCK, device="cuda")
    full[:m, :k] = x
    if scales == "row":
        v = full[:m].view(m, kb, BLOCK)
        s = (v.abs().amax(2) / TOP).clamp_min(TINY)
        q = (v / s[:, :, None]).view(m, kb * BLOCK)
    else:
        v = full.view(mb, BLOCK, kb, BLOCK)
        s = (v.abs().amax((1, 3)) / TOP).clamp_min(TINY)
        q = (v / s[:, None, :, None]).view(mb * BLOCK, kb * BLOCK)[:m]
    kp = _ceil(k, 16) * 16
    q = q[:, :kp].clamp(-TOP, TOP).to(torch.float8_e4m3fn).contiguous()[:, :k]
    return q, s.t().contiguous()


def _hadamard(bits):
    h = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(bits):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h * 2.0 ** (-bits / 2)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "rotate_quantize":
        shape = (k, m) if case["transpose"] else (m, k)
        x = _activations(g, *shape, DTYPES[case["dtype"]])
        return {"x": x}
    n = case["n"]
    if op == "scaled_matmul":
        a, sa = _codes(_activations(g, m, k, torch.float32), "row")
        b, sb = _codes(_weights(g, n, k, torch.float32), case["right"])
        return {"a": a, "sa": sa, "b": b, "sb": sb}
    f8 = case["dtype"] == "e4m3"
    dt = torch.float32 if f8 else DTYPES[case["dtype"]]
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    wg, wu = _weights(g, n, k, dt), _weights(g, n, k, dt)
    if f8:
        (x, sx), (wg, sg), (wu, su) = _codes(x, "row"), _codes(wg, "tile"), _codes(wu, "tile")
        return {"x": x, "sx": sx, "wg": wg, "sg": sg, "wu": wu, "su": su}
    if op == "gated_ffn":
        return {"x": x, "wg": wg, "wu": wu}
    grad = torch.randn(m, n, generator=g, device="cuda").mul_(0.1).to(dt)
    return {"x": x, "wg": wg, "wu": wu, "grad": grad}


def prepare(case, seed):
    state = dict(case=dict(case), **_inputs(case, seed))
    if case["op"] == "rotate_quantize":
        b = case["bits"]
        # the two Kronecker factors that the plain form multiplies by
        state["h_low"] = _hadamard(b // 2).float().cuda()
        state["h_high"] = _hadamard(b - b // 2).float().cuda()
    return state


# ---- one pass -------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _library(case, state)
    return {"rotate_quantize": _plain_rotate, "scaled_matmul": _plain_matmul,
            "gated_ffn": _plain_gated, "gated_ffn_backward": _plain_backward}[case["op"]](
                case, state)


def _library(case, st):
    import quantum_state_encoding_amd as qse
    if case["op"] == "rotate_quantize":
        return qse.rotate_quantize(st["x"], bits=case["bits"], scales=case["scales"],
                                   transpose=case["transpose"])
    if case["op"] == "scaled_matmul":
        return qse.scaled_matmul(st["a"], st["sa"], st["b"], st["sb"],
                                 out_dtype=DTYPES[case["out"]])
    if case["op"] == "gated_ffn":
        if case["dtype"] == "e4m3":
            return qse.gated_ffn(st["x"], st["wg"], st["wu"], act=case["act"],
                                 x_scales=st["sx"], gate_scales=st["sg"], up_scales=st["su"],
                                 out_dtype=torch.bfloat16)
        return qse.gated_ffn(st["x"], st["wg"], st["wu"], act=case["act"])
    return qse.gated_ffn_backward(st["x"], st["wg"], st["wu"], st["grad"], act=case["act"])


def _plain_rotate(case, st):
    m, k, bits = case["m"], case["k"], case["bits"]
    kb, mb = _ceil(k, BLOCK), _ceil(m, BLOCK)
    x = st["x"].float()
    x = x.t() if case["transpose"] else x
    x = x.reshape(m * (k >> bits), 1 << (bits - bits // 2), 1 << (bits // 2))
    x = torch.matmul(x, st["h_low"]) if bits > 1 else x
    x = torch.matmul(st["h_high"], x) if bits else x
    full = torch.nn.functional.pad(x.reshape(m, k), (0, kb * BLOCK - k, 0, mb * BLOCK - m))
    if case["scales"] == "row":
        v = full[:m].view(m, kb, BLOCK)
        s = (v.abs().amax(2) / TOP).clamp_min(TINY)
        q = v / s[:, :, None]
    else:
        v = full.view(mb, BLOCK, kb, BLOCK)
        s = (v.abs().amax((1, 3)) / TOP).clamp_min(TINY)
        q = v / s[:, None, :, None]
    q = q.reshape(-1, kb * BLOCK)[:m, :k].clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return q, s.t().contiguous()


def _wide(q, s):
    """The values that codes and scales stand for, in 32 bits."""
    m, k = q.shape
    s = s.repeat_interleave(BLOCK, 0)[:k]
    s = s if s.shape[1] == m else s.repeat_interleave(BLOCK, 1)[:, :m]
    return q.float() * s.t()


def _plain_matmul(case, st):
    c = torch.matmul(_wide(st["a"], st["sa"]), _wide(st["b"], st["sb"]).t())
    return c.to(DTYPES[case["out"]])


def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_gated(case, st):
    if case["dtype"] == "e4m3":
        x, wg, wu = (_wide(st["x"], st["sx"]), _wide(st["wg"], st["sg"]),
                     _wide(st["wu"], st["su"]))
        dt = torch.bfloat16
    else:
        x, wg, wu, dt = st["x"].float(), st["wg"].float(), st["wu"].float(), st["x"].dtype
    a, _ = _act(case["act"], torch.matmul(x, wg.t()))
    return (a * torch.matmul(x, wu.t())).to(dt)


def _plain_backward(case, st):
    x, wg, wu, dh = (st[n].float() for n in ("x", "wg", "wu", "grad"))
    a, d = _act(case["act"], torch.matmul(x, wg.t()))
    du = dh * a
    dg = dh * torch.matmul(x, wu.t()) * d
    dx = torch.matmul(dg, wg) + torch.matmul(du, wu)
    dt = st["x"].dtype
    return dx.to(dt), torch.matmul(dg.t(), x).to(dt), torch.matmul(du.t(), x).to(dt)


# ---- the definition, in 64 bits -------------------------------------------

def exact(case, seed):
    t = {n: v.double() for n, v in _inputs(case, seed).items()}
    op, m, k = case["op"], case["m"], case["k"]
    kb = _ceil(k, BLOCK)
    if op == "rotate_quantize":
        x = t["x"].t().contiguous() if case["transpose"] else t["x"]
        for b in range(case["bits"]):          # butterflies of stride 2^b
            x = x.reshape(-1, 2, 1 << b)
            x = torch.stack([x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]], 1)
        x = x.reshape(m, k) * 2.0 ** (-case["bits"] / 2)
        s = torch.stack([x[:, i * BLOCK:(i + 1) * BLOCK].abs().amax(1) for i in range(kb)])
        if case["scales"] == "tile":
            s = torch.stack([s[:, i:i + BLOCK].amax(1) for i in range(0, m, BLOCK)], 1)
        s = (s / TOP).clamp_min(TINY)
        by = s if case["scales"] == "row" else s.repeat_interleave(BLOCK, 1)[:, :m]
        for i in range(kb):
            x[:, i * BLOCK:(i + 1) * BLOCK] /= by[i][:, None]
        # e4m3: three bits after the leading one, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
        return (torch.round(x / step) * step).clamp(-TOP, TOP), s

    def operand(q, s):
        at = torch.arange(q.shape[1], device="cuda") // BLOCK
        row = torch.arange(q.shape[0], device="cuda")
        row = row if s.shape[1] == q.shape[0] else row // BLOCK
        return q * s[at][:, row].t()

    def product(a, b):                          # a b^T, rows of a at a time
        return torch.cat([a[i:i + 2048] @ b.t() for i in range(0, a.shape[0], 2048)])

    if op == "scaled_matmul":
        return product(operand(t["a"], t["sa"]), operand(t["b"], t["sb"]))
    if case["dtype"] == "e4m3":
        x, wg, wu = operand(t["x"], t["sx"]), operand(t["wg"], t["sg"]), operand(t["wu"], t["su"])
    else:
        x, wg, wu = t["x"], t["wg"], t["wu"]
    g, u = product(x, wg), product(x, wu)
    if case["act"] == "silu":
        p = torch.sigmoid(g)
        slope = p + g * p * (1 - p)
    else:
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        slope = p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if op == "gated_ffn":
        return g * p * u
    dg, du = t["grad"] * u * slope, t["grad"] * g * p
    return (dg @ wg + du @ wu, product(dg.t().contiguous(), x.t().contiguous()),
            product(du.t().contiguous(), x.t().contiguous()))
