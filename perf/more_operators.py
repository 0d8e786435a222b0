"""Cases of the 8-bit integer products and of the products grouped by expert,
for timing and for comparing the library's kernels with a plain form.

Four operators, used together in the feed-forward block of a model with
experts:

* ``rotate_quantize_int8``: x times I (x) H_b along the contraction axis (H_b
  the normalised Walsh-Hadamard matrix of 2^b), then 8-bit integers with one
  fp32 scale for each row (a token of activations, a channel of weights);
* ``int8_matmul``: a b^T of two such operands, exact sums, times the scale of
  the token and of the channel;
* ``grouped_matmul``: rows sorted by expert, each times its expert's weights,
  in 16 bits or in 8-bit integers; where the groups end is known on the GPU;
* ``grouped_matmul_backward``: its gradients for the rows and for the weights.

``run`` computes the plain form in 32 bits with elementary torch operations,
or, with ``own`` set, calls the library.
"""
import math

import numpy as np
import torch

own = False

TOP = 127.0      # largest code
TINY = 2.0 ** -126

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token's activations before an 8-bit projection: latency
        dict(name="quantize_token", op="rotate_quantize_int8", m=1, k=4096, bits=12,
             dtype="bf16"),
        # the hidden activations of a long prompt, rotated over the whole row
        dict(name="quantize_prompt", op="rotate_quantize_int8", m=8192, k=16384, bits=14,
             dtype="bf16"),
        # a weight matrix of no round size prepared for serving
        dict(name="quantize_weight", op="rotate_quantize_int8", m=4100, k=5000, bits=3,
             dtype="f32"),
        # one token through an 8-bit projection: the weights' bytes
        dict(name="int8_token", op="int8_matmul", m=1, n=16384, k=4096, out="bf16"),
        # a short ragged prompt
        dict(name="int8_ragged", op="int8_matmul", m=333, n=4100, k=2056, out="f16"),
        # a long prompt through a down projection
        dict(name="int8_prompt", op="int8_matmul", m=8192, n=4096, k=16384, out="bf16"),
        # sixteen sequences' next tokens, two experts each of 64: the bytes of
        # the experts that they reach
        dict(name="grouped_decode", op="grouped_matmul", m=32, e=64, n=2048, k=4096, rest=0,
             dtype="bf16", out="bf16"),
        # sizes that are multiples of nothing, in a buffer that is not full
        dict(name="grouped_odd", op="grouped_matmul", m=1021, e=7, n=1501, k=2047, rest=100,
             dtype="f16", out="f16"),
        # a long prompt through 16-bit experts
        dict(name="grouped_prompt", op="grouped_matmul", m=16384, e=8, n=8192, k=4096, rest=0,
             dtype="bf16", out="bf16"),
        # the same through 8-bit experts, many of them
        dict(name="grouped_int8", op="grouped_matmul", m=16384, e=32, n=4096, k=4096, rest=0,
             dtype="int8", out="bf16"),
        # a training step's gradients
        dict(name="grouped_grad", op="grouped_matmul_backward", m=16384, e=16, n=4096, k=4096,
             rest=0, dtype="bf16"),
        # few tokens for many narrow experts, some of which get none
        dict(name="grouped_grad_ragged", op="grouped_matmul_backward", m=3001, e=60, n=1408,
             k=2050, rest=57, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the logarithm of their ranges, half of the
    widths odd or ragged, half of the grouped buffers not full."""
    op = rng.choice(["rotate_quantize_int8", "int8_matmul", "grouped_matmul",
                     "grouped_matmul_backward"])
    while True:
        if op == "rotate_quantize_int8":
            bits = rng.randint(0, 14)
            m, k = _log(rng, 1, 8192), _log(rng, 64, 16384)
            k = max(1, k >> bits) << bits
            return dict(op=op, m=m, k=k, bits=bits, dtype=rng.choice(["bf16", "f16", "f32"]))
        n, k = _log(rng, 64, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.5:
            n, k = max(16, n // 16 * 16), max(16, k // 16 * 16)
        if op == "int8_matmul":
            c = dict(op=op, m=_log(rng, 1, 8192), n=n, k=k, out=rng.choice(["bf16", "f16", "f32"]))
            if work(c)["flops"] <= 2 * 8192 * 4096 * 16384:
                return c
            continue
        m, e = _log(rng, 1, 16384), _log(rng, 1, 128)
        rest = rng.randint(0, m // 4) if rng.random() < 0.5 else 0
        c = dict(op=op, m=m, e=e, n=n, k=k, rest=rest)
        if op == "grouped_matmul":
            c["dtype"] = rng.choice(["bf16", "f16", "int8"])
            c["out"] = rng.choice(["bf16", "f16", "f32"]) if c["dtype"] == "int8" else c["dtype"]
        else:
            c["dtype"] = rng.choice(["bf16", "f16"])
        if work(c)["flops"] <= 2 * 16384 * 8192 * 4096 and e * n * k <= 32 * 4096 * 4096:
            return c


def _popularity(e):
    """How often each expert is chosen: unevenly, as routers do."""
    p = np.arange(1, e + 1) ** -0.5
    return p / p.sum()


def work(case):
    """Each input read once, each output written once (of the experts those
    that are expected to be reached); the products' operations, and one
    addition for each element and rotation stage."""
    m, k = case["m"], case["k"]
    if case["op"] == "rotate_quantize_int8":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": m * k * (size + 1) + 4 * m, "flops": m * k * (case["bits"] + 2)}
    n = case["n"]
    out = {"f32": 4, "bf16": 2, "f16": 2}[case.get("out", "bf16")]
    if case["op"] == "int8_matmul":
        return {"bytes": (m + n) * k + 4 * (m + n) + m * n * out, "flops": 2 * m * n * k}
    used = m - case["rest"]
    reached = float((1.0 - (1.0 - _popularity(case["e"])) ** used).sum())
    size = 1 if case["dtype"] == "int8" else 2
    if case["op"] == "grouped_matmul":
        scales = 4 * (used + reached * n) if size == 1 else 0
        return {"bytes": size * (used * k + reached * n * k) + m * n * out + scales,
                "flops": 2 * used * n * k}
    return {"bytes": 2 * (used * (n + k) + reached * n * k + m * k + case["e"] * n * k),
            "flops": 4 * used * n * k}


# ---- inputs ---------------------------------------------------------------

def _activations(g, rows, cols, dtype):
    """N(0, 1) with about one channel in 64 thirty times as large, as the
    activations that a rotation is used for have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.rand(cols, generator=g, device="cuda") < 1.0 / 64
    return x.mul_(torch.where(loud, 30.0, 1.0)).to(dtype)


def _weights(g, shape, dtype):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(shape[-1] ** -0.5).to(dtype)


def _codes(x):
    """8-bit integers of x (rows padded to a multiple of 16) and scales."""
    k = x.shape[-1]
    s = (x.abs().amax(-1) / TOP).clamp_min(TINY)
    q = torch.zeros(*x.shape[:-1], -(-k // 16) * 16, dtype=torch.int8, device="cuda")
    q[..., :k] = torch.round(x / s[..., None])
    return q[..., :k], s


def _counts(case, seed):
    rng = np.random.RandomState(seed % (1 << 32))
    p = rng.permutation(_popularity(case["e"]))
    return [int(c) for c in rng.multinomial(case["m"] - case["rest"], p)]


def _hadamard(bits):
    h = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(bits):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h * 2.0 ** (-bits / 2)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "rotate_quantize_int8":
        return {"x": _activations(g, m, k, DTYPES[case["dtype"]])}
    n = case["n"]
    if op == "int8_matmul":
        a, sa = _codes(_activations(g, m, k, torch.float32))
        b, sb = _codes(_weights(g, (n, k), torch.float32))
        return {"a": a, "sa": sa, "b": b, "sb": sb}
    e = case["e"]
    if case["dtype"] == "int8":
        x, sx = _codes(torch.randn(m, k, generator=g, device="cuda"))
        w, sw = _codes(_weights(g, (e, n, k), torch.float32))
        return {"x": x, "sx": sx, "w": w, "sw": sw}
    dt = DTYPES[case["dtype"]]
    t = {"x": torch.randn(m, k, generator=g, device="cuda").to(dt),
         "w": _weights(g, (e, n, k), dt)}
    if op == "grouped_matmul_backward":
        t["grad"] = torch.randn(m, n, generator=g, device="cuda").mul_(0.1).to(dt)
    return t


def prepare(case, seed):
    state = dict(case=dict(case), **_inputs(case, seed))
    if case["op"] == "rotate_quantize_int8":
        b = case["bits"]
        # the two Kronecker factors that the plain form multiplies by
        state["h_low"] = _hadamard(min(b, 7)).float().cuda()
        state["h_high"] = _hadamard(max(b - 7, 0)).float().cuda()
    elif "e" in case:
        state["counts"] = _counts(case, seed)
        state["ends"] = torch.tensor(np.cumsum(state["counts"]), dtype=torch.int32, device="cuda")
    return state


# ---- one pass -------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _library(case, state)
    return {"rotate_quantize_int8": _plain_quantize, "int8_matmul": _plain_int8,
            "grouped_matmul": _plain_grouped,
            "grouped_matmul_backward": _plain_backward}[case["op"]](case, state)


def _values(q, s):
    """What codes and scales stand for."""
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    return torch.mul(q, s[:, None], out=out)


def _library(case, st):
    import quantum_state_encoding_amd as qse
    if case["op"] == "rotate_quantize_int8":
        q, s = qse.rotate_quantize_int8(st["x"], bits=case["bits"])
        return _values(q, s), s
    if case["op"] == "int8_matmul":
        return qse.int8_matmul(st["a"], st["sa"], st["b"], st["sb"],
                               out_dtype=DTYPES[case["out"]])
    if case["op"] == "grouped_matmul":
        if case["dtype"] == "int8":
            return qse.grouped_matmul(st["x"], st["w"], st["ends"], x_scales=st["sx"],
                                      w_scales=st["sw"], out_dtype=DTYPES[case["out"]])
        return qse.grouped_matmul(st["x"], st["w"], st["ends"])
    return qse.grouped_matmul_backward(st["x"], st["w"], st["ends"], st["grad"])


def _plain_quantize(case, st):
    m, k, bits = case["m"], case["k"], case["bits"]
    x = st["x"].float()
    low = min(bits, 7)
    if bits:
        x = torch.matmul(x.reshape(m * (k >> low), 1 << low), st["h_low"])
    if bits > low:
        x = torch.matmul(st["h_high"], x.reshape(m * (k >> bits), 1 << (bits - low), 1 << low))
    x = x.reshape(m, k)
    s = (x.abs().amax(1) / TOP).clamp_min(TINY)
    q = torch.round(x / s[:, None]).clamp(-TOP, TOP).to(torch.int8)
    return _values(q, s), s


def _plain_int8(case, st):
    c = torch.matmul(st["a"].float(), st["b"].float().t())
    return (c * st["sa"][:, None] * st["sb"]).to(DTYPES[case["out"]])


def _plain_grouped(case, st):
    y = torch.zeros(case["m"], case["n"], dtype=DTYPES[case["out"]], device="cuda")
    at = 0
    for e, rows in enumerate(st["counts"]):
        if rows:
            part = slice(at, at + rows)
            c = torch.matmul(st["x"][part].float(), st["w"][e].float().t())
            if case["dtype"] == "int8":
                c = c * st["sx"][part, None] * st["sw"][e]
            y[part] = c
            at += rows
    return y


def _plain_backward(case, st):
    dx, dw = torch.zeros_like(st["x"]), torch.zeros_like(st["w"])
    at = 0
    for e, rows in enumerate(st["counts"]):
        if rows:
            part = slice(at, at + rows)
            grad = st["grad"][part].float()
            dx[part] = torch.matmul(grad, st["w"][e].float())
            dw[e] = torch.matmul(grad.t(), st["x"][part].float())
            at += rows
    return dx, dw


# ---- the definition, in 64 bits -------------------------------------------

def exact(case, seed):
    t = _inputs(case, seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "rotate_quantize_int8":
        x = t["x"].double()
        for b in range(case["bits"]):          # butterflies of stride 2^b
            x = x.reshape(-1, 2, 1 << b)
            x = torch.stack([x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]], 1)
        x = x.reshape(m, k) * 2.0 ** (-case["bits"] / 2)
        s = torch.maximum(x.amax(1), -x.amin(1)) / TOP
        s = torch.where(s < TINY, TINY, s)
        # the nearest whole number of steps, of two the even one
        r = x / s[:, None] + 0.5
        n = torch.floor(r)
        n = n - ((r == n) & (n % 2 != 0)).double()
        return torch.minimum(torch.maximum(n, torch.full_like(n, -TOP)),
                             torch.full_like(n, TOP)) * s[:, None], s
    if op == "int8_matmul":
        a = t["a"].double() * t["sa"].double().view(m, 1)
        b = t["b"].double() * t["sb"].double().view(-1, 1)
        return torch.cat([a[i:i + 2048] @ b.t() for i in range(0, m, 2048)])
    ends = np.cumsum(_counts(case, seed)).tolist()
    groups = list(zip([0] + ends[:-1], ends))

    def weights(e):
        w = t["w"][e].double()
        return w * t["sw"][e].double().view(-1, 1) if "sw" in t else w

    def rows(lo, hi):
        x = t["x"][lo:hi].double()
        return x * t["sx"][lo:hi].double().view(-1, 1) if "sx" in t else x

    behind = m - ends[-1]                       # rows of no expert
    if op == "grouped_matmul":
        parts = [rows(lo, hi) @ weights(e).t() for e, (lo, hi) in enumerate(groups)]
        return torch.cat(parts + [torch.zeros(behind, case["n"], dtype=torch.float64,
                                              device="cuda")])
    grads = [t["grad"][lo:hi].double() for lo, hi in groups]
    dx = torch.cat([gr @ weights(e) for e, gr in enumerate(grads)] +
                   [torch.zeros(behind, k, dtype=torch.float64, device="cuda")])
    dw = torch.stack([gr.t().contiguous() @ rows(lo, hi) for gr, (lo, hi) in zip(grads, groups)])
    return dx, dw
