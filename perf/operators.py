"""The 8-bit linear layer measured: RMSNorm with the residual's addition
(forward, to 8 bits or not, and backward), rows to 8 bits with or without a
GELU, the 8-bit matrix product with its scales, and the norm followed by the
product.  Cases, inputs, one pass of each operator, and the work of a pass.

`own` false computes the operators in elementary torch operations in 32 bits;
`own` true calls memory_bound_fk_b200.
"""
import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -100          # rows whose largest magnitude is below this take it for their scale
QMAX = {"i8": 127.0, "e4m3": 448.0}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "i8": 1, "e4m3": 1}


def listed():
    return [
        # one token of a decode step: the norm before a linear layer, to 8 bits
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "out": "e4m3", "residual": True},
        # a decode batch, the norm left in bf16
        {"name": "norm_decode_batch", "op": "norm", "rows": 48, "cols": 8192, "dtype": "bf16", "out": "bf16", "residual": True},
        # a long prompt
        {"name": "norm_prompt", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "out": "e4m3", "residual": True},
        # odd width in fp32, no residual (a final norm, a small model)
        {"name": "norm_odd_f32", "op": "norm", "rows": 4099, "cols": 1001, "dtype": "f32", "out": "f32", "residual": False},
        # a training step's backward pass, with the gradient of the residual stream
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True},
        # the same, ragged and small, in fp32
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "rows": 1001, "cols": 2047, "dtype": "f32", "residual": False},
        # between the two products of an MLP: GELU, then 8 bits
        {"name": "gelu_to_8_bits", "op": "quant", "rows": 8192, "cols": 16384, "dtype": "bf16", "out": "e4m3", "gelu": "tanh"},
        # a weight matrix brought to 8 bits, odd sizes
        {"name": "weights_to_8_bits", "op": "quant", "rows": 5003, "cols": 2049, "dtype": "f32", "out": "e4m3", "gelu": "none"},
        # the product of one token: the weights are read once
        {"name": "mm_one_token", "op": "mm", "m": 1, "n": 16384, "k": 4096, "q": "i8", "out": "bf16", "gelu": "none", "bias": True},
        # a decode batch over an odd vocabulary, logits in fp32
        {"name": "mm_vocabulary", "op": "mm", "m": 48, "n": 32001, "k": 4096, "q": "e4m3", "out": "f32", "gelu": "none", "bias": False},
        # a long prompt through the MLP's first product and its GELU
        {"name": "mm_prompt", "op": "mm", "m": 8192, "n": 16384, "k": 4096, "q": "i8", "out": "bf16", "gelu": "tanh", "bias": True},
        # the norm to int8 and the product that reads it, a short prompt
        {"name": "norm_mm_short_prompt", "op": "norm_mm", "m": 509, "n": 4096, "k": 4096, "q": "i8", "out": "bf16", "gelu": "none", "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "quant", "mm", "mm", "mm", "norm_mm"])
    if op in ("norm", "norm_bwd", "quant"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = max(64, cols // 64 * 64)
        rows = _log(rng, 1, min(16384, 16384 * 4096 // cols))
        c = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "quant":
            return {**c, "out": "e4m3", "gelu": rng.choice(["none", "tanh", "erf"])}
        c["residual"] = rng.random() < 0.6
        if op == "norm":
            c["out"] = rng.choice(["e4m3", c["dtype"]])
        return c
    k = _log(rng, 256, 16384)
    k = max(16, k // 16 * 16) if rng.random() < 0.85 else k
    n = _log(rng, 256, 32768)
    n = n // 64 * 64 if rng.random() < 0.7 else n
    m = _log(rng, 1, min(8192, 8192 * 16384 * 4096 // (n * k)))
    return {"op": op, "m": m, "n": n, "k": k, "q": "i8" if op == "norm_mm" else rng.choice(["i8", "e4m3"]),
            # after the norm the product is left in bf16: a code next to a rounding border may be either of two
            "out": "bf16" if op == "norm_mm" else rng.choice(["bf16", "bf16", "f32"]),
            "gelu": rng.choice(["none", "none", "tanh", "erf"]),
            "bias": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _hidden(g, rows, cols, dtype):
    """Hidden states: a spread per row, and a few channels far larger than the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    channel = torch.ones(cols, device="cuda")
    channel[torch.randint(0, cols, (max(1, cols // 256),), generator=g, device="cuda")] = 12.0
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= channel
    return x.to(TORCH[dtype])


def _codes(g, rows, cols, q):
    """Codes of normal values scaled so that the largest of a row is near the type's largest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    s = QMAX[q] / 4.0
    x = (x * s).clamp_(-QMAX[q], QMAX[q])
    return (x.round_() if q == "i8" else x).to(TORCH[q])


def _scales(g, count, q, typical):
    return typical * 4.0 / QMAX[q] * torch.exp(0.3 * torch.randn(count, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op in ("norm", "norm_mm"):
        rows, cols = (case["rows"], case["cols"]) if op == "norm" else (case["m"], case["k"])
        dtype = case["dtype"] if op == "norm" else "bf16"
        s["x"] = _hidden(g, rows, cols, dtype)
        s["residual"] = _hidden(g, rows, cols, dtype) if op == "norm_mm" or case["residual"] else None
        s["weight"] = 1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    elif op == "norm_bwd":
        s["h"] = _hidden(g, case["rows"], case["cols"], case["dtype"])
        s["dy"] = torch.randn(case["rows"], case["cols"], generator=g, device="cuda").to(TORCH[case["dtype"]])
        s["dres"] = (torch.randn(case["rows"], case["cols"], generator=g, device="cuda").to(TORCH[case["dtype"]])
                     if case["residual"] else None)
        s["weight"] = 1.0 + 0.1 * torch.randn(case["cols"], generator=g, device="cuda")
    elif op == "quant":
        s["x"] = _hidden(g, case["rows"], case["cols"], case["dtype"])
    if op in ("mm", "norm_mm"):
        m, n, k, q = case["m"], case["n"], case["k"], case["q"]
        if op == "mm":
            s["a"] = _codes(g, m, k, q)
            s["sa"] = _scales(g, m, q, 1.0)
        s["b"] = _codes(g, n, k, q)
        s["sb"] = _scales(g, n, q, 1.0 / math.sqrt(k))
        s["bias"] = 0.1 * torch.randn(n, generator=g, device="cuda") if case["bias"] else None
    return s


# ---------------------------------------------------------------- the plain forms

def _gelu(v, kind):
    if kind == "tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if kind == "erf":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _to_8_bits(v, q):
    scale = v.abs().amax(dim=-1, keepdim=True).clamp(min=TINY) / QMAX[q]
    t = (v / scale).clamp(-QMAX[q], QMAX[q])
    return (t.round() if q == "i8" else t).to(TORCH[q]), scale.squeeze(-1)


def _norm_plain(x, residual, weight):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = h.float()
    return f * torch.rsqrt(f.square().mean(dim=-1, keepdim=True) + EPS) * weight, h


def _mm_plain(a, sa, b, sb, bias, kind, out):
    c = (a.float() @ b.float().t()) * sa[:, None] * sb
    return _gelu(c if bias is None else c + bias, kind).to(TORCH[out])


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        v, h = _norm_plain(s["x"], s["residual"], s["weight"])
        got = list(_to_8_bits(v, s["out"])) if s["out"] in QMAX else [v.to(TORCH[s["out"]])]
        return got + ([h] if s["residual"] is not None else [])
    if op == "norm_bwd":
        dy, h, w = s["dy"].float(), s["h"].float(), s["weight"]
        rstd = torch.rsqrt(h.square().mean(dim=-1, keepdim=True) + EPS)
        normed = h * rstd
        g = dy * w
        dx = rstd * (g - normed * (g * normed).mean(dim=-1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return [dx.to(s["h"].dtype), (dy * normed).sum(dim=0)]
    if op == "quant":
        return list(_to_8_bits(_gelu(s["x"].float(), s["gelu"]), s["out"]))
    if op == "mm":
        return _mm_plain(s["a"], s["sa"], s["b"], s["sb"], s["bias"], s["gelu"], s["out"])
    v, h = _norm_plain(s["x"], s["residual"], s["weight"])
    a, sa = _to_8_bits(v, s["q"])
    return [_mm_plain(a, sa, s["b"], s["sb"], s["bias"], s["gelu"], s["out"]), h]


# ---------------------------------------------------------------- the framework's operators

_GELU = {"none": None, "tanh": "tanh", "erf": "erf"}


def _run_own(s):
    import memory_bound_fk_b200 as fk
    op = s["op"]
    if op == "norm":
        got = fk.rmsnorm(s["x"], s["weight"], eps=EPS, residual=s["residual"], out_dtype=TORCH[s["out"]])
        return list(got) if isinstance(got, tuple) else [got]
    if op == "norm_bwd":
        return list(fk.rmsnorm_backward(s["dy"], s["h"], s["weight"], eps=EPS, dresidual=s["dres"]))
    if op == "quant":
        return list(fk.quantize_rows(s["x"], dtype=TORCH[s["out"]], gelu=_GELU[s["gelu"]]))
    if op == "mm":
        return fk.matmul_q8(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], gelu=_GELU[s["gelu"]],
                            out_dtype=TORCH[s["out"]])
    a, sa, h = fk.rmsnorm(s["x"], s["weight"], eps=EPS, residual=s["residual"], out_dtype=TORCH[s["q"]])
    return [fk.matmul_q8(a, sa, s["b"], s["sb"], bias=s["bias"], gelu=_GELU[s["gelu"]], out_dtype=TORCH[s["out"]]), h]


def run(state):
    if own:
        return _run_own(state)
    else:
        return _run_plain(state)


# ---------------------------------------------------------------- work

def _norm_work(rows, cols, size, out, residual):
    n = rows * cols
    bytes_ = n * size * (3 if residual else 1) + n * SIZE[out] + 4 * cols
    return bytes_ + (4 * rows if out in QMAX else 0), 8.0 * n


def _mm_work(m, n, k, out, bias):
    return m * k + n * k + m * n * SIZE[out] + 4 * (m + n) + (4 * n if bias else 0), 2.0 * m * n * k


def work(case):
    op = case["op"]
    if op == "norm":
        b, f = _norm_work(case["rows"], case["cols"], SIZE[case["dtype"]], case["out"], case["residual"])
    elif op == "norm_bwd":
        n = case["rows"] * case["cols"]
        b, f = n * SIZE[case["dtype"]] * (4 if case["residual"] else 3) + 8 * case["cols"], 14.0 * n
    elif op == "quant":
        n = case["rows"] * case["cols"]
        b, f = n * SIZE[case["dtype"]] + n + 4 * case["rows"], 4.0 * n + (12.0 * n if case["gelu"] != "none" else 0.0)
    elif op == "mm":
        b, f = _mm_work(case["m"], case["n"], case["k"], case["out"], case["bias"])
    else:
        # the 8-bit rows between the two operators are written and read
        nb, nf = _norm_work(case["m"], case["k"], 2, case["q"], True)
        b, f = _mm_work(case["m"], case["n"], case["k"], case["out"], case["bias"])
        b, f = b + nb, f + nf
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- 64 bits

def _gelu_64(v, kind):
    if kind == "tanh":  # x sigma(2u)
        return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if kind == "erf":   # x Phi(x), the tail kept exact
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
    return v


def _scale_64(v, q):
    return torch.maximum(v.abs().max(dim=-1).values, torch.tensor(TINY, dtype=v.dtype, device=v.device)) / QMAX[q]


def _norm_64(x, residual, weight):
    h = x.double() if residual is None else (x.double() + residual.double()).to(x.dtype).double()
    v = h * weight.double() / torch.sqrt((h * h).sum(dim=-1, keepdim=True) / h.shape[-1] + EPS)
    return v, h


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v, h = _norm_64(s["x"], s["residual"], s["weight"])
        if case["out"] in QMAX:
            scale = _scale_64(v, case["out"])
            got = [v / scale[:, None], scale]  # codes before their rounding
        else:
            got = [v]
        return got + ([h] if s["residual"] is not None else [])
    if op == "norm_bwd":
        dy, h, w = s["dy"].double(), s["h"].double(), s["weight"].double()
        r2 = 1.0 / ((h * h).sum(dim=-1, keepdim=True) / h.shape[-1] + EPS)
        r = torch.sqrt(r2)
        dot = (dy * w * h).sum(dim=-1, keepdim=True) / h.shape[-1]
        dx = r * dy * w - h * (r * r2 * dot)
        if s["dres"] is not None:
            dx = dx + s["dres"].double()
        return [dx, (dy * h * r).sum(dim=0)]
    if op == "quant":
        v = _gelu_64(s["x"].double(), case["gelu"])
        scale = _scale_64(v, case["out"])
        return [v / scale[:, None], scale]
    tail = []
    if op == "mm":
        a, sa = s["a"].double(), s["sa"].double()
    else:
        v, h = _norm_64(s["x"], s["residual"], s["weight"])
        sa = _scale_64(v, case["q"])
        a = torch.round(v / sa[:, None]).clamp(-QMAX[case["q"]], QMAX[case["q"]])
        tail = [h]
    c = torch.einsum("mk,nk->mn", a, s["b"].double())
    c = c * (sa[:, None] * s["sb"].double()[None, :])
    if s["bias"] is not None:
        c = c + s["bias"].double()
    c = _gelu_64(c, case["gelu"])
    return [c] + tail if tail else c
