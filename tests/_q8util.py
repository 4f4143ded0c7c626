"""Test-side helpers of the 8-bit linear layer: inputs, guarded device
buffers, and the error bounds every kernel is held to.

Notation: u = 2^-24 is the largest relative error of one fp32 rounding.  A
sum of positive terms that no accumulator adds more than `chain` of in a row
is off by at most chain * u relative; rsqrt is within 2 ulp (4 u); a product
or a division adds u each.
"""
from __future__ import annotations

import numpy as np

import oracle
from _util import Guarded
from oracle import q8

U = 2.0 ** -24
EPS_HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}     # largest relative error of the output's rounding
DENORMAL = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126}  # results below this may be flushed


def chain(cols: int) -> float:
    """Longest run of additions in a row sum: a thread's own values (at most
    32 where the row sits in registers, cols / 512 where it is streamed),
    then 5 steps across a warp and at most 32 across a block."""
    return max(32, -(-cols // 512)) + 37


def rel_v(cols: int) -> float:
    """Relative error of v = h rstd gamma in fp32: half that of the sum of
    squares (whose terms are rounded too), the mean and eps (2 u), rsqrt
    (4 u), two products."""
    return (0.5 * (chain(cols) + 3) + 6) * U


def to_np(t):
    """Values of a torch tensor as float64 (8-bit floats included)."""
    import torch
    return t.detach().cpu().to(torch.float64).numpy()


def make_rows(rows, cols, dtype, seed, spread=1.0):
    """Rows of differing size with a few large channels, exactly
    representable in `dtype`, as a CPU torch tensor."""
    import torch
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * np.exp(spread * g.standard_normal((rows, 1)))
    x[:, g.integers(0, cols, max(1, cols // 200))] *= 12.0
    return torch.from_numpy(x.astype(np.float32)).to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])


def guard(torch, t, offset=0):
    """A guarded device copy of a CPU tensor (`.t`: the payload in its shape)."""
    raw = t.view(torch.uint8) if t.element_size() == 1 else t
    g = Guarded(torch, raw.numel(), raw.dtype, torch.device("cuda:0"), offset=offset, fill=raw.reshape(-1))
    g.t = g.view.view(t.dtype).reshape(t.shape)
    return g


def guard_empty(torch, shape, dtype, offset=0):
    """A guarded device buffer whose payload starts as the canary."""
    n = int(np.prod(shape))
    raw = torch.uint8 if dtype in (torch.int8, torch.float8_e4m3fn) else dtype
    g = Guarded(torch, n, raw, torch.device("cuda:0"), offset=offset)
    g.t = g.view.view(dtype).reshape(shape)
    return g


def check_values(got, ref, rel, dtype, what="values", extra=0.0):
    """|got - ref| <= |ref| (rel + output rounding) + extra, NaN where ref is."""
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    err = np.abs(got - ref)[~nan]
    bound = (np.abs(ref) * ((1 + rel) * EPS_HALF[dtype] + rel) + DENORMAL[dtype] + extra)[~nan]
    assert err.size == 0 or np.max(err / bound) <= 1.0, f"{what}: {np.max(err / bound):.2f} x the bound"


def half_step(t, kind):
    """Half the distance between the codes around t."""
    if kind == "i8":
        return 0.5
    e = np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def check_codes(codes, scales, v, rel, kind):
    """Codes and scales of rows whose fp32 values are within `rel` of v: the
    scale within rel + 2 u; a code within half a step of v / scale, widened
    by the relative errors of v, of the scale and of two products."""
    t, s = q8.quantize(v, kind)
    nan = np.isnan(s)
    assert np.array_equal(np.isnan(scales), nan), "scale NaN in other places"
    assert np.all(codes[nan] == 0)
    assert np.all(np.abs(scales - s)[~nan] <= s[~nan] * (rel + 2 * U)), "scales"
    c, t = codes[~nan], t[~nan]
    assert np.all(np.abs(c) <= q8.QMAX[kind])
    # the step that counts is the one at the (slightly moved) value
    wide = np.abs(t) * (2 * rel + 4 * U)
    bound = np.maximum(half_step(np.abs(t) + wide, kind), half_step(t, kind)) + wide
    bad = np.abs(c - t) > bound
    assert not bad.any(), f"{bad.sum()} codes further than half a step from v / scale"


def gelu64(v, kind):
    if kind is None:
        return v
    f = oracle.gelu_tanh_f64 if kind == "tanh" else oracle.gelu_erf_f64
    nan = np.isnan(v)
    return np.where(nan, np.nan, f(np.where(nan, 0.0, v)))


GELU_ABS = 2e-6     # fk_gelu's fp32 bound, absolute
GELU_SLOPE = 1.13   # largest |GELU'|, either form
