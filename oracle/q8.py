"""CPU oracle of the 8-bit linear layer (double precision, numpy).

TEST INFRASTRUCTURE ONLY, as the rest of this package: the definitions written
out in IEEE double with no blocking, sharing no code with the CUDA library.

  * RMSNorm: h = x + residual rounded once to the rows' type,
    v = h / sqrt(mean(h^2) + eps) * gamma.
  * Its gradients: r = 1 / sqrt(mean(h^2) + eps), s = mean(dy gamma h),
    dx = r dy gamma - r^3 s h (+ dres), dgamma = sum over rows of dy h r.
  * Rows to 8 bits: scale = max(max |v|, 2^-100) / Q, codes v / scale before
    and after rounding (Q = 127 / 448).
  * The product: act((A B^T) * a_scale * b_scale + bias).

Pinned by ``tests/test_q8_oracle.py``.
"""
from __future__ import annotations

import numpy as np

QMAX = {"i8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 patterns (sign, 4 exponent bits with
    bias 7, 3 fraction bits; 0x7f and 0xff are NaN)."""
    b = np.arange(256)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


_POS = e4m3_values()[:127]      # 0 .. 448, ascending


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to the even pattern, saturating at 448."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 448.0)
    hi = np.searchsorted(_POS, a)           # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.copysign(np.where(up, _POS[hi], _POS[lo]), v)


def rmsnorm(h: np.ndarray, gamma=None, eps: float = 1e-6) -> np.ndarray:
    """v of each row of h (double in, double out).  A row that is not finite
    is NaN throughout."""
    h = np.asarray(h, np.float64)
    r = rstd(h, eps)
    return h * r if gamma is None else h * r * np.asarray(gamma, np.float64)


def rstd(h: np.ndarray, eps: float) -> np.ndarray:
    with np.errstate(all="ignore"):
        ms = np.mean(h * h, axis=-1, keepdims=True)
        return np.where(np.isfinite(ms), 1.0 / np.sqrt(ms + eps), np.nan)


def rmsnorm_backward(dy, h, gamma=None, eps: float = 1e-6, dres=None):
    """(dx, dgamma), double."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    r = rstd(h, eps)
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    s = np.mean(g * h, axis=-1, keepdims=True)
    dx = r * g - r ** 3 * s * h
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, np.sum(dy * h * r, axis=0)


def quantize(v: np.ndarray, kind: str):
    """(t, scale) of each row: t = v / scale before rounding.  A row that is
    not finite has the scale NaN and t = 0."""
    v = np.asarray(v, np.float64)
    ok = np.isfinite(v).all(axis=-1)
    amax = np.max(np.abs(np.where(ok[:, None], v, 0.0)), axis=-1)
    scale = np.maximum(amax, TINY) / QMAX[kind]
    t = np.where(ok[:, None], v, 0.0) / scale[:, None]
    return t, np.where(ok, scale, np.nan)


def round_codes(t: np.ndarray, kind: str) -> np.ndarray:
    return np.clip(np.rint(t), -127, 127) if kind == "i8" else round_e4m3(t)


def matmul(a, b, sa, sb, bias=None):
    """(A B^T) * sa * sb + bias in double (the int8 sums are exact in it), and
    the sum of magnitudes sum |a b| sa sb + |bias| that error bounds use."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    s = np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64)[None, :]
    c, mag = (a @ b.T) * s, (np.abs(a) @ np.abs(b).T) * np.abs(s)
    if bias is not None:
        bias = np.asarray(bias, np.float64)
        c, mag = c + bias, mag + np.abs(bias)
    return c, mag
