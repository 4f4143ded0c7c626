"""Rows to 8 bits through GELU where its values are small: the scale follows
the row, so that the values' errors count relative to the row's largest.

Relative error of GELU of a negative value in fp32, u = 2^-24, as far down as
2^-126: the tanh form x / (1 + 2^a) carries the roundings of a (4 u of up to
126, times ln 2: 350 u), the exponential's, sum's, reciprocal's and products'
(10 u).  The exact form carries those of w^2 - P(t) (7 u of up to 87 for the
exponent, through base 2), the fitted P (1.1e-7: 2 u) and 10 u of the rest:
621 u.  2^-14 = 1024 u is above both."""
import numpy as np
import pytest

from _q8util import U, gelu64, guard, guard_empty, half_step, make_rows, to_np
from oracle import q8

pytestmark = pytest.mark.gpu

REL = 2.0 ** -14


@pytest.fixture(scope="module")
def torch_mod(cuda_device):
    import torch
    return torch


def run(fk, torch, x, kind, gelu, xoff=0):
    gx = guard(torch, x, xoff)
    gq = guard_empty(torch, x.shape, torch.int8 if kind == "i8" else torch.float8_e4m3fn)
    gs = guard_empty(torch, x.shape[:1], torch.float32)
    st = fk.fk_quantize_rows(gx.t.data_ptr(), gq.t.data_ptr(), gs.t.data_ptr(), x.shape[0], x.shape[1],
                             fk.FK_F32 if x.dtype == torch.float32 else fk.FK_BF16,
                             fk.FK_I8 if kind == "i8" else fk.FK_E4M3, {"tanh": 1, "erf": 2}[gelu],
                             torch.cuda.current_stream().cuda_stream)
    assert st == fk.FK_OK, fk.fk_status_string(st)
    torch.cuda.synchronize()
    assert gx.canaries_intact() and gq.canaries_intact() and gs.canaries_intact()
    return to_np(gq.t), to_np(gs.t)


def check(x, kind, gelu, got):
    """Scales within REL and the two roundings of max / Q; codes within half
    a step of v / scale, widened by REL for the value, REL for the scale and
    the roundings."""
    codes, scales = got
    t, s = q8.quantize(gelu64(to_np(x), gelu), kind)
    nan = np.isnan(s)
    assert np.array_equal(np.isnan(scales), nan) and np.all(codes[nan] == 0)
    codes, scales, t, s = codes[~nan], scales[~nan], t[~nan], s[~nan]
    assert np.all(np.abs(scales - s) <= s * (REL + 2 * U))
    wide = np.abs(t) * (2 * REL + 4 * U)
    bound = np.maximum(half_step(np.abs(t) + wide, kind), half_step(t, kind)) + wide
    bad = np.abs(codes - t) > bound
    assert not bad.any(), f"{bad.sum()} codes off, rows {np.unique(np.nonzero(bad)[0])}"


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,off", [(40, 0), (64, 0), (255, 0), (1000, 0), (2049, 0), (4096, 0), (9000, 0), (16384, 0),
                                      (16384, 1), (20000, 0), (20001, 0), (40000, 0), (140000, 0)])
def test_rows_far_below_zero(fk, torch_mod, cols, off, dtype, gelu):
    torch = torch_mod
    g = np.random.default_rng(cols)
    x = torch.empty(12, cols)
    for i, (lo, hi) in enumerate([(-5, -4), (-6.5, -6), (-8, -6), (-9.5, -9), (-9.95, -9.7), (-11, -9.5), (-13, -9),
                                  (-16, -12), (-40, -9.9)]):
        x[i] = torch.from_numpy(g.uniform(lo, hi, cols).astype(np.float32))
    x[9] = -11.0
    x[9, cols // 2] = -9.5                       # -11 is nothing beside it
    x[10] = -20.0                                # GELU is below every code: the smallest scale, codes 0
    x[11] = -float("inf")
    x = x.to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    for kind in ("i8", "e4m3"):
        c, s = got = run(fk, torch, x, kind, gelu, off)
        check(x, kind, gelu, got)
        assert np.all(c[10:] == 0) and np.all(s[10:] == np.float32(2.0 ** -100) * (np.float32(1) / np.float32(q8.QMAX[kind])))


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("rows,cols", [(700, 8200), (1000, 8704), (640, 12000), (450, 16384), (2000, 16376)])
def test_wide_rows_of_both_kinds_in_turn(fk, torch_mod, rows, cols, kind, gelu):
    """More rows than blocks stay resident, so that each block walks several:
    rows whose scale their largest value decides, rows of small or negative
    values only, NaN, zeros and far values follow each other in every order."""
    torch = torch_mod
    g = np.random.default_rng(rows)
    x = make_rows(rows, cols, "f32", cols)
    sort = g.integers(0, 8, rows)
    for i in np.nonzero(sort == 1)[0]:
        x[i] *= 0.01                                       # all below the dip
    for i in np.nonzero(sort == 2)[0]:
        x[i] = -x[i].abs() - 0.01                          # all negative
    for i in np.nonzero(sort == 3)[0]:
        x[i, int(g.integers(cols))] = float("nan")
    for i in np.nonzero(sort == 4)[0]:
        x[i] = x[i].clamp(-3.0, 0.2)
        x[i, int(g.integers(cols))] = -0.75                # the dip, in one place
    for i in np.nonzero(sort == 5)[0]:
        x[i] = 0.0 if i % 3 else -25.0
    for i in np.nonzero(sort == 6)[0]:
        x[i, int(g.integers(cols))] = 1.0e30 if i % 2 else float("inf")
    x = x.bfloat16()
    check_rows = np.unique(np.concatenate([g.integers(0, rows, 60), [0, 1, rows - 2, rows - 1]]))
    c, s = run(fk, torch, x, kind, gelu)
    check(x[check_rows], kind, gelu, (c[check_rows], s[check_rows]))
    # a row's codes do not depend on its place: every row again, in reverse
    c2, s2 = run(fk, torch, x.flip(0).contiguous(), kind, gelu)
    assert np.array_equal(c, c2[::-1]) and np.array_equal(s, s2[::-1], equal_nan=True)


@pytest.mark.parametrize("gelu", [None, "tanh", "erf"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_wide_rows_one_by_one_and_together(fk, torch_mod, kind, gelu):
    """Rows of a long matrix get the codes that each gets alone."""
    torch = torch_mod
    x = make_rows(1500, 9216, "bf16", 4).cuda()
    x[::7] *= 0.02
    dt = torch.int8 if kind == "i8" else torch.float8_e4m3fn
    q, s = fk.quantize_rows(x, dt, gelu=gelu)
    for i in list(range(0, 1500, 97)) + [295, 296, 297, 443, 444, 445, 1499]:
        q1, s1 = fk.quantize_rows(x[i:i + 1].contiguous(), dt, gelu=gelu)
        assert torch.equal(q[i].view(torch.uint8), q1[0].view(torch.uint8)) and torch.equal(s[i], s1[0])
