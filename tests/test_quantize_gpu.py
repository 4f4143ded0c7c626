"""fk_quantize_rows on the GPU against the double-precision oracle; bounds in
_q8util.  Values that go through GELU carry its fp32 error, 2e-6 absolute (or
2^-20 relative where that is more), so codes may sit that much further from
v / scale."""
import numpy as np
import pytest

from _q8util import GELU_ABS, U, gelu64, guard, guard_empty, half_step, make_rows, to_np
from oracle import q8

pytestmark = pytest.mark.gpu

SHAPES = [(37, 1), (3, 7), (65, 64), (33, 1000), (17, 1024), (17, 1025), (9, 2048), (9, 2049), (6, 4096), (3, 11008),
          (3, 16384), (2, 16385), (2, 32768), (2, 32769), (2, 100003), (1, 262144), (1300, 256), (700, 1000), (900, 4096),
          (9, 1), (9, 2), (9, 5), (9, 9), (9, 31), (9, 253), (9, 257), (9, 509), (9, 1017), (9, 1021), (9, 2047), (9, 4091),
          (9, 4093), (9, 8193), (9, 16381), (9, 32761), (9, 32765),
          (5003, 64), (5001, 61), (333, 57), (2999, 128), (2999, 122), (7, 128), (1, 48), (3, 113)]


@pytest.fixture(scope="module")
def torch_mod(cuda_device):
    import torch
    return torch


def run(fk, torch, x, kind, gelu=None, xoff=0, qoff=0):
    gx = guard(torch, x, xoff)
    gq = guard_empty(torch, x.shape, torch.int8 if kind == "i8" else torch.float8_e4m3fn, qoff)
    gs = guard_empty(torch, x.shape[:1], torch.float32)
    epi = {None: 0, "tanh": 1, "erf": 2}[gelu]
    st = fk.fk_quantize_rows(gx.t.data_ptr(), gq.t.data_ptr(), gs.t.data_ptr(), x.shape[0], x.shape[1],
                             fk.FK_F32 if x.dtype == torch.float32 else fk.FK_BF16,
                             fk.FK_I8 if kind == "i8" else fk.FK_E4M3, epi, torch.cuda.current_stream().cuda_stream)
    assert st == fk.FK_OK, fk.fk_status_string(st)
    torch.cuda.synchronize()
    assert gx.canaries_intact() and gq.canaries_intact() and gs.canaries_intact()
    return to_np(gq.t), to_np(gs.t)


def check(x, kind, gelu, got):
    codes, scales = got
    v = gelu64(to_np(x), gelu)
    t, s = q8.quantize(v, kind)
    nan = np.isnan(s)
    assert np.array_equal(np.isnan(scales), nan) and np.all(codes[nan] == 0)
    # absolute error of the values: the bf16 / fp32 input is exact
    err = np.zeros_like(v) if gelu is None else GELU_ABS + 2.0 ** -20 * np.abs(v)
    ok = ~nan
    q = q8.QMAX[kind]
    amax_err = err[ok].max(axis=-1) if v.shape[1] else 0.0
    assert np.all(np.abs(scales[ok] - s[ok]) <= amax_err / q + 2 * U * s[ok])
    c, t, s, err = codes[ok], t[ok], s[ok, None], err[ok]
    assert np.all(np.abs(c) <= q)
    # the rounding error of the two products, the value's, and the scale's
    wide = np.abs(t) * 4 * U + err / s + np.abs(t) * (amax_err[:, None] / q / s)
    bound = np.maximum(half_step(np.abs(t) + wide, kind), half_step(t, kind)) + wide
    assert np.all(np.abs(c - t) <= bound)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows(fk, torch_mod, rows, cols, dtype, kind):
    x = make_rows(rows, cols, dtype, rows + cols)
    check(x, kind, None, run(fk, torch_mod, x, kind))


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [5, 1000, 2048, 4096, 16384, 40000])
def test_gelu(fk, torch_mod, cols, dtype, kind, gelu):
    x = make_rows(6, cols, dtype, cols)
    check(x, kind, gelu, run(fk, torch_mod, x, kind, gelu))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [48, 1000, 4096, 40000])
def test_misaligned(fk, torch_mod, cols, dtype, kind):
    x = make_rows(5, cols, dtype, cols)
    for xo, qo in ((1, 0), (0, 1), (3, 5), (0, 8)):
        check(x, kind, "tanh", run(fk, torch_mod, x, kind, "tanh", xo, qo))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("cols", [31, 2048, 50001])
def test_special_rows(fk, torch_mod, cols, kind):
    x = make_rows(8, cols, "f32", 1)
    x[0] = 0.0
    x[1, cols - 1] = float("nan")
    x[2, 0] = float("inf")
    x[3, cols // 2] = -float("inf")
    x[4] = 2.0 ** -120                     # below the smallest scale: codes 0
    x[5] = 3.0e38                          # near the largest finite value
    x[6] = -0.0
    c, s = got = run(fk, torch_mod, x, kind)
    check(x, kind, None, got)
    assert np.all(c[[0, 1, 2, 3, 4, 6]] == 0) and np.isnan(s[1:4]).all()
    assert np.all(c[5] == q8.QMAX[kind])


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [40, 64, 255, 1000, 2049, 4096, 9000, 16383, 16384, 40000])
def test_gelu_of_special_rows(fk, torch_mod, cols, dtype, gelu):
    """Rows whose largest magnitude is not at their largest value (all of them
    negative or small), and rows with what is not finite: GELU(-inf) is -0, so
    such a row keeps its scale."""
    x = make_rows(12, cols, dtype, cols + 5)
    x[0] = 0.0
    x[1] = -x[1].abs() - 0.01                 # all negative
    x[2] = -0.75                              # where GELU is lowest
    x[3] = x[3].clamp(-0.7, 0.05)             # the dip outweighs the largest value
    x[4] = -20.0                              # GELU vanishes
    x[5, cols // 2] = float("nan")
    x[6, cols - 1] = float("inf")
    x[7, 0] = -float("inf")
    x[8] = -x[8].abs()
    x[8, cols // 3] = float("nan")            # a NaN among negative values
    x[9] = x[9].clamp(-3.0, 0.17)
    x[10, 0] = 1.0e30
    for kind in ("i8", "e4m3"):
        c, s = got = run(fk, torch_mod, x, kind, gelu)
        check(x, kind, gelu, got)
        assert np.isnan(s[[5, 6, 8]]).all() and np.isfinite(s[[0, 1, 2, 3, 4, 7, 9, 10]]).all()


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [64, 4096, 16384, 20000])
def test_gelu_of_far_values_next_to_each_other(fk, torch_mod, cols, dtype, gelu):
    """Large and far negative values side by side, in either order: what one
    of them exponentiates must not reach the other."""
    x = make_rows(4, cols, dtype, cols + 6)
    x[0, 0] = 1.0e30
    x[0, 2::4], x[0, 3::4] = 1.0e27, -9.0
    x[1, 1] = 3.0e38
    x[1, 2::4], x[1, 3::4] = -40.0, 2.0e37
    x[2] = -7.4
    x[2, 1::2] = 0.4
    x[3] = -7.6
    x[3, ::2] = 60.0
    for kind in ("i8", "e4m3"):
        check(x, kind, gelu, run(fk, torch_mod, x, kind, gelu))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_every_code_and_ties(fk, torch_mod, kind):
    """Rows built to hit every code exactly, and every border between two:
    with the largest value equal to Q the scale is 1 and nothing is rounded
    before the code is; a border goes to the even code."""
    torch = torch_mod
    if kind == "i8":
        vals = np.arange(-127, 128, dtype=np.float64)
    else:
        vals = q8.e4m3_values()
        vals = np.unique(vals[~np.isnan(vals)])
    ties = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, ties])
    x[0] = -q8.QMAX[kind]
    c, s = run(fk, torch, torch.from_numpy(x.astype(np.float32))[None].contiguous(), kind)
    assert s[0] == 1.0
    assert np.array_equal(c[0], q8.round_codes(x, kind))


def test_helper(fk, torch_mod):
    torch = torch_mod
    x = make_rows(6, 96, "bf16", 3).cuda().reshape(2, 3, 96)
    q, s = fk.quantize_rows(x)
    assert q.dtype == torch.int8 and s.shape == (2, 3)
    q2, s2 = fk.quantize_rows(x, torch.float8_e4m3fn, gelu="erf")
    assert q2.dtype == torch.float8_e4m3fn
    out, sc = torch.empty_like(q), torch.empty_like(s)
    assert fk.quantize_rows(x, out=out, scales=sc)[0] is out and torch.equal(out, q) and torch.equal(sc, s)
    assert fk.quantize_rows(x[:0])[0].shape == (0, 3, 96)
    with pytest.raises(TypeError):
        fk.quantize_rows(x, torch.uint8)
    with pytest.raises(ValueError):
        fk.quantize_rows(x, gelu="relu")
    with pytest.raises(ValueError):
        fk.quantize_rows(x[..., :0])
