"""Codes of 8-bit rows, bit for bit: with the scale s = fl32(max fl32(1 / Q))
that a call returns, the code of an fp32 value v is fl32(v / s) rounded to nearest
even.  Rows of bf16 values make this sharp: their quotients by max / Q stand
often exactly on a border between two codes, and only the rounding of s and
of the quotient says which code it is."""
import numpy as np
import pytest

from _q8util import guard, guard_empty, make_rows, to_np
from oracle import q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_mod(cuda_device):
    import torch
    return torch


def tdtype(torch, kind):
    return torch.int8 if kind == "i8" else torch.float8_e4m3fn


def want(v, kind):
    """(codes, scales) of fp32 values by numpy's fp32 arithmetic."""
    v = v.astype(np.float32)
    assert np.isfinite(v).all()
    s = np.maximum(np.abs(v).max(axis=-1), np.float32(2.0 ** -100)) * (np.float32(1) / np.float32(q8.QMAX[kind]))
    t = (v / s[:, None]).astype(np.float64)
    return q8.round_codes(t, kind), s


def check(got, v, kind):
    codes, scales = want(v, kind)
    assert np.array_equal(to_np(got[1]).astype(np.float32), scales)
    bad = to_np(got[0]) != codes
    assert not bad.any(), f"{bad.sum()} of {bad.size} codes are not those of v / scale"


# every kind of team: parts of a warp, a warp, blocks, resident blocks past their first row, clusters of two,
# four and eight, shifted rows, the streamed ones
SHAPES = [(9, 40), (9, 61), (33, 128), (33, 250), (33, 1000), (33, 1024), (17, 4096), (17, 4095), (7, 12288),
          (700, 8200), (320, 16384), (9, 16383), (5, 20000), (5, 20001), (3, 32768), (3, 40000), (2, 100003), (1, 140000)]


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_of_rows(fk, torch_mod, rows, cols, dtype, kind):
    torch = torch_mod
    x = make_rows(rows, cols, dtype, rows + cols)
    check(fk.quantize_rows(x.cuda(), tdtype(torch, kind)), x.float().numpy(), kind)
    # the fp32 values of a bf16 row, whose quotients are the same
    if dtype == "f32":
        b = x.bfloat16().float()
        check(fk.quantize_rows(b.cuda(), tdtype(torch, kind)), b.numpy(), kind)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_are_those_of_the_elementary_operations(fk, torch_mod, dtype, kind):
    torch = torch_mod
    x = make_rows(1000, 2048, dtype, 9).cuda()
    q, s = fk.quantize_rows(x, tdtype(torch, kind))
    scale = x.float().abs().amax(dim=-1, keepdim=True) / q8.QMAX[kind]
    t = x.float() / scale
    assert torch.equal(s, scale[:, 0])
    assert torch.equal(q.float(), (t.round() if kind == "i8" else t.clamp(-448, 448)).to(q.dtype).float())


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_through_gelu_where_it_is_the_identity(fk, torch_mod, rows, cols, dtype, kind, gelu):
    """GELU(x) = x to fp32 from 6 on (1 - GELU(x) / x is 1e-9 at 6): rows of
    values of 8 to 800 have codes that nothing but the quotient decides."""
    torch = torch_mod
    g = np.random.default_rng(rows + cols)
    x = torch.from_numpy(np.exp(g.uniform(np.log(8.0), np.log(800.0), (rows, cols))).astype(np.float32)).bfloat16()
    x = x if dtype == "bf16" else x.float()
    check(fk.quantize_rows(x.cuda(), tdtype(torch, kind), gelu=gelu), x.float().numpy(), kind)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("rows,cols", [(33, 64), (33, 1000), (17, 4096), (9, 4095), (5, 20000), (3, 40000), (1, 140000)])
def test_codes_of_the_norm(fk, torch_mod, rows, cols, kind):
    """The fp32 norm and the one to 8 bits hold the same fp32 values: the
    codes are those of the stored ones."""
    torch = torch_mod
    x, r = make_rows(rows, cols, "f32", cols).cuda(), make_rows(rows, cols, "f32", cols + 1).cuda()
    w = torch.from_numpy((1 + 0.3 * np.random.default_rng(cols).standard_normal(cols)).astype(np.float32)).cuda()
    y, _ = fk.rmsnorm(x, w, residual=r)
    q, s, _ = fk.rmsnorm(x, w, residual=r, out_dtype=tdtype(torch, kind))
    check((q, s), y.cpu().numpy(), kind)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_rows_of_every_size_and_off_16_bytes(fk, torch_mod, kind):
    """Rows from 2^-96 to 2^110 (values of up to 2^7 times a power of two)."""
    torch = torch_mod
    for cols in (24, 57, 2048, 2049):
        x = make_rows(24, cols, "bf16", cols, 0.1).float()
        x *= 2.0 ** torch.linspace(-96, 103, 24).floor()[:, None]
        gx = guard(torch, x, 1)
        gq, gs = guard_empty(torch, x.shape, tdtype(torch, kind), 3), guard_empty(torch, x.shape[:1], torch.float32)
        st = fk.fk_quantize_rows(gx.t.data_ptr(), gq.t.data_ptr(), gs.t.data_ptr(), 24, cols, fk.FK_F32,
                                 fk.FK_I8 if kind == "i8" else fk.FK_E4M3, 0, torch.cuda.current_stream().cuda_stream)
        assert st == fk.FK_OK
        torch.cuda.synchronize()
        assert gx.canaries_intact() and gq.canaries_intact() and gs.canaries_intact()
        check((gq.t, gs.t), x.numpy(), kind)
