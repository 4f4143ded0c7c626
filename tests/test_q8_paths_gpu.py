"""Row kernels of the 8-bit layer on the paths that few shapes reach: aligned
rows of 65537 to 131072 columns (clusters of eight), the two-block GELU
quantiser on shifted rows, sums of dgamma to which every row counts, products
with k off 16 at every lead."""
import numpy as np
import pytest

from _q8util import chain, check_codes, check_values, guard, guard_empty, make_rows, rel_v, to_np
from oracle import q8

pytestmark = pytest.mark.gpu


def dt(torch, kind):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}[kind]


@pytest.mark.parametrize("out", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(5, 65536), (3, 65544), (3, 80000), (2, 98304), (40, 100000), (2, 131072)])
def test_norm_of_very_long_aligned_rows(fk, cuda_device, rows, cols, dtype, out):
    import torch
    x, r = make_rows(rows, cols, dtype, 1), make_rows(rows, cols, dtype, 2)
    g = (1.0 + 0.3 * np.random.default_rng(cols).standard_normal(cols)).astype(np.float32)
    w = torch.from_numpy(g).cuda()
    got = fk.rmsnorm(x.cuda(), w, residual=r.cuda(), out_dtype=dt(torch, out) if out else None)
    h = (x.float() + r.float()).to(x.dtype)
    assert torch.equal(got[-1].cpu(), h)
    v = q8.rmsnorm(to_np(h), g)
    if out:
        check_codes(to_np(got[0]), to_np(got[1]), v, rel_v(cols), out)
    else:
        check_values(to_np(got[0]), v, rel_v(cols), dtype, "y")


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(5, 65536), (3, 65544), (2, 98304), (40, 100000), (2, 131072)])
def test_codes_of_very_long_aligned_rows(fk, cuda_device, rows, cols, dtype, kind):
    import torch
    x = make_rows(rows, cols, dtype, 3)
    c, s = fk.quantize_rows(x.cuda(), dt(torch, kind))
    check_codes(to_np(c), to_np(s), to_np(x), 0.0, kind)


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("cols", [16385, 16392, 20001, 24571, 32765, 32768])
def test_gelu_rows_of_two_blocks(fk, cuda_device, cols, kind, gelu):
    """bf16 rows of 16385 to 32768 columns, at every lead a row and a buffer
    can have: equal to the same rows one by one in fp32."""
    import torch
    x = make_rows(9, cols, "bf16", cols)
    x[3] *= 0.02
    for off in (0, 1, 4):
        gx = guard(torch, x, off)
        gq, gs = guard_empty(torch, x.shape, dt(torch, kind), off), guard_empty(torch, x.shape[:1], torch.float32)
        st = fk.fk_quantize_rows(gx.t.data_ptr(), gq.t.data_ptr(), gs.t.data_ptr(), 9, cols, fk.FK_BF16,
                                 fk.FK_I8 if kind == "i8" else fk.FK_E4M3, {"tanh": 1, "erf": 2}[gelu],
                                 torch.cuda.current_stream().cuda_stream)
        assert st == fk.FK_OK
        torch.cuda.synchronize()
        assert gx.canaries_intact() and gq.canaries_intact() and gs.canaries_intact()
        for i in range(9):
            # the same values as fp32, through another kernel
            c, s = fk.quantize_rows(x[i:i + 1].float().cuda(), dt(torch, kind), gelu=gelu)
            assert torch.equal(gs.t[i], s[0]) and torch.equal(gq.t[i].view(torch.uint8), c[0].view(torch.uint8))


SUM_SHAPES = [(20001, 59), (9001, 128), (9001, 119), (5003, 64), (333, 57), (7, 128), (3001, 255), (2400, 512), (1300, 511),
              (1201, 1001), (1200, 1000), (1500, 1088), (999, 2047), (4001, 4096), (700, 5120), (331, 6144), (170, 8193),
              (401, 12288), (501, 16384), (333, 16383), (90, 20001), (251, 32768), (161, 32767), (41, 40000), (37, 65536),
              (5, 70000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SUM_SHAPES)
def test_every_row_counts_once_in_dgamma(fk, cuda_device, rows, cols, dtype):
    """h of +-1 with eps = 0 has r = 1 (cols times its rounded reciprocal
    rounds to 1), so that dgamma is a sum of integers, exact in any order: a
    row left out, or counted twice, shows."""
    import torch
    assert np.float32(np.float64(cols) * np.float64(np.float32(1) / np.float32(cols))) == 1
    g = torch.Generator(device="cuda").manual_seed(rows)
    h = (torch.randint(0, 2, (rows, cols), generator=g, device="cuda") * 2 - 1).to(dt(torch, dtype))
    dy = torch.randint(-4, 5, (rows, cols), generator=g, device="cuda").to(dt(torch, dtype))
    want = (dy.double() * h.double()).sum(0)
    for res in (None, h):
        _, dw = fk.rmsnorm_backward(dy, h, eps=0.0, dresidual=res)
        assert torch.equal(dw.double(), want)
    # value by value: dgamma's other way
    w = torch.ones(cols + 1, device="cuda")[1:]
    dx, dw = fk.rmsnorm_backward(dy, h, w, eps=0.0)
    assert torch.equal(dw.double(), want)
    # dx = dy - mean(dy h) h, the mean an exact sum over cols rounded
    s = (dy.double() * h.double()).mean(dim=1, keepdim=True)
    ref = dy.double() - s * h.double()
    assert bool(((dx.double() - ref).abs() <= (ref.abs() * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
                                               + (s.abs() + dy.double().abs()) * chain(cols) * 2.0 ** -24)).all())


@pytest.mark.parametrize("m,n,k", [(3, 50, 15), (3, 50, 17), (2, 33, 31), (1, 17, 127), (5, 40, 129), (2, 300, 2049), (90, 70, 143)])
def test_products_at_every_lead(fk, cuda_device, m, n, k):
    """The copies of operands off 16 bytes take 16 codes a thread: rows that end in every way within them, bases at
    every place, one operand copied and both."""
    import torch
    g = np.random.default_rng(k)
    a, b = (torch.from_numpy(g.integers(-128, 128, s).astype(np.int8)) for s in ((m, k), (n, k)))
    one = torch.ones(max(m, n), device="cuda")
    want = to_np(a) @ to_np(b).T
    for off in range(16):
        for ga, gb in ((guard(torch, a, off), guard(torch, b, 0)), (guard(torch, a, off), guard(torch, b, 15 - off))):
            c = guard_empty(torch, (m, n), torch.float32, off % 3)
            st = fk.fk_matmul_q8(ga.t.data_ptr(), gb.t.data_ptr(), one.data_ptr(), one.data_ptr(), 0, c.t.data_ptr(), m, n,
                                 k, fk.FK_I8, fk.FK_F32, 0, torch.cuda.current_stream().cuda_stream)
            assert st == fk.FK_OK
            torch.cuda.synchronize()
            assert ga.canaries_intact() and gb.canaries_intact() and c.canaries_intact()
            assert np.array_equal(to_np(c.t), want)
