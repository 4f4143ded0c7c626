"""fk_matmul_q8 on the GPU against exact sums in double.

int8: the sum is exact; its conversion to fp32, two products with the scales
and the addition of the bias round once each: 4 u (|sum sa sb| + |bias|).
e4m3: products are exact in fp32; each of the k / 32 accumulation steps of the
tensor cores may drop what lies 2^-22 below the largest magnitude in it, at
most the sum of magnitudes: (k / 32 + 8) 2^-22 of it.  GELU carries these
through its slope (at most 1.13) and adds its own 2e-6.
"""
import numpy as np
import pytest

from _q8util import GELU_ABS, GELU_SLOPE, U, check_values, gelu64, guard, guard_empty, to_np
from oracle import q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_mod(cuda_device):
    import torch
    return torch


def codes(torch, rows, cols, kind, seed, full=False):
    g = np.random.default_rng(seed)
    if kind == "i8":
        c = g.integers(-128, 128, (rows, cols)) if full else np.clip(np.rint(g.standard_normal((rows, cols)) * 30), -127, 127)
        return torch.from_numpy(c.astype(np.int8))
    v = g.standard_normal((rows, cols)) * (448 if full else 100)
    return torch.from_numpy(np.clip(v, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn)


def operands(torch, m, n, k, kind, bias, seed=0, full=False):
    g = np.random.default_rng(seed + 1000)
    sa = (0.01 * np.exp(0.5 * g.standard_normal(m))).astype(np.float32)
    sb = (0.01 / np.sqrt(k) * np.exp(0.5 * g.standard_normal(n))).astype(np.float32)
    b = (0.1 * g.standard_normal(n)).astype(np.float32) if bias else None
    return codes(torch, m, k, kind, seed, full), codes(torch, n, k, kind, seed + 1, full), sa, sb, b


def run(fk, torch, a, b, sa, sb, bias, out, gelu=None, off=(0, 0, 0), ws=False):
    m, k = a.shape
    n = b.shape[0]
    ga, gb = guard(torch, a, off[0]), guard(torch, b, off[1])
    gsa, gsb = guard(torch, torch.from_numpy(sa)), guard(torch, torch.from_numpy(sb))
    gbias = None if bias is None else guard(torch, torch.from_numpy(bias))
    gc = guard_empty(torch, (m, n), torch.float32 if out == "f32" else torch.bfloat16, off[2])
    args = (ga.t.data_ptr(), gb.t.data_ptr(), gsa.t.data_ptr(), gsb.t.data_ptr(), gbias.t.data_ptr() if gbias else 0,
            gc.t.data_ptr(), m, n, k, fk.FK_I8 if a.dtype == torch.int8 else fk.FK_E4M3,
            fk.FK_F32 if out == "f32" else fk.FK_BF16, {None: 0, "tanh": 1, "erf": 2}[gelu])
    s = torch.cuda.current_stream().cuda_stream
    if ws:
        need = fk.fk_matmul_q8_workspace(m, n, k, ga.t.data_ptr() % 16 == 0 and gb.t.data_ptr() % 16 == 0)
        w = guard_empty(torch, (max(need, 16),), torch.uint8)
        st = fk.fk_matmul_q8_ws(*args, w.t.data_ptr(), need, s)
        torch.cuda.synchronize()
        assert w.canaries_intact()
    else:
        st = fk.fk_matmul_q8(*args, s)
    assert st == fk.FK_OK, fk.fk_status_string(st)
    torch.cuda.synchronize()
    for g in (ga, gb, gsa, gsb, gbias, gc):
        assert g is None or g.canaries_intact(), "write outside a buffer"
    assert fk.fk_wait_timeouts() == 0
    return to_np(gc.t)


def check(a, b, sa, sb, bias, out, gelu, got):
    ref, mag = q8.matmul(to_np(a), to_np(b), sa, sb, bias)
    extra = 4 * U * mag if a.dtype.is_floating_point is False else ((a.shape[1] / 32 + 8) * 2.0 ** -22 + 4 * U) * mag
    if gelu:
        ref, extra = gelu64(ref, gelu), GELU_SLOPE * extra + GELU_ABS
    check_values(got, ref, U, out, "c", extra)


SHAPES = [(1, 1, 1), (1, 1, 16), (1, 17, 16), (2, 128, 32), (1, 4096, 4096), (3, 130, 144), (16, 256, 1024), (17, 255, 272),
          (31, 1000, 512), (33, 129, 4096), (64, 512, 2048), (65, 385, 400), (100, 1024, 160), (128, 128, 128),
          (129, 257, 1040), (200, 300, 8192), (255, 640, 96), (257, 513, 48), (500, 1152, 1600), (513, 2049, 512),
          (1000, 1000, 1008), (2051, 777, 256), (4100, 260, 128), (24, 32001, 64), (7, 5000, 16384), (1, 40, 65536)]


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes(fk, torch_mod, m, n, k, out, kind):
    ops = operands(torch_mod, m, n, k, kind, bias=(m + n) % 2 == 0, seed=m + n + k)
    check(*ops, out, None, run(fk, torch_mod, *ops, out))


@pytest.mark.parametrize("gelu", ["tanh", "erf"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 300, 256), (40, 512, 512), (300, 385, 320), (1030, 520, 144)])
def test_gelu(fk, torch_mod, m, n, k, out, kind, gelu):
    ops = operands(torch_mod, m, n, k, kind, bias=True, seed=m)
    ops = (*ops[:3], ops[3] * 30, ops[4])       # outputs of order 1, both signs
    check(*ops, out, gelu, run(fk, torch_mod, *ops, out, gelu))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 17), (5, 130, 1001), (130, 257, 333), (70, 65, 15), (300, 300, 2047)])
def test_any_k_and_misaligned(fk, torch_mod, m, n, k, kind):
    """k off 16, and a and b off 16 bytes, with and without own workspace."""
    ops = operands(torch_mod, m, n, k, kind, bias=True, seed=k)
    a = run(fk, torch_mod, *ops, "f32")
    check(*ops, "f32", None, a)
    assert np.array_equal(a, run(fk, torch_mod, *ops, "f32", ws=True))
    ops = operands(torch_mod, m, n, k // 16 * 16 + 16, kind, bias=False, seed=k)
    plain = run(fk, torch_mod, *ops, "f32")
    for off in ((1, 0, 0), (0, 3, 0), (5, 7, 1)):
        assert np.array_equal(plain, run(fk, torch_mod, *ops, "f32", off=off))
    check(*ops, "bf16", None, run(fk, torch_mod, *ops, "bf16", off=(0, 0, 1)))


@pytest.mark.parametrize("m,n,k", [(1, 17, 2049), (3, 50, 4097), (90, 9, 6145), (2, 700, 2031), (1, 1, 1), (2, 3, 16385)])
def test_rows_copied_in_several_strips(fk, torch_mod, m, n, k):
    """The copies of operands off 16 bytes, around the 2048 codes that a warp takes of a row, at every lead."""
    ops = operands(torch_mod, m, n, k, "i8", bias=False, seed=k)
    want = run(fk, torch_mod, *ops, "f32")
    check(*ops, "f32", None, want)
    for off in range(1, 16, 2):
        assert np.array_equal(want, run(fk, torch_mod, *ops, "f32", off=(off, 16 - off, 0)))


@pytest.mark.parametrize("m,n", [(1, 64), (40, 200), (300, 260)])
def test_int8_sums_are_exact_at_the_largest_k(fk, torch_mod, m, n):
    """All codes -128 at k = 131071: the sum 2147467264 is below 2^31."""
    torch = torch_mod
    k = 131071 if m == 1 else 131056
    a = torch.full((m, k), -128, dtype=torch.int8)
    b = torch.full((n, k), -128, dtype=torch.int8)
    one = np.ones(m, np.float32), np.ones(n, np.float32)
    c = run(fk, torch, a, b, *one, None, "f32")
    assert np.all(c == np.float32(16384.0 * k))


@pytest.mark.parametrize("m,n,k", [(3, 200, 4096), (150, 140, 1024), (600, 700, 512)])
def test_full_range_int8(fk, torch_mod, m, n, k):
    """Random codes of the whole range with scales 1: sums below 2^24 come out exactly."""
    torch = torch_mod
    a, b, *_ = operands(torch, m, n, k, "i8", False, 5, full=True)
    c = run(fk, torch, a, b, np.ones(m, np.float32), np.ones(n, np.float32), None, "f32")
    ref = to_np(a) @ to_np(b).T
    assert np.max(np.abs(ref)) < 2 ** 24 and np.array_equal(c, ref)


@pytest.mark.parametrize("m,n,k", [(2, 140, 512), (140, 200, 256), (520, 300, 96)])
def test_nan_scales_and_codes_stay_in_their_row(fk, torch_mod, m, n, k):
    torch = torch_mod
    a, b, sa, sb, bias = operands(torch, m, n, k, "e4m3", True, 6)
    sa[0] = np.nan
    sb[3] = np.inf
    a.view(torch.uint8)[1, k - 1] = 0x7F
    c = run(fk, torch, a, b, sa, sb, bias, "f32")
    bad = np.zeros((m, n), bool)
    bad[0], bad[1], bad[:, 3] = True, True, True
    assert np.isnan(c[0]).all() and np.isnan(c[1]).all() and not np.isfinite(c[:, 3]).any()
    assert np.isfinite(c[~bad]).all()


def test_rows_behind_the_last_are_left(fk, torch_mod):
    torch = torch_mod
    a, b, sa, sb, _ = operands(torch, 9, 100, 64, "i8", False, 7)
    a, b, sa, sb = a.cuda(), b.cuda(), torch.from_numpy(sa).cuda(), torch.from_numpy(sb).cuda()
    c = torch.full((9, 100), 7.0, device="cuda")
    st = fk.fk_matmul_q8(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), 0, c.data_ptr(), 5, 100, 64, fk.FK_I8,
                         fk.FK_F32, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and (c[5:] == 7).all() and not (c[:5] == 7).any()


def test_offsets_past_32_bits(fk, torch_mod):
    """An output of more than 2^31 elements: the last rows land in place."""
    torch = torch_mod
    m, n, k = 70001, 32768, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    c = fk.matmul_q8(a, one[0], b, one[1])
    assert c.numel() > 2 ** 31
    for r in (0, 65535, 65536, 70000):
        ref = (a[r].double() @ b.double().T)
        assert torch.equal(c[r], ref.float().bfloat16())


def test_helper_streams_and_graphs(fk, torch_mod):
    torch = torch_mod
    a, b, sa, sb, bias = operands(torch, 24, 320, 1001, "i8", True, 8)
    a, b = a.cuda().reshape(4, 6, 1001), b.cuda()
    sa, sb, bias = torch.from_numpy(sa).cuda().reshape(4, 6), torch.from_numpy(sb).cuda(), torch.from_numpy(bias).cuda()
    want = fk.matmul_q8(a, sa, b, sb, bias, gelu="tanh")
    assert want.shape == (4, 6, 320) and want.dtype == torch.bfloat16
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fk.matmul_q8(a, sa, b, sb, bias, gelu="tanh")
    s.synchronize()
    assert torch.equal(want, got)
    # two graphs with workspaces of their own (k is odd), replayed on two streams at once
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fk.matmul_q8(a, sa, b, sb, bias, gelu="tanh"))
        graphs.append(g)
    for _ in range(3):
        with torch.cuda.stream(s):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert fk.matmul_q8(a[:0], sa[:0], b, sb).shape == (0, 6, 320)
    with pytest.raises(ValueError):
        fk.matmul_q8(a, sa, b[:, :-1].contiguous(), sb)
    with pytest.raises(TypeError):
        fk.matmul_q8(a, sa, b.float(), sb)
    with pytest.raises(ValueError):
        fk.matmul_q8(a, sa[..., :-1].contiguous(), b, sb)
    with pytest.raises(TypeError):
        fk.matmul_q8(a, sa, b, sb, out_dtype=torch.float16)
    with pytest.raises(fk.FkError):
        fk.matmul_q8(a[..., :0].contiguous(), sa, b[:, :0].contiguous(), sb)
