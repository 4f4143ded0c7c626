"""fk_rmsnorm_rows and fk_rmsnorm_rows_bwd on the GPU against the
double-precision oracle; bounds in _q8util."""
import numpy as np
import pytest

from _q8util import (EPS_HALF, U, chain, check_codes, check_values, guard, guard_empty, make_rows, rel_v, to_np)
from oracle import q8

pytestmark = pytest.mark.gpu

SHAPES = [(37, 1), (3, 7), (65, 64), (33, 1000), (5, 1023), (17, 1024), (17, 1025), (9, 2048), (9, 2049), (6, 4096),
          (5, 4097), (1, 8192), (5, 8200), (3, 16384), (2, 16385), (2, 32768), (2, 32769), (2, 100003), (1, 262144)]


@pytest.fixture(scope="module")
def torch_mod(cuda_device):
    import torch
    return torch


def tdtype(torch, kind):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}[kind]


def code(fk, kind):
    return {"f32": fk.FK_F32, "bf16": fk.FK_BF16, "i8": fk.FK_I8, "e4m3": fk.FK_E4M3}[kind]


def gamma_of(cols, seed):
    return (1.0 + 0.3 * np.random.default_rng(seed).standard_normal(cols)).astype(np.float32)


def forward(fk, torch, x, res, gamma, out, eps=1e-6, keep_h=True, off=(0, 0, 0, 0, 0), alias=None):
    """Through the C ABI into guarded buffers: (y, scales, h) as float64.
    alias: "h=x", "h=r", "y=x", "y=r"."""
    dt = "f32" if x.dtype == torch.float32 else "bf16"
    out = dt if out is None else out
    gx = guard(torch, x, off[0])
    gr = None if res is None else guard(torch, res, off[1])
    gg = None if gamma is None else guard(torch, torch.from_numpy(gamma), off[4])
    q = out in q8.QMAX
    gy = {"y=x": gx, "y=r": gr}.get(alias) or guard_empty(torch, x.shape, tdtype(torch, out), off[2])
    gh = None
    if res is not None and keep_h:
        gh = {"h=x": gx, "h=r": gr}.get(alias) or guard_empty(torch, x.shape, x.dtype, off[3])
    gs = guard_empty(torch, x.shape[:1], torch.float32) if q else None
    p = lambda g: g.t.data_ptr() if g is not None else 0  # noqa: E731
    st = fk.fk_rmsnorm_rows(p(gx), p(gr), p(gg), p(gy), p(gs), p(gh), x.shape[0], x.shape[1], code(fk, dt),
                            code(fk, out), eps, torch.cuda.current_stream().cuda_stream)
    assert st == fk.FK_OK, fk.fk_status_string(st)
    torch.cuda.synchronize()
    for g in (gx, gr, gg, gy, gs, gh):
        assert g is None or g.canaries_intact(), "write outside a buffer"
    if alias is None:   # inputs are left as they were
        assert torch.equal(gx.t.cpu(), x) or torch.isnan(x.float()).any()
    return to_np(gy.t), None if gs is None else to_np(gs.t), None if gh is None else to_np(gh.t)


def check_forward(x, res, gamma, out, got, eps=1e-6):
    y, s, h = got
    dt = "f32" if x.dtype.itemsize == 4 else "bf16"
    hh = x if res is None else (x.float() + res.float()).to(x.dtype)
    if h is not None:
        assert np.array_equal(h, to_np(hh), equal_nan=True), "h is not the rounded sum"
    v = q8.rmsnorm(to_np(hh), gamma, eps)
    cols = x.shape[1]
    if out in q8.QMAX:
        check_codes(y, s, v, rel_v(cols), out)
    else:
        check_values(y, v, rel_v(cols), dt, "y")


@pytest.mark.parametrize("out", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(fk, torch_mod, rows, cols, dtype, out):
    x, r = make_rows(rows, cols, dtype, cols + 1), make_rows(rows, cols, dtype, cols + 2)
    g = gamma_of(cols, cols)
    check_forward(x, r, g, out, forward(fk, torch_mod, x, r, g, out))
    check_forward(x, None, None, out, forward(fk, torch_mod, x, None, None, out))
    check_forward(x, r, None, out, forward(fk, torch_mod, x, r, None, out, keep_h=False))


@pytest.mark.parametrize("out", [None, "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 256), (149, 256), (1200, 256), (2400, 512), (1, 4096), (300, 4096),
                                       (1500, 4096), (701, 1003), (4000, 129), (5003, 64),
                                       (5001, 63), (333, 57), (2999, 128), (2999, 122), (7, 128), (1, 48), (3, 113)])
def test_many_rows(fk, torch_mod, rows, cols, dtype, out):
    """Row counts on both sides of what fills the GPU (kernel shapes depend on it)."""
    x, r = make_rows(rows, cols, dtype, rows), make_rows(rows, cols, dtype, rows + 1)
    g = gamma_of(cols, 5)
    check_forward(x, r, g, out, forward(fk, torch_mod, x, r, g, out))


@pytest.mark.parametrize("out", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [64, 1000, 4096, 40000])
def test_misaligned_buffers(fk, torch_mod, cols, dtype, out):
    x, r, g = make_rows(4, cols, dtype, 1), make_rows(4, cols, dtype, 2), gamma_of(cols, 3)
    for off in ((1, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 1, 0, 0), (0, 0, 0, 1, 0), (0, 0, 0, 0, 1), (1, 3, 5, 2, 1), (1, 1, 1, 1, 0), (3, 3, 3, 3, 0),
                (2, 2, 7, 2, 0)):
        check_forward(x, r, g, out, forward(fk, torch_mod, x, r, g, out, off=off))


@pytest.mark.parametrize("out", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 8, 9, 15, 31, 33, 250, 255, 257, 505, 513, 1017, 1021, 1025, 2047, 4089, 4091,
                                  4093, 4097, 8191, 16379, 32761, 32765])
def test_rows_that_start_off_16_bytes(fk, torch_mod, cols, dtype, out):
    """Every lead a row can have (nine rows of an odd width), around the widths where the kernels change."""
    x, r, g = make_rows(9, cols, dtype, cols), make_rows(9, cols, dtype, cols + 1), gamma_of(cols, 3)
    check_forward(x, r, g, out, forward(fk, torch_mod, x, r, g, out))
    check_forward(x, r, g, out, forward(fk, torch_mod, x, r, g, out, off=(1, 1, 1, 1, 0)))
    if out is None:
        check_forward(x, r, g, out, forward(fk, torch_mod, x, r, g, out, alias="h=r"))
        dy = make_rows(9, cols, dtype, cols + 2)
        check_backward(dy, x, g, r, backward(fk, torch_mod, dy, x, g, r))
        check_backward(dy, x, g, r, backward(fk, torch_mod, dy, x, g, r, off=0, alias="dy"))


@pytest.mark.parametrize("alias", ["h=x", "h=r", "y=x", "y=r"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [65, 1024, 4096, 40000])
def test_in_place(fk, torch_mod, cols, dtype, alias):
    x, r, g = make_rows(5, cols, dtype, 4), make_rows(5, cols, dtype, 5), gamma_of(cols, 6)
    out = None if alias[0] == "y" else "i8"
    for o in {out, None}:
        check_forward(x, r, g, o, forward(fk, torch_mod, x, r, g, o, alias=alias))
        if alias[0] == "y":
            check_forward(x, r, g, o, forward(fk, torch_mod, x, r, g, o, alias=alias, keep_h=False))


@pytest.mark.parametrize("out", [None, "i8", "e4m3"])
@pytest.mark.parametrize("cols", [33, 2048, 50001])
def test_special_rows(fk, torch_mod, cols, out):
    x = make_rows(7, cols, "f32", 8)
    x[0] = 0.0
    x[1, cols // 2] = float("nan")
    x[2, cols - 1] = float("inf")
    x[3] = 1e-30
    x[4, 0] = -float("inf")
    x[5] = 0.0
    x[5, cols // 3] = -3.0
    g = gamma_of(cols, 9)
    got = forward(fk, torch_mod, x, None, g, out)
    check_forward(x, None, g, out, got)
    if out in q8.QMAX:
        assert got[1][0] == np.float32(np.float32(q8.TINY) / np.float32(q8.QMAX[out])) and np.all(got[0][0] == 0)
        assert np.isnan(got[1][[1, 2, 4]]).all() and np.all(got[0][[1, 2, 4]] == 0)
        assert abs(got[0][5, cols // 3]) == q8.QMAX[out]
    else:
        assert np.all(got[0][0] == 0) and np.isnan(got[0][[1, 2, 4]]).all()


@pytest.mark.parametrize("eps", [0.0, 1e-5, 1.0])
def test_eps_and_zero_gamma(fk, torch_mod, eps):
    x, g = make_rows(6, 640, "f32", 10), gamma_of(640, 11)
    check_forward(x, None, g, None, forward(fk, torch_mod, x, None, g, None, eps), eps)
    z = np.zeros(640, np.float32)
    y, s, _ = forward(fk, torch_mod, x, None, z, "e4m3", eps)
    assert np.all(y == 0) and np.all(s > 0)


def test_residual_cancels_to_zero(fk, torch_mod):
    x = make_rows(3, 512, "bf16", 12)
    y, _, h = forward(fk, torch_mod, x, -x, None, None)
    assert np.all(h == 0) and np.all(y == 0)


# ---------------------------------------------------------------- backward

def backward(fk, torch, dy, h, gamma, dres, want=True, eps=1e-6, off=0, alias=None, ws=None):
    dt = "f32" if h.dtype == torch.float32 else "bf16"
    gd, gh = guard(torch, dy, off), guard(torch, h, off)
    gr = None if dres is None else guard(torch, dres)
    gg = None if gamma is None else guard(torch, torch.from_numpy(gamma), off)
    gx = {"dy": gd, "h": gh, "dres": gr}.get(alias) or guard_empty(torch, h.shape, h.dtype, off)
    gw = guard_empty(torch, h.shape[1:], torch.float32) if want else None
    p = lambda g: g.t.data_ptr() if g is not None else 0  # noqa: E731
    args = (p(gd), p(gh), p(gg), p(gr), p(gx), p(gw), h.shape[0], h.shape[1], code(fk, dt), eps)
    s = torch.cuda.current_stream().cuda_stream
    if ws is None:
        st = fk.fk_rmsnorm_rows_bwd(*args, s)
    else:
        n = fk.fk_rmsnorm_rows_bwd_workspace(h.shape[0], h.shape[1], code(fk, dt), want)
        w = guard_empty(torch, (max(n, 16),), torch.uint8)
        st = fk.fk_rmsnorm_rows_bwd_ws(*args, p(w), n, s)
        torch.cuda.synchronize()
        assert w.canaries_intact()
    assert st == fk.FK_OK, fk.fk_status_string(st)
    torch.cuda.synchronize()
    for g in (gd, gh, gr, gg, gx, gw):
        assert g is None or g.canaries_intact()
    return to_np(gx.t), None if gw is None else to_np(gw.t)


def check_backward(dy, h, gamma, dres, got, eps=1e-6):
    """dx's error: the two terms' own roundings; r's error (3 times over in
    r^3); and that of s, which is relative to the sum of magnitudes."""
    dx, dw = got
    d, hh = to_np(dy), to_np(h)
    rdx, rdw = q8.rmsnorm_backward(d, hh, gamma, eps, None if dres is None else to_np(dres))
    r = q8.rstd(hh, eps)
    g = d if gamma is None else d * gamma
    n, rv = h.shape[1], rel_v(h.shape[1])
    sabs = np.mean(np.abs(g * hh), axis=-1, keepdims=True)
    t1, t2 = np.abs(r * g), np.abs(r ** 3 * hh) * sabs
    extra = (rv + 3 * U) * t1 + (3 * rv + (chain(n) + 8) * U) * t2
    if dres is not None:
        extra = extra + U * (t1 + t2)
    check_values(dx, rdx, 2 * U, "f32" if h.dtype.itemsize == 4 else "bf16", "dx", extra)
    if dw is not None:
        mag = np.sum(np.abs(d * hh * r), axis=0)
        check_values(dw, rdw, 2 * U, "f32", "dgamma", (rv + (h.shape[0] + 4) * U) * mag)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(300, 64), (1200, 1000), (999, 4096), (150, 8192), (130, 16384), (999, 2047), (3001, 255),
                                                (1300, 511), (1201, 1001), (170, 8193), (90, 20001), (5003, 64), (20001, 61),
                                                (333, 57), (9001, 128), (9001, 122), (7, 128), (1, 48)])
def test_backward(fk, torch_mod, rows, cols, dtype):
    dy, h, dr = (make_rows(rows, cols, dtype, cols + i, 0.3) for i in range(3))
    g = gamma_of(cols, cols)
    check_backward(dy, h, g, dr, backward(fk, torch_mod, dy, h, g, dr))
    check_backward(dy, h, None, None, backward(fk, torch_mod, dy, h, None, None))
    check_backward(dy, h, g, None, backward(fk, torch_mod, dy, h, g, None, want=False))


@pytest.mark.parametrize("alias", ["dy", "h", "dres"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [100, 4096, 40000])
def test_backward_in_place(fk, torch_mod, cols, dtype, alias):
    dy, h, dr = (make_rows(40, cols, dtype, 7 + i, 0.3) for i in range(3))
    g = gamma_of(cols, 1)
    check_backward(dy, h, g, dr, backward(fk, torch_mod, dy, h, g, dr, alias=alias))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [64, 2048, 40000])
def test_backward_misaligned_and_own_workspace(fk, torch_mod, cols, dtype):
    dy, h, dr = (make_rows(9, cols, dtype, 20 + i, 0.3) for i in range(3))
    g = gamma_of(cols, 2)
    a = backward(fk, torch_mod, dy, h, g, dr, off=1)
    check_backward(dy, h, g, dr, a)
    b = backward(fk, torch_mod, dy, h, g, dr, ws=True)
    check_backward(dy, h, g, dr, b)
    c = backward(fk, torch_mod, dy, h, g, dr)
    assert np.array_equal(b[0], c[0]) and np.array_equal(b[1], c[1]), "workspace changes the result"


def test_backward_matches_differences(fk, torch_mod):
    """dx and dgamma against central differences of the kernel's own forward
    pass: with step d and third derivatives of order 1 the difference is off
    by d^2 and by the forward's rounding over d (2^-20 |y| summed over a row
    of 24, over 2 d)."""
    torch = torch_mod
    rng = np.random.default_rng(0)
    h = torch.from_numpy(rng.standard_normal((4, 24)).astype(np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((4, 24)).astype(np.float32)).cuda()
    w = torch.from_numpy(gamma_of(24, 3)).cuda()
    dx, dw = fk.rmsnorm_backward(dy, h, w, 1e-3)
    step = 2.0 ** -6
    loss = lambda hh, ww: (fk.rmsnorm(hh, ww, 1e-3).double() * dy.double()).sum().item()  # noqa: E731
    tol = 4 * step ** 2 + 24 * 4 * 2.0 ** -20 / step
    for i, j in [(0, 0), (1, 5), (2, 23), (3, 11)]:
        p, m = h.clone(), h.clone()
        p[i, j] += step
        m[i, j] -= step
        assert abs((loss(p, w) - loss(m, w)) / (2 * step) - dx[i, j].item()) < tol
        p, m = w.clone(), w.clone()
        p[j] += step
        m[j] -= step
        assert abs((loss(h, p) - loss(h, m)) / (2 * step) - dw[j].item()) < tol


def test_backward_special_rows_and_no_rows(fk, torch_mod):
    torch = torch_mod
    dy, h = make_rows(4, 300, "f32", 30), make_rows(4, 300, "f32", 31)
    h[0] = 0.0
    h[1, 7] = float("inf")
    dx, _ = backward(fk, torch, dy, h, None, None)
    with np.errstate(invalid="ignore"):
        assert np.isnan(dx[1]).all() and np.isfinite(dx[[0, 2, 3]]).all()
    assert np.allclose(dx[0], to_np(dy)[0] * 1e3, rtol=1e-5)     # r = 1 / sqrt(eps)
    e = torch.empty(0, 64, device="cuda")
    dxe, dwe = fk.rmsnorm_backward(e, e)
    assert dxe.shape == (0, 64) and torch.equal(dwe.cpu(), torch.zeros(64))


def test_equal_calls_give_equal_bits(fk, torch_mod):
    torch = torch_mod
    dy, h = (make_rows(2000, 1536, "bf16", i).cuda() for i in range(2))
    w = torch.from_numpy(gamma_of(1536, 3)).cuda()
    a, b = fk.rmsnorm_backward(dy, h, w), fk.rmsnorm_backward(dy, h, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- helpers, streams, graphs

def test_tensor_helper(fk, torch_mod):
    torch = torch_mod
    x = make_rows(12, 768, "bf16", 40).cuda().reshape(3, 4, 768)
    r, w = make_rows(12, 768, "bf16", 41).cuda().reshape(3, 4, 768), torch.from_numpy(gamma_of(768, 42)).cuda()
    y, h = fk.rmsnorm(x, w, residual=r)
    assert y.shape == x.shape and torch.equal(h, (x.float() + r.float()).bfloat16())
    check_values(to_np(y).reshape(12, 768), q8.rmsnorm(to_np(h).reshape(12, 768), w.cpu().numpy()), rel_v(768), "bf16")
    q, s = fk.rmsnorm(x, w, out_dtype=torch.int8)
    assert q.dtype == torch.int8 and s.shape == (3, 4)
    buf = r.clone()
    q2, s2, h2 = fk.rmsnorm(x, w, residual=buf, residual_out=buf, out=torch.empty_like(q))
    assert h2 is buf and torch.equal(buf, h) and q2.dtype == torch.int8
    assert fk.rmsnorm(x[:0], w).shape == (0, 4, 768)
    with pytest.raises(ValueError):
        fk.rmsnorm(x.transpose(0, 1), w)
    with pytest.raises(ValueError):
        fk.rmsnorm(x, w[:-1])
    with pytest.raises(TypeError):
        fk.rmsnorm(x, w, out_dtype=torch.float32)
    with pytest.raises(ValueError):
        fk.rmsnorm(x, w, residual_out=buf)
    with pytest.raises(TypeError):
        fk.rmsnorm(x.half(), w)
    with pytest.raises(fk.FkError):
        fk.rmsnorm(x, w, eps=-1.0)


def test_another_stream_and_a_captured_graph(fk, torch_mod):
    """Calls go to the current stream; a graph of both directions replays on
    new contents while eager calls run beside it."""
    torch = torch_mod
    dy, x, r = (make_rows(64, 2048, "bf16", 50 + i).cuda() for i in range(3))
    w = torch.from_numpy(gamma_of(2048, 1)).cuda()
    want = fk.rmsnorm(x, w, residual=r), fk.rmsnorm_backward(dy, x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fk.rmsnorm(x, w, residual=r), fk.rmsnorm_backward(dy, x, w)
    s.synchronize()
    assert all(torch.equal(a, b) for p, q in zip(want, got) for a, b in zip(p, q))
    g = torch.cuda.CUDAGraph()
    xs, rs, ds = torch.zeros_like(x), torch.zeros_like(r), torch.zeros_like(dy)
    with torch.cuda.graph(g):
        outs = fk.rmsnorm(xs, w, residual=rs), fk.rmsnorm_backward(ds, xs, w)
    for src, dst in ((x, xs), (r, rs), (dy, ds)):
        dst.copy_(src)
    for _ in range(2):
        g.replay()
        eager = fk.rmsnorm_backward(dy, x, w)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(want, outs) for a, b in zip(p, q))
        assert torch.equal(eager[1], want[1][1])


def test_rows_behind_the_last_are_left(fk, torch_mod):
    torch = torch_mod
    x = make_rows(10, 1024, "bf16", 60).cuda()
    out = torch.full_like(x, 7.0)
    scales = torch.full((10,), 3.0, device="cuda")
    codes = torch.full((10, 1024), 9, dtype=torch.int8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert fk.fk_rmsnorm_rows(x.data_ptr(), 0, 0, out.data_ptr(), 0, 0, 6, 1024, fk.FK_BF16, fk.FK_BF16, 1e-6, s) == 0
    assert fk.fk_rmsnorm_rows(x.data_ptr(), 0, 0, codes.data_ptr(), scales.data_ptr(), 0, 6, 1024, fk.FK_BF16, fk.FK_I8,
                              1e-6, s) == 0
    torch.cuda.synchronize()
    assert (out[6:] == 7).all() and (scales[6:] == 3).all() and (codes[6:] == 9).all() and EPS_HALF["f32"] == U


@pytest.mark.parametrize("cols", [64, 1001, 4096, 12000, 40000])
def test_backward_of_tiny_rows(fk, torch_mod, cols):
    """Rows of about 1e-14 with eps = 0: r is about 1e14 and r^3 beyond fp32, the gradients are not."""
    h = make_rows(5, cols, "f32", cols) * 1e-14
    dy, g = make_rows(5, cols, "f32", cols + 1), gamma_of(cols, 3)
    got = backward(fk, torch_mod, dy, h, g, None, True, 0.0)
    assert np.isfinite(got[0]).all() and np.abs(got[0]).max() > 1e13
    check_backward(dy, h, g, None, got, 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1500, 1056), (700, 5120), (330, 6144), (500, 16384), (333, 16383), (401, 12288), (250, 32768),
                                       (161, 32767)])
def test_backward_many_rows_a_team(fk, torch_mod, rows, cols, dtype):
    """Long rows, several to each resident team: every place of the two that are staged is used again, in place too."""
    dy, h, dr = (make_rows(rows, cols, dtype, cols + i, 0.3) for i in range(3))
    g = gamma_of(cols, cols)
    want = backward(fk, torch_mod, dy, h, g, dr)
    check_backward(dy, h, g, dr, want)
    for alias in ("dy", "h", "dres"):
        got = backward(fk, torch_mod, dy, h, g, dr, alias=alias)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    check_backward(dy, h, g, None, backward(fk, torch_mod, dy, h, g, None))


def test_calls_from_two_threads(fk, torch_mod):
    """Two host threads, each on its stream, with shapes that share a kernel and differ in its shared memory."""
    import threading

    torch = torch_mod
    cases = [(300, 1100, False), (300, 8192, True), (40, 16384, True), (64, 1056, False)]
    data, want, got, errors = [], [], [None] * len(cases), []
    for i, (rows, cols, res) in enumerate(cases):
        t = [make_rows(rows, cols, "f32", 10 * i + j).cuda() for j in range(3)]
        data.append((t[0], t[1], t[2] if res else None))
        want.append(fk.rmsnorm_backward(t[0], t[1], dresidual=data[i][2]))
    torch.cuda.synchronize()

    def work(mine):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    for i in mine:
                        got[i] = fk.rmsnorm_backward(data[i][0], data[i][1], dresidual=data[i][2])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(m,)) for m in ((0, 2), (1, 3))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
