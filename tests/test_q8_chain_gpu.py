"""The 8-bit linear layer as it is used: a block's norm -> product -> GELU to
8 bits -> product -> next norm, for a prompt and for single tokens.

Each step is held to the oracle on its own inputs (a code next to a border
may go either way, so later steps start from the codes that were made); the
whole is held to the unquantised block.  Rounding to codes moves a value by
at most half a step, amax / 254 for int8 (rms amax / 254 / sqrt 3): with rows
whose amax is at most 14 times their rms (12-fold channels on normal values
reach that only rarely, and rows of 4096 would need 50 for the bound below to
fail), relative errors of the two operands of a product are each below
50 / 254 / sqrt 3 = 0.12, random in sign, and those of two products in a row
add: 4 * 0.12 = 0.5 of the result's norm at the very worst; e4m3 (half a step
is 2^-4 relative): 4 * 2^-4 = 0.25."""
import numpy as np
import pytest

from _q8util import (GELU_ABS, U, check_codes, check_values, gelu64, guard_empty, half_step, make_rows, rel_v, to_np)
from oracle import q8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,worst", [("i8", 0.5), ("e4m3", 0.25)])
@pytest.mark.parametrize("rows", [1, 5, 200])
def test_block(fk, cuda_device, rows, kind, worst):
    import torch
    hid, mid = 512, 1536
    dt = torch.int8 if kind == "i8" else torch.float8_e4m3fn
    rng = np.random.default_rng(rows)
    x, r = make_rows(rows, hid, "bf16", 1, 0.3).cuda(), make_rows(rows, hid, "bf16", 2, 0.3).cuda()
    g = (1 + 0.1 * rng.standard_normal(hid)).astype(np.float32)
    w1 = (rng.standard_normal((mid, hid)) / np.sqrt(hid)).astype(np.float32)
    w2 = (rng.standard_normal((hid, mid)) / np.sqrt(mid)).astype(np.float32)
    b1 = (0.1 * rng.standard_normal(mid)).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    gw = dev(g)
    q1, s1 = fk.quantize_rows(dev(w1), dt)          # weights, once
    q2, s2 = fk.quantize_rows(dev(w2), dt)
    a, sa, h = fk.rmsnorm(x, gw, residual=r, out_dtype=dt)
    u = fk.matmul_q8(a, sa, q1, s1, bias=dev(b1))
    c, sc = fk.quantize_rows(u, dt, gelu="tanh")
    y = fk.matmul_q8(c, sc, q2, s2)
    z, h2 = fk.rmsnorm(y, gw, residual=h)
    torch.cuda.synchronize()
    # step by step
    v = q8.rmsnorm(to_np(h), g)
    check_codes(to_np(a), to_np(sa), v, rel_v(hid), kind)
    step = lambda k: (4 * U) if kind == "i8" else (k / 32 + 8) * 2.0 ** -22 + 4 * U  # noqa: E731
    ref, mag = q8.matmul(to_np(a), to_np(q1), to_np(sa), to_np(s1), b1)
    check_values(to_np(u), ref, U, "bf16", "u", step(hid) * mag)
    t, ts = q8.quantize(gelu64(to_np(u), "tanh"), kind)
    wide = GELU_ABS / ts[:, None] * 2 + np.abs(t) * 8 * U
    assert np.all(np.abs(to_np(c) - t) <= half_step(np.abs(t) + wide, kind) + wide)
    ref, mag = q8.matmul(to_np(c), to_np(q2), to_np(sc), to_np(s2))
    check_values(to_np(y), ref, U, "bf16", "y", step(mid) * mag)
    assert torch.equal(h2, (y.float() + h.float()).bfloat16())
    check_values(to_np(z), q8.rmsnorm(to_np(h2), g), rel_v(hid), "bf16", "z")
    # the whole, against the block without 8 bits
    full = gelu64(v @ w1.astype(np.float64).T + b1, "tanh") @ w2.astype(np.float64).T
    assert np.linalg.norm(to_np(y) - full) <= worst * np.linalg.norm(full)


def test_block_captured_and_replayed_on_new_tokens(fk, cuda_device):
    """A decode step in a graph: the residual stream is updated in place, the
    replays see the tokens that were copied in, and equal eager calls."""
    import torch
    hid, mid, rows = 256, 1024, 3
    x, r = make_rows(rows, hid, "bf16", 3).cuda(), make_rows(rows, hid, "bf16", 4).cuda()
    w1, w2 = make_rows(mid, hid, "f32", 5, 0.1).cuda() / 16, make_rows(hid, mid, "f32", 6, 0.1).cuda() / 32
    q1, s1 = fk.quantize_rows(w1)
    q2, s2 = fk.quantize_rows(w2)
    gamma = torch.ones(hid, device="cuda")

    def step(x, stream):
        a, sa, _ = fk.rmsnorm(x, gamma, residual=stream, residual_out=stream, out_dtype=torch.int8)
        c, sc = fk.quantize_rows(fk.matmul_q8(a, sa, q1, s1), gelu="erf")
        return fk.matmul_q8(c, sc, q2, s2)

    sx, sr = torch.zeros_like(x), torch.zeros_like(r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sy = step(sx, sr)
    for seed in range(3):
        xs, rs = make_rows(rows, hid, "bf16", 10 + seed).cuda(), make_rows(rows, hid, "bf16", 20 + seed).cuda()
        sx.copy_(xs)
        sr.copy_(rs)
        graph.replay()
        want = step(xs, rs)     # rs becomes the updated stream
        torch.cuda.synchronize()
        assert torch.equal(sy, want) and torch.equal(sr, rs)
    assert guard_empty(torch, (4,), torch.float32).canaries_intact()
