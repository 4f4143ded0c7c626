"""Pins of the 8-bit linear layer's oracle: closed forms, differences,
invariants, and torch's own float64 and float8 arithmetic (CPU only)."""
import numpy as np
import pytest

from oracle import q8


def test_e4m3_table_matches_torch():
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = q8.e4m3_values()
    assert np.array_equal(np.isnan(t), np.isnan(v))
    ok = ~np.isnan(v)
    assert np.array_equal(t[ok], v[ok]) and np.nanmax(v) == 448.0


def test_round_e4m3_matches_torch_and_ties_go_to_even():
    import torch
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.01]).astype(np.float32)
    pos = q8._POS
    x = np.concatenate([x, ((pos[1:] + pos[:-1]) / 2).astype(np.float32), pos.astype(np.float32)])
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q8.round_e4m3(x), t)
    assert q8.round_e4m3(np.array([1000.0, -1000.0])).tolist() == [448.0, -448.0]


def test_rmsnorm_closed_forms():
    assert np.allclose(q8.rmsnorm(np.array([[3.0, -3.0, 3.0]]), eps=0.0), [[1, -1, 1]], rtol=1e-15)
    assert np.allclose(q8.rmsnorm(np.array([[3.0, 4.0]]), np.array([2.0, 1.0]), 0.0),
                       np.array([[6.0, 4.0]]) / np.sqrt(12.5), rtol=1e-15)
    x = np.random.default_rng(1).standard_normal((4, 33))
    assert np.allclose(q8.rmsnorm(x * 8, eps=64e-6), q8.rmsnorm(x, eps=1e-6), rtol=1e-14)   # scale invariance
    assert np.isnan(q8.rmsnorm(np.array([[np.inf, 1.0]]))).all()


@pytest.mark.parametrize("gamma", [False, True])
def test_rmsnorm_gradients_match_differences(gamma):
    rng = np.random.default_rng(2)
    h, dy, dres = (rng.standard_normal((3, 7)) for _ in range(3))
    g = rng.standard_normal(7) if gamma else None
    dx, dg = q8.rmsnorm_backward(dy, h, g, 1e-3, dres)
    loss = lambda h, g: np.sum(q8.rmsnorm(h, g, 1e-3) * dy) + np.sum(h * dres)  # noqa: E731
    step = 1e-6
    for i in range(3):
        for j in range(7):
            d = np.zeros_like(h)
            d[i, j] = step
            assert abs((loss(h + d, g) - loss(h - d, g)) / (2 * step) - dx[i, j]) < 1e-8
    base = np.ones(7) if g is None else g
    for j in range(7):
        d = np.zeros(7)
        d[j] = step
        assert abs((loss(h, base + d) - loss(h, base - d)) / (2 * step) - dg[j]) < 1e-8


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_quantize_rows(kind):
    rng = np.random.default_rng(3)
    v = rng.standard_normal((5, 64))
    v[1] = 0.0
    v[2, 3] = np.nan
    v[3, 0] = -100.0
    t, s = q8.quantize(v, kind)
    assert np.all(t[1] == 0) and s[1] == q8.TINY / q8.QMAX[kind]
    assert np.isnan(s[2]) and np.all(t[2] == 0)
    assert np.isclose(t[3, 0], -q8.QMAX[kind], rtol=1e-15)
    c = q8.round_codes(t, kind)
    ok = [0, 1, 3, 4]
    step = 1.0 if kind == "i8" else 32.0
    assert np.max(np.abs(c[ok] - t[ok])) <= step / 2
    assert q8.round_codes(np.array([0.5, 1.5, 2.5, -0.5]), "i8").tolist() == [0, 2, 2, 0]


def test_matmul_against_integers():
    rng = np.random.default_rng(4)
    a, b = rng.integers(-128, 128, (3, 50)), rng.integers(-128, 128, (4, 50))
    sa, sb, bias = rng.uniform(0.1, 1, 3), rng.uniform(0.1, 1, 4), rng.standard_normal(4)
    c, mag = q8.matmul(a, b, sa, sb, bias)
    for i in range(3):
        for j in range(4):
            acc = sum(int(x) * int(y) for x, y in zip(a[i], b[j]))
            assert np.isclose(c[i, j], acc * sa[i] * sb[j] + bias[j], rtol=1e-14)
    assert np.all(mag >= np.abs(c) - 1e-9)
