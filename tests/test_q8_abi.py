"""The C ABI of the 8-bit linear layer without a GPU: refusals that come
before the device is looked at, no-ops, and workspace sizes."""
import pytest

X, Y, Z, S, W = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000   # addresses that are never dereferenced


def rms(fk, x=X, r=0, g=0, y=Y, s=0, h=0, rows=8, cols=64, dt=0, out=0, eps=1e-6):
    return fk.fk_rmsnorm_rows(x, r, g, y, s, h, rows, cols, dt, out, eps)


def bwd(fk, dy=X, h=Z, g=0, dres=0, dx=Y, dw=0, rows=8, cols=64, dt=0, eps=1e-6):
    return fk.fk_rmsnorm_rows_bwd(dy, h, g, dres, dx, dw, rows, cols, dt, eps)


def qnt(fk, x=X, q=Y, s=S, rows=8, cols=64, dt=0, out=2, epi=0):
    return fk.fk_quantize_rows(x, q, s, rows, cols, dt, out, epi)


def mm(fk, a=X, b=Y, sa=S, sb=S + 4096, bias=0, c=Z, m=8, n=64, k=64, dt=2, out=0, epi=0):
    return fk.fk_matmul_q8(a, b, sa, sb, bias, c, m, n, k, dt, out, epi)


def test_dtypes(fk):
    bad = fk.FK_ERR_UNSUPPORTED_DTYPE
    assert rms(fk, dt=2) == bad and rms(fk, dt=0, out=1) == bad and rms(fk, out=4, s=S) == bad
    assert bwd(fk, dt=2) == bad and bwd(fk, dt=-1) == bad
    assert qnt(fk, out=0) == bad and qnt(fk, dt=3) == bad
    assert mm(fk, dt=0) == bad and mm(fk, out=2) == bad
    # the other entry points do not take the 8-bit types
    assert fk.fk_softmax_rows(X, Y, 1, 1, fk.FK_I8) == bad
    assert fk.fk_gelu(X, Y, 1, fk.FK_E4M3, 0) == bad
    assert fk.fk_layernorm_rows(X, Y, 0, 0, 1, 1, fk.FK_I8, 0.0) == bad


def test_zero_sizes_are_noops(fk):
    assert rms(fk, x=0, y=0, rows=0) == 0 and rms(fk, x=0, y=0, cols=0) == 0
    assert bwd(fk, dy=0, h=0, dx=0, rows=0) == 0 and bwd(fk, dy=0, h=0, dx=0, cols=0) == 0
    assert qnt(fk, x=0, q=0, s=0, rows=0) == 0
    assert mm(fk, a=0, b=0, c=0, m=0) == 0 and mm(fk, a=0, b=0, c=0, n=0) == 0


def test_nulls_and_scalars(fk):
    bad = fk.FK_ERR_INVALID_ARG
    assert rms(fk, x=0) == bad and rms(fk, y=0) == bad
    assert rms(fk, eps=-1.0) == bad and rms(fk, eps=float("nan")) == bad and rms(fk, eps=float("inf")) == bad
    assert rms(fk, out=2) == bad                # 8-bit rows need scales
    assert rms(fk, s=S) == bad                  # and others have none
    assert rms(fk, h=Z) == bad                  # h without a residual
    assert bwd(fk, dy=0) == bad and bwd(fk, h=0) == bad and bwd(fk, dx=0) == bad and bwd(fk, eps=-1.0) == bad
    assert qnt(fk, x=0) == bad and qnt(fk, q=0) == bad and qnt(fk, s=0) == bad and qnt(fk, epi=3) == bad
    for name in ("a", "b", "sa", "sb", "c"):
        assert mm(fk, **{name: 0}) == bad
    assert mm(fk, epi=-1) == bad and mm(fk, k=0) == bad
    assert mm(fk, k=131072) == bad              # int8 sums could overflow
    assert mm(fk, m=1 << 31) == bad and mm(fk, n=1 << 31) == bad and mm(fk, dt=3, k=1 << 31) == bad


def test_alignment_and_size_overflow(fk):
    bad = fk.FK_ERR_INVALID_ARG
    assert rms(fk, x=X + 2) == bad and rms(fk, y=Y + 1) == bad and rms(fk, g=Z + 2) == bad
    assert rms(fk, out=2, s=S + 2) == bad and rms(fk, dt=1, out=1, r=Z + 1) == bad
    assert bwd(fk, dw=W + 2) == bad and bwd(fk, dt=1, dres=W + 1) == bad
    assert qnt(fk, s=S + 1) == bad and mm(fk, sa=S + 2) == bad and mm(fk, out=1, c=Z + 1) == bad
    big = 1 << 62
    assert rms(fk, rows=big, cols=4) == bad and bwd(fk, rows=big, cols=4) == bad and qnt(fk, rows=big, cols=8) == bad


def test_overlap(fk):
    bad, dev = fk.FK_ERR_INVALID_ARG, fk.FK_ERR_UNSUPPORTED_DEVICE
    n = 8 * 64 * 4
    assert rms(fk, y=X + 4) == bad and rms(fk, y=X, out=2, s=S) == bad and rms(fk, r=Z, h=Z + 4) == bad
    assert rms(fk, r=Z, h=Y) == bad and rms(fk, r=Z, y=X, h=X) == bad        # two outputs in one place
    assert rms(fk, g=Y + n - 4) == bad and rms(fk, out=3, s=X) == bad and rms(fk, out=3, s=Y) == bad
    assert rms(fk, r=Z, h=W, g=W + 64) == bad
    assert bwd(fk, dx=X + 4) == bad and bwd(fk, dx=Z + n - 4) == bad and bwd(fk, g=Y + 4) == bad
    assert bwd(fk, dw=X) == bad and bwd(fk, dw=Y) == bad and bwd(fk, g=W, dw=W) == bad
    assert qnt(fk, q=X) == bad and qnt(fk, s=X) == bad and qnt(fk, s=Y) == bad
    assert mm(fk, c=X) == bad and mm(fk, c=Y + 64) == bad and mm(fk, bias=Z) == bad and mm(fk, c=S) == bad
    # allowed in place: these get as far as the memory (or the device) check
    for st in (rms(fk, y=X), rms(fk, r=Z, y=Z), rms(fk, r=Z, h=X), rms(fk, r=Z, h=Z), bwd(fk, dx=X), bwd(fk, dx=Z),
               bwd(fk, dres=W, dx=W)):
        assert st in (bad, dev)


def test_looks_valid_but_is_not_device_memory(fk):
    ok = (fk.FK_ERR_INVALID_ARG, fk.FK_ERR_UNSUPPORTED_DEVICE)
    assert rms(fk) in ok and bwd(fk) in ok and qnt(fk) in ok and mm(fk) in ok


def test_workspaces(fk):
    assert fk.fk_rmsnorm_rows_bwd_workspace(0, 64, 0) == 0
    for rows, cols in ((1, 1), (100, 4096), (16384, 4096), (64, 40000)):
        w = fk.fk_rmsnorm_rows_bwd_workspace(rows, cols, 1)
        assert w >= cols * 4 and w >= fk.fk_rmsnorm_rows_bwd_workspace(rows, cols, 1, False)
    with pytest.raises(fk.FkError):
        fk.fk_rmsnorm_rows_bwd_workspace(4, 4, 2)
    assert fk.fk_matmul_q8_workspace(100, 100, 64) == 0
    assert fk.fk_matmul_q8_workspace(0, 100, 63) == 0
    with pytest.raises(fk.FkError):
        fk.fk_matmul_q8_workspace(1, 1, 0)


def test_headers_and_binding_agree(fk):
    names = fk.header_functions()
    for n in ("fk_rmsnorm_rows", "fk_rmsnorm_rows_bwd", "fk_rmsnorm_rows_bwd_ws", "fk_rmsnorm_rows_bwd_workspace",
              "fk_quantize_rows", "fk_matmul_q8", "fk_matmul_q8_ws", "fk_matmul_q8_workspace"):
        assert n in names and hasattr(fk, n)


def test_helpers_refuse_what_is_not_a_cuda_tensor(fk):
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        fk.rmsnorm(x)
    with pytest.raises(TypeError):
        fk.rmsnorm_backward(x, x)
    with pytest.raises(TypeError):
        fk.quantize_rows(x)
    with pytest.raises(TypeError):
        fk.matmul_q8(x, x, x, x)
