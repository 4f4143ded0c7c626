"""Chains of the 8-bit layer over one set of buffers: each kernel may start
before its predecessor has ended, and reads what the predecessor writes into
places that earlier kernels of the chain have read too."""
import numpy as np
import pytest

from _q8util import make_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("rows", [1, 5, 40, 100, 300])
@pytest.mark.parametrize("hid,mid", [(256, 640), (1024, 2048), (500, 264)])
def test_codes_and_scales_rewritten_between_products(fk, cuda_device, rows, hid, mid, kind):
    import torch
    dt = torch.int8 if kind == "i8" else torch.float8_e4m3fn
    steps = 6
    w, ws = fk.quantize_rows(make_rows(mid, hid, "f32", 1, 0.1).cuda(), dt)
    gamma = torch.from_numpy((1 + 0.2 * np.random.default_rng(0).standard_normal(hid)).astype(np.float32)).cuda()
    xs = [make_rows(rows, hid, "bf16", 10 + i, 1.0).cuda() for i in range(steps)]
    ys = [make_rows(rows, mid, "bf16", 30 + i, 1.0).cuda() for i in range(steps)]

    def chain(buffers):
        out = []
        stream = torch.zeros(rows, hid, dtype=torch.bfloat16, device="cuda")
        for x, y in zip(xs, ys):
            a, sa, c, sc, u = buffers()
            fk.rmsnorm(x, gamma, residual=stream, residual_out=stream, out_dtype=dt, out=a, scales=sa)
            fk.matmul_q8(a, sa, w, ws, out=u)
            # the product's buffer is read again, and codes and scales are written over those of the step before
            fk.quantize_rows(u, dt, gelu="tanh", out=c, scales=sc)
            out.append((u.clone(), c.clone(), sc.clone()))
            fk.quantize_rows(y, dt, out=c, scales=sc)
            out.append((c.clone(), sc.clone()))
        return out + [(stream,)]

    def fresh():
        e = lambda *s, t=dt: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        return (e(rows, hid), e(rows, t=torch.float32), e(rows, mid), e(rows, t=torch.float32),
                e(rows, mid, t=torch.bfloat16))

    one = fresh()
    want = chain(fresh)
    got = chain(lambda: one)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = chain(lambda: one)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for other in (got, captured):
        for p, q in zip(want, other):
            assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(p, q))
