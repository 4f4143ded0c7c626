"""Calls of several streams at once: kernels with tensor memory and clusters
beside each other and beside the row kernels and attention give the bits that
they give alone, and no wait gives up.  (Attention without a mask adds the two
halves of a split unit in the order in which they finish, alone too: it is held
to one rounding of bf16, 2^-7 relative, and fp32's of its sums.)"""
import pytest

from _q8util import make_rows

pytestmark = pytest.mark.gpu


def test_operators_of_four_streams(fk, cuda_device):
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q8 = lambda *s: fk.quantize_rows(r(*s))  # noqa: E731

    def product(m, n, k, **kw):
        (a, sa), (b, sb) = q8(m, k), q8(n, k)
        return lambda: fk.matmul_q8(a, sa, b, sb, **kw)

    def attend(d, causal):
        q = r(24, 512, d).bfloat16()
        return lambda: fk.attention(q, q, q, causal=causal)

    x, y = make_rows(2000, 4096, "bf16", 1).cuda(), make_rows(400, 16384, "bf16", 2).cuda()
    z = make_rows(40, 40000, "bf16", 3).cuda()
    streams = [
        [product(1, 4096, 4096), product(1000, 4096, 1024, gelu="tanh"), attend(64, False), product(300, 700, 4096)],
        [product(509, 4096, 2048), product(64, 8192, 1024), product(16, 300, 16384), attend(128, True)],
        [attend(64, True), product(5, 512, 1001), product(256, 1000, 1024, out_dtype=torch.float32), product(40, 9000, 512)],
        [lambda: fk.rmsnorm(x, residual=x, out_dtype=torch.int8)[0], lambda: fk.quantize_rows(y, gelu="erf")[0],
         lambda: fk.rmsnorm_backward(x, x)[0], lambda: fk.rmsnorm(z), product(768, 1024, 2048), product(2, 640, 8192)],
    ]
    want = [[c().clone() for c in calls] for calls in streams]
    torch.cuda.synchronize()
    fk.fk_wait_timeouts(reset=True)
    cuda = [torch.cuda.Stream() for _ in streams]
    got = [[] for _ in streams]
    for turn in range(25):
        for s, calls, out in zip(cuda, streams, got):
            with torch.cuda.stream(s):
                for i in range(len(calls)):
                    out.append((i + turn) % len(calls))
                    out.append(calls[(i + turn) % len(calls)]())
    torch.cuda.synchronize()
    assert fk.fk_wait_timeouts() == 0
    for out, ref in zip(got, want):
        for i, t in zip(out[::2], out[1::2]):
            if t.dim() == 3 and t.shape[2] == 64:
                a, b = t.float(), ref[i].float()
                assert bool(((a - b).abs() <= b.abs() * 2.0 ** -7 + 2.0 ** -20).all())
            else:
                assert torch.equal(t.view(torch.uint8), ref[i].view(torch.uint8))
