"""fk_matmul_q8 on every cut of a product for more than 64 tokens, each over
several steps of k, in both types, with and without bias and GELU: pairs of
SMs that walk two and more tiles (stages and accumulators running on from
tile to tile), and two or four pairs to a tile.

Held to sums in double on the device; bounds as in test_matmul_q8_gpu: the
sum's conversion, two scales and bias round to 4 u of the sum of magnitudes,
e4m3 sums lose at most (k / 32 + 8) 2^-22 of it, GELU carries these through
its slope and adds its own 2e-6, and the output is rounded once."""
import math

import pytest

from _q8util import DENORMAL, EPS_HALF, GELU_ABS, GELU_SLOPE, U

pytestmark = pytest.mark.gpu

# 256 tokens a tile: 120 tiles, 432, 711 on 74 pairs; 128 tokens: 79 and 157 tiles; k over two pairs (tiles of 256 and
# 128), over four, ragged each
SHAPES = [(1500, 5000, 640), (3001, 8999, 592), (2100, 20001, 144), (97, 20000, 1040), (100, 40000, 640),
          (509, 4096, 4096), (300, 3000, 2048), (510, 2100, 4080), (256, 4096, 4096), (385, 1100, 16384),
          (768, 1024, 8192), (512, 900, 6000), (700, 1000, 4096), (100, 1024, 1024), (66, 130, 4096), (1000, 300, 2000)]


def gelu64(torch, v, kind):
    if kind == "tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v * 0.5 * torch.special.erfc(-v / math.sqrt(2)) if kind == "erf" else v


@pytest.mark.parametrize("out,gelu,bias", [("f32", None, False), ("bf16", None, True), ("bf16", "tanh", True),
                                           ("f32", "erf", True)])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_cuts(fk, cuda_device, m, n, k, kind, out, gelu, bias):
    import torch
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q = lambda t: (t * 30).round().clamp(-127, 127).to(torch.int8) if kind == "i8" else (t * 100).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    a, b = q(r(m, k)), q(r(n, k))
    unit = (30 if kind == "i8" else 100) ** 2 * math.sqrt(k)
    sa, sb = torch.exp(0.5 * r(m)), torch.exp(0.5 * r(n)) / unit
    bs = 0.1 * r(n) if bias else None
    odt = torch.float32 if out == "f32" else torch.bfloat16
    want = torch.full((m + 3, n), 7.5, device="cuda", dtype=odt)
    got = fk.matmul_q8(a, sa, b, sb, bias=bs, gelu=gelu, out=want[:m])
    s = sa.double()[:, None] * sb.double()
    ref, mag = (a.double() @ b.double().T) * s, (a.double().abs() @ b.double().abs().T) * s
    if bias:
        ref, mag = ref + bs.double(), mag + bs.double().abs()
    extra = (4 * U if kind == "i8" else (k / 32 + 8) * 2.0 ** -22 + 4 * U) * mag
    if gelu:
        ref, extra = gelu64(torch, ref, gelu), GELU_SLOPE * extra + GELU_ABS
    bound = ref.abs() * ((1 + U) * EPS_HALF[out] + U) + DENORMAL[out] + extra
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), f"{float((err / bound).max()):.2f} x the bound"
    assert bool((want[m:] == 7.5).all()) and fk.fk_wait_timeouts() == 0
    # equal calls, equal bits
    assert torch.equal(got, fk.matmul_q8(a, sa, b, sb, bias=bs, gelu=gelu, out_dtype=odt))
