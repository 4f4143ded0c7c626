"""A wait for a finished product that gives up leaves C unwritten: the
self-test makes these waits run out at once (nothing else is disturbed: loads
and MMAs run on to their end), in every kernel of the product."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

# up to 64 tokens: 1, 2, 4 and 8 blocks to a tile; more: pairs of SMs with one tile each and with two, then two and
# four pairs to a tile, of 128 and 256 tokens; operands copied first
SHAPES = [(1, 19200, 256), (16, 9500, 512), (30, 4700, 1024), (64, 300, 4096), (3, 300, 4096), (300, 512, 128),
          (129, 9000, 1024), (1030, 520, 144), (1000, 4096, 640), (1500, 5000, 640), (256, 4096, 4096), (509, 4096, 4096),
          (100, 1024, 1024), (768, 1024, 8192), (300, 512, 1001), (5, 512, 1001)]


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_c_is_left_when_the_wait_for_it_gives_up(fk, cuda_device, m, n, k, kind):
    import torch
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    a = torch.randint(-20, 21, (m, k), generator=g, device="cuda").to(torch.int8)
    b = torch.randint(-20, 21, (n, k), generator=g, device="cuda").to(torch.int8)
    if kind == "e4m3":
        a, b = (t.float().clamp(-16, 16).to(torch.float8_e4m3fn) for t in (a, b))
    sa, sb = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    c = torch.full((m, n), 7.5, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    fk.fk_wait_timeouts(reset=True)
    st = fk.fk_matmul_q8_wait_selftest(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), c.data_ptr(), m, n, k,
                                       fk.FK_I8 if kind == "i8" else fk.FK_E4M3, s)
    assert st == fk.FK_OK
    torch.cuda.synchronize()
    assert fk.fk_wait_timeouts(reset=True) > 0
    assert bool((c == 7.5).all()), "a block that gave up wrote C"
    # the next call is whole: integers below 2^24 come out exactly
    got = fk.matmul_q8(a, sa, b, sb, out_dtype=torch.float32, out=c)
    rows = np.unique(np.linspace(0, m - 1, 5).astype(int))
    assert torch.equal(got[rows].double(), a[rows].double() @ b.double().T)
    assert fk.fk_wait_timeouts() == 0
