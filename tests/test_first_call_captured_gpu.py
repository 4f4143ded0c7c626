"""A process whose first call of the library stands in a stream capture: what
the library sets up once must not end the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import torch
import memory_bound_fk_b200 as fk
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, generator=g, device="cuda")
q = lambda *s: torch.randint(-9, 10, s, generator=g, device="cuda").to(torch.int8)
"""
RUN = """
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
want = call()
assert all(torch.equal(a, b) for a, b in zip(out, want)), "replay differs"
assert fk.fk_wait_timeouts() == 0
print("captured")
"""
CALLS = {
    # a workspace from the library's pool each
    "product_k_odd": "a, b, one = q(5, 1001), q(300, 1001), torch.ones(300, device='cuda')\n"
                     "call = lambda: (fk.matmul_q8(a, one[:5].contiguous(), b, one),)\n",
    "gradients": "h, d = r(100, 1500), r(100, 1500)\ncall = lambda: fk.rmsnorm_backward(d, h)\n",
    "softmax_split": "x = r(2, 3000001)\ncall = lambda: (fk.softmax_rows(x),)\n",
    # none
    "product": "a, b, one = q(500, 512), q(300, 512), torch.ones(500, device='cuda')\n"
               "call = lambda: (fk.matmul_q8(a, one, b, one[:300].contiguous()),)\n",
    "norm_and_codes": "x = r(40, 4096)\n"
                      "call = lambda: (*[t.float() for t in fk.rmsnorm(x, residual=x, out_dtype=torch.int8)],\n"
                      "                *[t.float() for t in fk.quantize_rows(x, gelu='tanh')])\n",
}


@pytest.mark.parametrize("name", CALLS)
def test_first_call_in_a_capture(fk, cuda_device, name):
    env = {**os.environ, "PYTHONPATH": ROOT}
    p = subprocess.run([sys.executable, "-c", SETUP + CALLS[name] + RUN], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=120)
    assert p.returncode == 0 and "captured" in p.stdout, p.stderr[-2000:]
