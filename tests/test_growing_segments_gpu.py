"""Tensors of an allocator that grows its segments in place (virtual memory
mapped piece by piece, PYTORCH_CUDA_ALLOC_CONF=expandable_segments:True): a
tensor over several pieces is taken whole, and a span that reaches past what is
mapped is refused on the host, though its reservation goes on."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
import memory_bound_fk_b200 as fk
BAD = fk.FK_ERR_INVALID_ARG
s = torch.cuda.current_stream().cuda_stream
x = torch.randn(30000, 1024, device="cuda")                  # 123 MB: seven pieces of 20
b = x.bfloat16()
part = slice(29000, 30000)
for f in (fk.softmax_rows, fk.gelu, fk.layernorm, fk.rmsnorm, lambda t: fk.quantize_rows(t)[0],
          lambda t: fk.rmsnorm(t, residual=t)[0], lambda t: fk.rmsnorm_backward(t, t)[0]):
    for t in (x, b):
        assert torch.equal(f(t)[part], f(t[part].clone()))
w, ws = fk.quantize_rows(x)
a, sa = fk.quantize_rows(x[:4].clone())
assert torch.equal(fk.matmul_q8(a, sa, w, ws)[:, part], fk.matmul_q8(a, sa, w[part].clone(), ws[part].clone()))
q = torch.randn(8, 8192, 128, device="cuda", dtype=torch.bfloat16)
one = q[7:].clone()
assert (fk.attention(q, q, q)[7].float() - fk.attention(one, one, one)[0].float()).abs().max() < 2.0 ** -5   # two roundings of |o| < 8
torch.cuda.synchronize()
# rows that would reach 100 GB past the tensor: nothing is launched
rows, cols, p = 25_000_000, 1024, x.data_ptr()
o = torch.empty(64, device="cuda").data_ptr()
assert fk.fk_rmsnorm_rows(p, 0, 0, p, 0, 0, rows, cols, fk.FK_F32, fk.FK_F32, 1e-6, s) == BAD
assert fk.fk_softmax_rows(p, p, rows, cols, fk.FK_F32, s) == BAD
assert fk.fk_gelu_tanh(p, p, rows * cols, s) == BAD
assert fk.fk_matmul_q8(w.data_ptr(), w.data_ptr(), o, o, 0, p, 1, 1, 1 << 30, fk.FK_E4M3, fk.FK_F32, 0, s) == BAD
torch.cuda.synchronize()
print("whole")
"""


@pytest.mark.parametrize("conf", ["expandable_segments:True", "backend:cudaMallocAsync", "expandable_segments:False"])
def test_tensors_over_several_pieces(fk, cuda_device, conf):
    env = {**os.environ, "PYTHONPATH": ROOT, "PYTORCH_CUDA_ALLOC_CONF": conf}
    p = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "whole" in p.stdout, p.stderr[-2000:]
