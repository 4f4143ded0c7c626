"""What the calls of the 8-bit layer allocate: a workspace only where kernels
of that call use one.  Counted on captured calls, where each allocation is a
node of the graph."""
import pytest

pytestmark = pytest.mark.gpu

KERNEL, ALLOC, FREE = 0, 10, 11   # cudaGraphNodeType


def nodes(torch, call):
    """Numbers of (kernel, allocation, free) nodes that a call adds to a graph."""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.12")
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    raw = ctypes.c_void_p(g.raw_cuda_graph())
    n = ctypes.c_size_t(0)
    assert rt.cudaGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    arr = (ctypes.c_void_p * max(n.value, 1))()
    assert rt.cudaGraphGetNodes(raw, arr, ctypes.byref(n)) == 0
    kinds = []
    for i in range(n.value):
        t = ctypes.c_int(-1)
        assert rt.cudaGraphNodeGetType(ctypes.c_void_p(arr[i]), ctypes.byref(t)) == 0
        kinds.append(t.value)
    return kinds.count(KERNEL), kinds.count(ALLOC), kinds.count(FREE)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(40, 64), (300, 1000), (50, 4096), (9, 4095), (5, 40000), (3, 70000)])
def test_gradients(fk, cuda_device, rows, cols, dtype):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    h, dy, dx = (torch.randn(rows, cols, device="cuda").to(dt) for _ in range(3))
    w, dw = torch.ones(cols + 1, device="cuda"), torch.empty(cols, device="cuda")
    streamed = cols > 65536
    # without dgamma one kernel, and no workspace; value by value two kernels and the rows' statistics
    call = lambda w: fk.rmsnorm_backward(dy, h, w, out=dx, need_dweight=False)  # noqa: E731
    assert nodes(torch, lambda: call(w[:cols])) == ((2, 1, 1) if streamed else (1, 0, 0))
    assert nodes(torch, lambda: call(w[1:])) == (2, 1, 1)
    # with it the partial sums and the step that adds them
    assert nodes(torch, lambda: fk.rmsnorm_backward(dy, h, w[:cols], out=dx, dweight=dw)) == \
        ((4, 1, 1) if streamed else (2, 1, 1))


def test_products(fk, cuda_device):
    import torch
    for m, n, k in ((1, 256, 512), (100, 256, 512), (5, 64, 1001)):
        a = torch.zeros(m, k, dtype=torch.int8, device="cuda")
        b = torch.zeros(n, k, dtype=torch.int8, device="cuda")
        sa, sb, c = torch.ones(m, device="cuda"), torch.ones(n, device="cuda"), torch.empty(m, n, device="cuda")
        got = nodes(torch, lambda: fk.matmul_q8(a, sa, b, sb, out=c))
        assert got == ((1, 0, 0) if k % 16 == 0 else (2, 1, 1))
