"""memory_bound_fk_b200 -- fused memory-bound operators for NVIDIA B200 (sm_100a).

Python binding of ``libfk.so`` (declared in ``include/fk.h`` and
``include/fk_q8.h``).  This module only marshals arguments: every step of the computation runs in the
library's CUDA kernels.  PyTorch provides device memory and streams.

Raw C-ABI mirrors (same names, pointers as integers, stream as a
``cudaStream_t`` integer):
    fk_gelu_tanh(x, y, n, stream) -> status
    fk_gelu(x, y, n, dtype, kind, stream) -> status
    fk_copy(src, dst, bytes, stream) -> status     (bandwidth reference)
    fk_softmax_rows(x, y, rows, cols, dtype, stream) -> status
    fk_softmax_rows_ex(x, y, rows, cols, dtype, plan, stream) -> status
    fk_softmax_rows_plan(rows, cols, dtype, path=FK_PATH_AUTO) -> SoftmaxPlan
    fk_softmax_rows_workspace(rows, cols, dtype, plan=None) -> bytes
    fk_softmax_rows_ws(x, y, rows, cols, dtype, plan, workspace, workspace_bytes, stream) -> status
    fk_softmax_rows_causal(x, y, rows, cols, dtype, scale, period, offset, stream) -> status
    fk_softmax_rows_causal_ex(x, y, rows, cols, dtype, scale, period, offset, flags, plan, stream) -> status
    fk_layernorm_rows(x, y, gamma, beta, rows, cols, dtype, eps, epilogue, stream) -> status
    fk_layernorm_rows_ex(x, y, gamma, beta, rows, cols, dtype, eps, epilogue, plan, stream) -> status
    fk_layernorm_rows_plan(rows, cols, dtype, path=FK_PATH_AUTO) -> SoftmaxPlan
    fk_attention_fwd(q, k, v, o, bh, t, d, causal, scale, stream) -> status
    fk_rmsnorm_rows(x, residual, gamma, y, scales, h, rows, cols, dtype, out_dtype, eps, stream) -> status
    fk_rmsnorm_rows_bwd(dy, h, gamma, dres, dx, dgamma, rows, cols, dtype, eps, stream) -> status
    fk_rmsnorm_rows_bwd_workspace(rows, cols, dtype, want_dgamma) -> bytes
    fk_rmsnorm_rows_bwd_ws(..., eps, workspace, workspace_bytes, stream) -> status
    fk_quantize_rows(x, q, scales, rows, cols, dtype, out_dtype, epilogue, stream) -> status
    fk_matmul_q8(a, b, a_scales, b_scales, bias, c, m, n, k, dtype, out_dtype, epilogue, stream) -> status
    fk_matmul_q8_workspace(m, n, k, aligned) -> bytes
    fk_matmul_q8_ws(..., epilogue, workspace, workspace_bytes, stream) -> status
    fk_matmul_q8_wait_selftest(a, b, a_scales, b_scales, c, m, n, k, dtype, stream) -> status
    fk_status_string(status) -> str
    fk_wait_timeouts(reset=False) -> int     (bounded-wait give-ups, synchronous)
    fk_wait_selftest(timeout_us, stream) -> status

Tensor conveniences (contiguous CUDA tensors; the current torch stream):
    gelu_tanh(x, out=None)
    gelu(x, out=None, approximate="tanh")   # fp32 / bf16; "tanh" or "none" (exact)
    softmax_rows(x, out=None, plan=None)    # softmax over the last dimension
    softmax_causal(x, scale, period=None, offset=0, out=None, plan=None)
    layernorm(x, eps=1e-5, weight=None, bias=None, gelu=None, out=None, plan=None)
    attention(q, k, v, causal=True, scale=None, out=None)   # [..., t, d] bf16
    rmsnorm(x, weight=None, eps=1e-6, residual=None, out_dtype=None, ...)   # + residual, to 8 bits or not
    rmsnorm_backward(dy, h, weight=None, eps=1e-6, dresidual=None, ...) -> (dx, dweight)
    quantize_rows(x, dtype=torch.int8, gelu=None, ...) -> (codes, scales)
    matmul_q8(a, a_scales, b, b_scales, bias=None, gelu=None, out_dtype=torch.bfloat16, ...)

There is no fallback: if the library is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfk.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "fk.h")
Q8_HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "fk_q8.h")

# fk_status
FK_OK = 0
FK_ERR_INVALID_ARG = 1
FK_ERR_UNSUPPORTED_DTYPE = 2
FK_ERR_UNSUPPORTED_DEVICE = 3
FK_ERR_CUDA = 4
# fk_dtype
FK_F32 = 0
FK_BF16 = 1
# fk_q8type
FK_I8 = 2
FK_E4M3 = 3
# fk_gelu_kind
FK_GELU_TANH = 0
FK_GELU_ERF = 1
# fk_softmax_rows_causal_ex flags
FK_SOFTMAX_SKIP_MASKED = 1
# fk_epilogue
FK_EPILOGUE_NONE = 0
FK_EPILOGUE_GELU_TANH = 1
FK_EPILOGUE_GELU_ERF = 2
# fk_softmax_path
FK_PATH_AUTO = 0
FK_PATH_WARP = 1
FK_PATH_CTA = 2
FK_PATH_CLUSTER = 3
FK_PATH_TWOPHASE = 4
FK_PATH_SPLIT = 5
PATH_NAMES = {FK_PATH_WARP: "warp", FK_PATH_CTA: "cta", FK_PATH_CLUSTER: "cluster",
              FK_PATH_TWOPHASE: "twophase", FK_PATH_SPLIT: "split"}


class FkError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {fk_status_string(status)}"
                         + (f" (cudaError {fk_last_cuda_error()})" if status == FK_ERR_CUDA else ""))


class SoftmaxPlan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("threads", ctypes.c_int),
                ("vpt", ctypes.c_int), ("cluster", ctypes.c_int), ("chunks", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {"path": PATH_NAMES.get(self.path, self.path), "threads": self.threads,
                "vpt": self.vpt, "cluster": self.cluster, "chunks": self.chunks}

    def __repr__(self) -> str:
        return f"SoftmaxPlan({self.as_dict()})"


_lib = None


def lib() -> ctypes.CDLL:
    """Load libfk.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libfk.so not found at {LIB_PATH}; build it with "
                              "`python -m memory_bound_fk_b200.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.fk_gelu_tanh.argtypes = [vp, vp, sz, vp]
        L.fk_gelu_tanh.restype = ci
        L.fk_copy.argtypes = [vp, vp, sz, vp]
        L.fk_copy.restype = ci
        L.fk_gelu.argtypes = [vp, vp, sz, ci, ci, vp]
        L.fk_gelu.restype = ci
        L.fk_softmax_rows.argtypes = [vp, vp, sz, sz, ci, vp]
        L.fk_softmax_rows.restype = ci
        L.fk_softmax_rows_ex.argtypes = [vp, vp, sz, sz, ci, ctypes.POINTER(SoftmaxPlan), vp]
        L.fk_softmax_rows_ex.restype = ci
        L.fk_softmax_rows_plan.argtypes = [sz, sz, ci, ci, ctypes.POINTER(SoftmaxPlan)]
        L.fk_softmax_rows_plan.restype = ci
        L.fk_status_string.argtypes = [ci]
        L.fk_status_string.restype = ctypes.c_char_p
        L.fk_last_cuda_error.argtypes = []
        L.fk_last_cuda_error.restype = ci
        L.fk_version.argtypes = []
        L.fk_version.restype = ci
        L.fk_softmax_rows_workspace.argtypes = [sz, sz, ci, ctypes.POINTER(SoftmaxPlan),
                                                ctypes.POINTER(ctypes.c_size_t)]
        L.fk_softmax_rows_workspace.restype = ci
        L.fk_softmax_rows_ws.argtypes = [vp, vp, sz, sz, ci, ctypes.POINTER(SoftmaxPlan), vp, sz, vp]
        L.fk_softmax_rows_ws.restype = ci
        L.fk_softmax_rows_causal.argtypes = [vp, vp, sz, sz, ci, ctypes.c_float, sz, sz, vp]
        L.fk_softmax_rows_causal.restype = ci
        L.fk_softmax_rows_causal_ex.argtypes = [vp, vp, sz, sz, ci, ctypes.c_float, sz, sz, ctypes.c_uint,
                                                ctypes.POINTER(SoftmaxPlan), vp]
        L.fk_softmax_rows_causal_ex.restype = ci
        L.fk_layernorm_rows.argtypes = [vp, vp, vp, vp, sz, sz, ci, ctypes.c_float, ci, vp]
        L.fk_layernorm_rows.restype = ci
        L.fk_layernorm_rows_ex.argtypes = [vp, vp, vp, vp, sz, sz, ci, ctypes.c_float, ci,
                                           ctypes.POINTER(SoftmaxPlan), vp]
        L.fk_layernorm_rows_ex.restype = ci
        L.fk_attention_fwd.argtypes = [vp, vp, vp, vp, sz, sz, sz, ci, ctypes.c_float, vp]
        L.fk_attention_fwd.restype = ci
        L.fk_layernorm_rows_plan.argtypes = [sz, sz, ci, ci, ctypes.POINTER(SoftmaxPlan)]
        L.fk_layernorm_rows_plan.restype = ci
        f, szp = ctypes.c_float, ctypes.POINTER(ctypes.c_size_t)
        L.fk_rmsnorm_rows.argtypes = [vp, vp, vp, vp, vp, vp, sz, sz, ci, ci, f, vp]
        L.fk_rmsnorm_rows.restype = ci
        L.fk_rmsnorm_rows_bwd.argtypes = [vp, vp, vp, vp, vp, vp, sz, sz, ci, f, vp]
        L.fk_rmsnorm_rows_bwd.restype = ci
        L.fk_rmsnorm_rows_bwd_ws.argtypes = [vp, vp, vp, vp, vp, vp, sz, sz, ci, f, vp, sz, vp]
        L.fk_rmsnorm_rows_bwd_ws.restype = ci
        L.fk_rmsnorm_rows_bwd_workspace.argtypes = [sz, sz, ci, ci, szp]
        L.fk_rmsnorm_rows_bwd_workspace.restype = ci
        L.fk_quantize_rows.argtypes = [vp, vp, vp, sz, sz, ci, ci, ci, vp]
        L.fk_quantize_rows.restype = ci
        L.fk_matmul_q8.argtypes = [vp, vp, vp, vp, vp, vp, sz, sz, sz, ci, ci, ci, vp]
        L.fk_matmul_q8.restype = ci
        L.fk_matmul_q8_ws.argtypes = [vp, vp, vp, vp, vp, vp, sz, sz, sz, ci, ci, ci, vp, sz, vp]
        L.fk_matmul_q8_ws.restype = ci
        L.fk_matmul_q8_wait_selftest.argtypes = [vp, vp, vp, vp, vp, sz, sz, sz, ci, vp]
        L.fk_matmul_q8_wait_selftest.restype = ci
        L.fk_matmul_q8_workspace.argtypes = [sz, sz, sz, ci, szp]
        L.fk_matmul_q8_workspace.restype = ci
        L.fk_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint), ci]
        L.fk_wait_timeouts.restype = ci
        L.fk_wait_selftest.argtypes = [ctypes.c_uint, vp]
        L.fk_wait_selftest.restype = ci
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the entry points declared in include/fk.h and include/fk_q8.h."""
    names = []
    for path in (HEADER_PATH, Q8_HEADER_PATH):
        with open(path) as f:
            names += re.findall(r"FK_API\s+[\w\s\*]+?\b(fk_\w+)\s*\(", f.read())
    return names


# ---------------------------------------------------------------- raw mirrors

def fk_gelu_tanh(x: int, y: int, n: int, stream: int = 0) -> int:
    return lib().fk_gelu_tanh(x, y, n, stream)


def fk_copy(src: int, dst: int, nbytes: int, stream: int = 0) -> int:
    return lib().fk_copy(src, dst, nbytes, stream)


def fk_gelu(x: int, y: int, n: int, dtype: int, kind: int, stream: int = 0) -> int:
    return lib().fk_gelu(x, y, n, dtype, kind, stream)


def fk_softmax_rows(x: int, y: int, rows: int, cols: int, dtype: int, stream: int = 0) -> int:
    return lib().fk_softmax_rows(x, y, rows, cols, dtype, stream)


def fk_softmax_rows_ex(x: int, y: int, rows: int, cols: int, dtype: int,
                       plan: SoftmaxPlan | None, stream: int = 0) -> int:
    return lib().fk_softmax_rows_ex(x, y, rows, cols, dtype,
                                    ctypes.byref(plan) if plan is not None else None, stream)


def fk_softmax_rows_plan(rows: int, cols: int, dtype: int, path: int = FK_PATH_AUTO) -> SoftmaxPlan:
    p = SoftmaxPlan()
    st = lib().fk_softmax_rows_plan(rows, cols, dtype, path, ctypes.byref(p))
    if st != FK_OK:
        raise FkError(st, "fk_softmax_rows_plan")
    return p


def fk_softmax_rows_workspace(rows: int, cols: int, dtype: int, plan: SoftmaxPlan | None = None) -> int:
    """Workspace bytes a softmax call of this shape (and plan) needs."""
    b = ctypes.c_size_t(0)
    st = lib().fk_softmax_rows_workspace(rows, cols, dtype, ctypes.byref(plan) if plan is not None else None,
                                         ctypes.byref(b))
    if st != FK_OK:
        raise FkError(st, "fk_softmax_rows_workspace")
    return b.value


def fk_softmax_rows_ws(x: int, y: int, rows: int, cols: int, dtype: int, plan: SoftmaxPlan | None,
                       workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    return lib().fk_softmax_rows_ws(x, y, rows, cols, dtype, ctypes.byref(plan) if plan is not None else None,
                                    workspace, workspace_bytes, stream)


def fk_softmax_rows_causal(x: int, y: int, rows: int, cols: int, dtype: int, scale: float, period: int,
                           offset: int = 0, stream: int = 0) -> int:
    return lib().fk_softmax_rows_causal(x, y, rows, cols, dtype, scale, period, offset, stream)


def fk_softmax_rows_causal_ex(x: int, y: int, rows: int, cols: int, dtype: int, scale: float, period: int,
                              offset: int, plan: SoftmaxPlan | None, stream: int = 0, flags: int = 0) -> int:
    return lib().fk_softmax_rows_causal_ex(x, y, rows, cols, dtype, scale, period, offset, flags,
                                           ctypes.byref(plan) if plan is not None else None, stream)


def fk_layernorm_rows(x: int, y: int, gamma: int, beta: int, rows: int, cols: int, dtype: int, eps: float,
                      epilogue: int = FK_EPILOGUE_NONE, stream: int = 0) -> int:
    return lib().fk_layernorm_rows(x, y, gamma or None, beta or None, rows, cols, dtype, eps, epilogue, stream)


def fk_layernorm_rows_ex(x: int, y: int, gamma: int, beta: int, rows: int, cols: int, dtype: int, eps: float,
                         epilogue: int, plan: SoftmaxPlan | None, stream: int = 0) -> int:
    return lib().fk_layernorm_rows_ex(x, y, gamma or None, beta or None, rows, cols, dtype, eps, epilogue,
                                      ctypes.byref(plan) if plan is not None else None, stream)


def fk_layernorm_rows_plan(rows: int, cols: int, dtype: int, path: int = FK_PATH_AUTO) -> SoftmaxPlan:
    p = SoftmaxPlan()
    st = lib().fk_layernorm_rows_plan(rows, cols, dtype, path, ctypes.byref(p))
    if st != FK_OK:
        raise FkError(st, "fk_layernorm_rows_plan")
    return p


def fk_attention_fwd(q: int, k: int, v: int, o: int, bh: int, t: int, d: int, causal: int, scale: float,
                     stream: int = 0) -> int:
    return lib().fk_attention_fwd(q, k, v, o, bh, t, d, causal, scale, stream)


def fk_rmsnorm_rows(x: int, residual: int, gamma: int, y: int, scales: int, h: int, rows: int, cols: int, dtype: int,
                    out_dtype: int, eps: float, stream: int = 0) -> int:
    return lib().fk_rmsnorm_rows(x, residual, gamma, y, scales, h, rows, cols, dtype, out_dtype, eps, stream)


def fk_rmsnorm_rows_bwd(dy: int, h: int, gamma: int, dres: int, dx: int, dgamma: int, rows: int, cols: int,
                        dtype: int, eps: float, stream: int = 0) -> int:
    return lib().fk_rmsnorm_rows_bwd(dy, h, gamma, dres, dx, dgamma, rows, cols, dtype, eps, stream)


def fk_rmsnorm_rows_bwd_workspace(rows: int, cols: int, dtype: int, want_dgamma: bool = True) -> int:
    """Workspace bytes fk_rmsnorm_rows_bwd of this shape uses."""
    b = ctypes.c_size_t(0)
    st = lib().fk_rmsnorm_rows_bwd_workspace(rows, cols, dtype, int(bool(want_dgamma)), ctypes.byref(b))
    if st != FK_OK:
        raise FkError(st, "fk_rmsnorm_rows_bwd_workspace")
    return b.value


def fk_rmsnorm_rows_bwd_ws(dy: int, h: int, gamma: int, dres: int, dx: int, dgamma: int, rows: int, cols: int,
                           dtype: int, eps: float, workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    return lib().fk_rmsnorm_rows_bwd_ws(dy, h, gamma, dres, dx, dgamma, rows, cols, dtype, eps, workspace,
                                        workspace_bytes, stream)


def fk_quantize_rows(x: int, q: int, scales: int, rows: int, cols: int, dtype: int, out_dtype: int,
                     epilogue: int = FK_EPILOGUE_NONE, stream: int = 0) -> int:
    return lib().fk_quantize_rows(x, q, scales, rows, cols, dtype, out_dtype, epilogue, stream)


def fk_matmul_q8(a: int, b: int, a_scales: int, b_scales: int, bias: int, c: int, m: int, n: int, k: int, dtype: int,
                 out_dtype: int, epilogue: int = FK_EPILOGUE_NONE, stream: int = 0) -> int:
    return lib().fk_matmul_q8(a, b, a_scales, b_scales, bias, c, m, n, k, dtype, out_dtype, epilogue, stream)


def fk_matmul_q8_workspace(m: int, n: int, k: int, aligned: bool = True) -> int:
    """Workspace bytes fk_matmul_q8 uses (aligned: a and b on 16-byte boundaries)."""
    b = ctypes.c_size_t(0)
    st = lib().fk_matmul_q8_workspace(m, n, k, int(bool(aligned)), ctypes.byref(b))
    if st != FK_OK:
        raise FkError(st, "fk_matmul_q8_workspace")
    return b.value


def fk_matmul_q8_ws(a: int, b: int, a_scales: int, b_scales: int, bias: int, c: int, m: int, n: int, k: int,
                    dtype: int, out_dtype: int, epilogue: int, workspace: int, workspace_bytes: int,
                    stream: int = 0) -> int:
    return lib().fk_matmul_q8_ws(a, b, a_scales, b_scales, bias, c, m, n, k, dtype, out_dtype, epilogue, workspace,
                                 workspace_bytes, stream)


def fk_matmul_q8_wait_selftest(a: int, b: int, a_scales: int, b_scales: int, c: int, m: int, n: int, k: int,
                               dtype: int, stream: int = 0) -> int:
    return lib().fk_matmul_q8_wait_selftest(a, b, a_scales, b_scales, c, m, n, k, dtype, stream)


def fk_status_string(status: int) -> str:
    return lib().fk_status_string(status).decode()


def fk_last_cuda_error() -> int:
    return lib().fk_last_cuda_error()


def fk_version() -> int:
    return lib().fk_version()


def fk_wait_timeouts(reset: bool = False) -> int:
    """Threads whose bounded cluster wait gave up on the current device
    (synchronous).  Raises FkError on failure."""
    c = ctypes.c_uint(0)
    st = lib().fk_wait_timeouts(ctypes.byref(c), 1 if reset else 0)
    if st != FK_OK:
        raise FkError(st, "fk_wait_timeouts")
    return c.value


def fk_wait_selftest(timeout_us: int, stream: int = 0) -> int:
    return lib().fk_wait_selftest(timeout_us, stream)


def fk_softmax_rows_noalloc(x: int, y: int, rows: int, cols: int, dtype: int, stream: int = 0) -> int:
    """fk_softmax_rows that never allocates device memory (scratch is a fixed
    1 MiB array inside the library; see include/fk.h)."""
    f = lib().fk_softmax_rows_noalloc
    if f.argtypes is None:
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        f.argtypes = [vp, vp, sz, sz, ctypes.c_int, vp]
        f.restype = ctypes.c_int
    return f(x, y, rows, cols, dtype, stream)


def fk_softmax_rows_noalloc_cap(x: int, y: int, rows: int, cols: int, dtype: int, capacity_pairs: int,
                                stream: int = 0) -> int:
    """fk_softmax_rows_noalloc on the first capacity_pairs entries of the
    library's scratch array (more batches on smaller inputs)."""
    f = lib().fk_softmax_rows_noalloc_cap
    if f.argtypes is None:
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        f.argtypes = [vp, vp, sz, sz, ctypes.c_int, sz, vp]
        f.restype = ctypes.c_int
    return f(x, y, rows, cols, dtype, capacity_pairs, stream)


def make_plan(path: int, threads: int = 0, vpt: int = 0, cluster: int = 0, chunks: int = 0) -> SoftmaxPlan:
    return SoftmaxPlan(path, threads, vpt, cluster, chunks)


# ---------------------------------------------------------------- tensors

_raw_stream = None     # torch's current-stream lookup by device index, found at first use


def _stream_handle(t) -> int:
    global _raw_stream
    if _raw_stream is None:
        import torch
        # the handle itself, without building a Stream object around it
        # (2.4 us); older or newer torch may not have it under this name
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(t.get_device())


def _check_tensor(t, name: str):
    torch = _torch or _load_torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def gelu_tanh(x, out=None):
    """tanh-GELU of a contiguous fp32 CUDA tensor (``out`` may be ``x``)."""
    import torch
    _check_tensor(x, "x")
    if x.dtype != torch.float32:
        raise TypeError("gelu_tanh takes float32")
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.numel() != x.numel() or out.device != x.device:
        raise ValueError("out must match x in dtype, size and device")
    st = fk_gelu_tanh(x.data_ptr(), out.data_ptr(), x.numel(), _stream_handle(x))
    if st != FK_OK:
        raise FkError(st, "fk_gelu_tanh")
    return out


def _dtype_code(dt) -> int:
    import torch
    if dt == torch.float32:
        return FK_F32
    if dt == torch.bfloat16:
        return FK_BF16
    raise TypeError("fk operators take float32 or bfloat16")


_GELU_KINDS = {"tanh": FK_GELU_TANH, "none": FK_GELU_ERF}


def gelu(x, out=None, approximate: str = "tanh"):
    """GELU of a contiguous fp32/bf16 CUDA tensor; ``approximate`` is "tanh"
    (the tanh form) or "none" (the exact x * Phi(x)), as in torch's gelu.
    ``out`` may be ``x``."""
    import torch
    _check_tensor(x, "x")
    code = _dtype_code(x.dtype)
    if approximate not in _GELU_KINDS:
        raise ValueError("approximate must be 'tanh' or 'none'")
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.numel() != x.numel() or out.device != x.device:
        raise ValueError("out must match x in dtype, size and device")
    st = fk_gelu(x.data_ptr(), out.data_ptr(), x.numel(), code, _GELU_KINDS[approximate], _stream_handle(x))
    if st != FK_OK:
        raise FkError(st, "fk_gelu")
    return out


def softmax_rows(x, out=None, plan: SoftmaxPlan | None = None, workspace=None):
    """Softmax over the last dimension of a contiguous fp32/bf16 CUDA tensor.
    `workspace` (a CUDA tensor of at least fk_softmax_rows_workspace bytes)
    makes the call allocation-free; without it the split path allocates its
    workspace stream-ordered."""
    import torch
    _check_tensor(x, "x")
    code = _dtype_code(x.dtype)
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.shape != x.shape or out.device != x.device:
        raise ValueError("out must match x in dtype, shape and device")
    cols = x.shape[-1] if x.dim() > 0 else 1
    rows = x.numel() // cols if cols else 0
    if workspace is not None:
        _check_tensor(workspace, "workspace")
        st = fk_softmax_rows_ws(x.data_ptr(), out.data_ptr(), rows, cols, code, plan, workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream_handle(x))
    else:
        st = fk_softmax_rows_ex(x.data_ptr(), out.data_ptr(), rows, cols, code, plan, _stream_handle(x))
    if st != FK_OK:
        raise FkError(st, "fk_softmax_rows")
    return out


def softmax_causal(x, scale: float, period: int | None = None, offset: int = 0, out=None,
                   plan: SoftmaxPlan | None = None, skip_masked: bool = False):
    """Scaled, causally masked softmax over the last dimension of a
    contiguous fp32/bf16 CUDA tensor of attention scores [..., T_q, T_k]: row
    i of each [T_q, T_k] block keeps keys j <= i + offset.  `period` defaults
    to T_q (x.shape[-2]); 0 means no mask.  skip_masked: masked outputs are
    not stored (left as they were, or 0)."""
    import torch
    _check_tensor(x, "x")
    code = _dtype_code(x.dtype)
    if x.dim() < 2 and period is None:
        raise ValueError("period is needed for a 1-D tensor")
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.shape != x.shape or out.device != x.device:
        raise ValueError("out must match x in dtype, shape and device")
    cols = x.shape[-1] if x.dim() > 0 else 1
    rows = x.numel() // cols if cols else 0
    p = x.shape[-2] if period is None else period
    st = fk_softmax_rows_causal_ex(x.data_ptr(), out.data_ptr(), rows, cols, code, scale, p, offset, plan,
                                   _stream_handle(x), FK_SOFTMAX_SKIP_MASKED if skip_masked else 0)
    if st != FK_OK:
        raise FkError(st, "fk_softmax_rows_causal")
    return out


_EPILOGUES = {None: FK_EPILOGUE_NONE, "tanh": FK_EPILOGUE_GELU_TANH, "none": FK_EPILOGUE_GELU_ERF,
              "erf": FK_EPILOGUE_GELU_ERF}


def layernorm(x, eps: float = 1e-5, weight=None, bias=None, gelu: str | None = None, out=None,
              plan: SoftmaxPlan | None = None):
    """LayerNorm over the last dimension of a contiguous fp32/bf16 CUDA
    tensor (as F.layer_norm(x, x.shape[-1:], weight, bias, eps)), then GELU
    when `gelu` is "tanh" or "erf" (or torch's "none", the exact form).
    weight / bias: contiguous fp32 CUDA tensors of x.shape[-1] values."""
    import torch
    _check_tensor(x, "x")
    code = _dtype_code(x.dtype)
    if gelu not in _EPILOGUES:
        raise ValueError("gelu must be None, 'tanh' or 'erf'")
    cols = x.shape[-1] if x.dim() > 0 else 1
    rows = x.numel() // cols if cols else 0
    ptrs = []
    for name, p in (("weight", weight), ("bias", bias)):
        if p is None:
            ptrs.append(0)
            continue
        _check_tensor(p, name)
        if p.dtype != torch.float32 or p.numel() != cols or p.device != x.device:
            raise ValueError(f"{name} must be float32 with x.shape[-1] values on x's device")
        ptrs.append(p.data_ptr())
    if out is None:
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.dtype != x.dtype or out.shape != x.shape or out.device != x.device:
        raise ValueError("out must match x in dtype, shape and device")
    st = fk_layernorm_rows_ex(x.data_ptr(), out.data_ptr(), ptrs[0], ptrs[1], rows, cols, code, eps,
                              _EPILOGUES[gelu], plan, _stream_handle(x))
    if st != FK_OK:
        raise FkError(st, "fk_layernorm_rows")
    return out


def attention(q, k, v, causal: bool = True, scale: float | None = None, out=None):
    """Attention forward on contiguous bf16 CUDA tensors [..., t, d] (all
    leading dimensions are independent slices): softmax(scale q k^T, causal)
    v, with scale = 1/sqrt(d) by default."""
    import math

    import torch
    for name, a in (("q", q), ("k", k), ("v", v)):
        _check_tensor(a, name)
        if a.dtype != torch.bfloat16 or a.shape != q.shape:
            raise ValueError(f"{name} must be bfloat16 with q's shape")
    t, d = q.shape[-2], q.shape[-1]
    bh = q.numel() // (t * d) if t * d else 0
    if out is None:
        out = torch.empty_like(q)
    _check_tensor(out, "out")
    st = fk_attention_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), bh, t, d, int(bool(causal)),
                          1.0 / math.sqrt(d) if scale is None else scale, _stream_handle(q))
    if st != FK_OK:
        raise FkError(st, "fk_attention_fwd")
    return out


# ---------------------------------------------------------------- the 8-bit linear layer
#
# At decode sizes the host side of a call outlasts its kernel, so these
# helpers look up what they need of torch once, test operands in line and
# leave the wording of a refusal to _like().

_torch = None           # the torch module, at first use
_FLOAT_CODES: dict = {}  # torch.float32 / torch.bfloat16 -> fk_dtype
_Q8_CODES: dict = {}     # torch.int8 / torch.float8_e4m3fn -> fk_q8type


def _load_torch():
    global _torch
    import torch
    _FLOAT_CODES.update({torch.float32: FK_F32, torch.bfloat16: FK_BF16})
    _Q8_CODES.update({torch.int8: FK_I8, torch.float8_e4m3fn: FK_E4M3})
    _torch = torch
    return torch


def _like(t, name: str, shape, dtype, device: int) -> int:
    """Address of an operand that must be contiguous CUDA memory of this
    shape, type and device index (0 for None)."""
    if t is None:
        return 0
    if (isinstance(t, _torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    _check_tensor(t, name)
    raise ValueError(f"{name} must have shape {tuple(shape)} and type {dtype}, on cuda:{device}")


def _new(lead, n: int | None, dtype, like):
    """Empty contiguous tensor of the shape [*lead] or [*lead, n] where `like`
    is.  (One leading dimension is nearly always what there is; empty_strided
    takes 1.4 us of host time, new_empty 2.0.)"""
    if len(lead) == 1:
        m = lead[0]
        return (_torch.empty_strided((m,), (1,), dtype=dtype, device=like.device) if n is None else
                _torch.empty_strided((m, n), (n if n > 0 else 1, 1), dtype=dtype, device=like.device))
    return like.new_empty(lead if n is None else (*lead, n), dtype=dtype)


def _rows_input(x, name: str):
    """(fk_dtype, shape, rows, columns) of a contiguous fp32/bf16 CUDA tensor."""
    _check_tensor(x, name)
    code = _FLOAT_CODES.get(x.dtype)
    if code is None:
        raise TypeError("fk operators take float32 or bfloat16")
    shape = x.shape
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    cols = shape[-1]
    return code, shape, (x.numel() // cols if cols else 0), cols


def rmsnorm(x, weight=None, eps: float = 1e-6, residual=None, out_dtype=None, out=None, scales=None,
            residual_out=None):
    """Root-mean-square norm over the last dimension of a contiguous fp32/bf16
    CUDA tensor, h / sqrt(mean(h^2) + eps) * weight with h = x + residual
    (rounded to x's type; h = x without a residual).

    out_dtype: x's type (default), or torch.int8 / torch.float8_e4m3fn for
    8-bit codes with one fp32 scale per row.  Returns y, or (codes, scales);
    with a residual, h comes last: (y, h) or (codes, scales, h).  weight: fp32,
    x.shape[-1] values.  residual_out may be residual or x (updated in place)."""
    torch = _torch or _load_torch()
    code, shape, rows, cols = _rows_input(x, "x")
    dtype, dev = x.dtype, x.get_device()
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    q8 = _Q8_CODES.get(out_dtype)
    p_scales = p_h = 0
    # what is made here needs no checks
    if out is None:
        out = torch.empty_like(x, dtype=out_dtype)
        p_out = out.data_ptr()
    else:
        p_out = _like(out, "out", shape, out_dtype, dev)
    if q8 is None:
        if out_dtype is not dtype:
            raise TypeError("out_dtype must be x's dtype, torch.int8 or torch.float8_e4m3fn")
        if scales is not None:
            raise ValueError("scales belong to 8-bit outputs")
    elif cols == 0:
        raise ValueError("rows without columns have no scale")
    elif scales is None:
        scales = _new(shape[:-1], None, torch.float32, x)
        p_scales = scales.data_ptr()
    else:
        p_scales = _like(scales, "scales", shape[:-1], torch.float32, dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
    elif residual_out is None:
        residual_out = torch.empty_like(x)
        p_h = residual_out.data_ptr()
    else:
        p_h = _like(residual_out, "residual_out", shape, dtype, dev)
    st = lib().fk_rmsnorm_rows(x.data_ptr(), _like(residual, "residual", shape, dtype, dev),
                               _like(weight, "weight", (cols,), torch.float32, dev), p_out, p_scales, p_h, rows, cols,
                               code, code if q8 is None else q8, eps, _stream_handle(x))
    if st != FK_OK:
        raise FkError(st, "fk_rmsnorm_rows")
    if q8 is None:
        return out if residual is None else (out, residual_out)
    return (out, scales) if residual is None else (out, scales, residual_out)


def rmsnorm_backward(dy, h, weight=None, eps: float = 1e-6, dresidual=None, out=None, dweight=None,
                     need_dweight: bool = True, workspace=None):
    """Gradients of rmsnorm (its output in x's type): returns (dx, dweight).

    h: what was normalised (rmsnorm's last result, or its x without a
    residual); dresidual: gradient that arrives at h from the residual stream,
    added to dx.  dx is the gradient of x and of residual alike; it may be
    written over dy, h or dresidual (out=).  dweight is fp32, None when
    need_dweight is false.  `workspace` (a CUDA tensor of at least
    fk_rmsnorm_rows_bwd_workspace bytes) makes the call allocation-free."""
    torch = _torch or _load_torch()
    code, shape, rows, cols = _rows_input(h, "h")
    dtype, dev = h.dtype, h.get_device()
    p_dw = 0
    if not need_dweight:
        if dweight is not None:
            raise ValueError("dweight given, but need_dweight is false")
    elif dweight is None:
        dweight = _new((cols,), None, torch.float32, h)
        p_dw = dweight.data_ptr()
    else:
        p_dw = _like(dweight, "dweight", (cols,), torch.float32, dev)
    if out is None:
        out = torch.empty_like(h)
        p_out = out.data_ptr()
    else:
        p_out = _like(out, "out", shape, dtype, dev)
    if dy is None:
        raise TypeError("dy must be a CUDA tensor")
    args = (_like(dy, "dy", shape, dtype, dev), h.data_ptr(), _like(weight, "weight", (cols,), torch.float32, dev),
            _like(dresidual, "dresidual", shape, dtype, dev), p_out, p_dw, rows, cols, code, eps)
    if workspace is None:
        st = lib().fk_rmsnorm_rows_bwd(*args, _stream_handle(h))
    else:
        _check_tensor(workspace, "workspace")
        st = lib().fk_rmsnorm_rows_bwd_ws(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                          _stream_handle(h))
    if st != FK_OK:
        raise FkError(st, "fk_rmsnorm_rows_bwd")
    return out, dweight


def quantize_rows(x, dtype=None, gelu: str | None = None, out=None, scales=None):
    """Rows (the last dimension) of a contiguous fp32/bf16 CUDA tensor to 8-bit
    codes and one fp32 scale each: (codes, scales), codes * scales[..., None]
    being the values.  dtype: torch.int8 (default) or torch.float8_e4m3fn;
    gelu: None, "tanh" or "erf" (or torch's "none", the exact form), applied
    first."""
    torch = _torch or _load_torch()
    code, shape, rows, cols = _rows_input(x, "x")
    epilogue = _EPILOGUES.get(gelu)
    if epilogue is None:
        raise ValueError("gelu must be None, 'tanh' or 'erf'")
    if cols == 0:
        raise ValueError("rows without columns have no scale")
    if dtype is None:
        dtype = torch.int8 if out is None else out.dtype
    q8 = _Q8_CODES.get(dtype)
    if q8 is None:
        raise TypeError("dtype must be torch.int8 or torch.float8_e4m3fn")
    if out is None:
        out = torch.empty_like(x, dtype=dtype)
        p_out = out.data_ptr()
    else:
        p_out = _like(out, "out", shape, dtype, x.get_device())
    if scales is None:
        scales = _new(shape[:-1], None, torch.float32, x)
        p_scales = scales.data_ptr()
    else:
        p_scales = _like(scales, "scales", shape[:-1], torch.float32, x.get_device())
    st = lib().fk_quantize_rows(x.data_ptr(), p_out, p_scales, rows, cols, code, q8, epilogue, _stream_handle(x))
    if st != FK_OK:
        raise FkError(st, "fk_quantize_rows")
    return out, scales


def matmul_q8(a, a_scales, b, b_scales, bias=None, gelu: str | None = None, out_dtype=None, out=None,
              workspace=None):
    """act((a @ b.T) * a_scales[..., None] * b_scales + bias) of 8-bit codes:
    a [..., k] and b [n, k] (a Linear weight), both torch.int8 or both
    torch.float8_e4m3fn, contiguous CUDA tensors; a_scales [...], b_scales [n]
    and bias [n] fp32; act: None, "tanh" or "erf" GELU.  Returns [..., n] in
    out_dtype (bfloat16 by default, or float32).  `workspace` (a CUDA tensor
    of at least fk_matmul_q8_workspace bytes) makes a call that needs one
    allocation-free."""
    torch = _torch or _load_torch()
    _check_tensor(a, "a")
    _check_tensor(b, "b")
    q8 = _Q8_CODES.get(a.dtype)
    if q8 is None or b.dtype is not a.dtype:
        raise TypeError("a and b must both be torch.int8 or both torch.float8_e4m3fn")
    shape, dev, f32 = a.shape, a.get_device(), torch.float32
    if not shape or b.dim() != 2 or b.shape[1] != shape[-1] or b.get_device() != dev:
        raise ValueError("a is [..., k] and b is [n, k], on one device")
    epilogue = _EPILOGUES.get(gelu)
    if epilogue is None:
        raise ValueError("gelu must be None, 'tanh' or 'erf'")
    n, k = b.shape
    lead = shape[:-1]
    if a_scales is None or b_scales is None:
        raise TypeError("a_scales and b_scales must be CUDA tensors")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    out_code = _FLOAT_CODES.get(out_dtype)
    if out_code is None:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    if out is None:
        out = _new(lead, n, out_dtype, a)
        p_out = out.data_ptr()
    else:
        p_out = _like(out, "out", (*lead, n), out_dtype, dev)
    args = (a.data_ptr(), b.data_ptr(), _like(a_scales, "a_scales", lead, f32, dev),
            _like(b_scales, "b_scales", (n,), f32, dev), _like(bias, "bias", (n,), f32, dev), p_out, lead.numel(), n, k,
            q8, out_code, epilogue)
    if workspace is None:
        st = lib().fk_matmul_q8(*args, _stream_handle(a))
    else:
        _check_tensor(workspace, "workspace")
        st = lib().fk_matmul_q8_ws(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream_handle(a))
    if st != FK_OK:
        raise FkError(st, "fk_matmul_q8")
    return out


__all__ = [
    "FK_OK", "FK_ERR_INVALID_ARG", "FK_ERR_UNSUPPORTED_DTYPE", "FK_ERR_UNSUPPORTED_DEVICE",
    "FK_ERR_CUDA", "FK_F32", "FK_BF16", "FK_GELU_TANH", "FK_GELU_ERF", "FK_PATH_AUTO", "FK_PATH_WARP", "FK_PATH_CTA",
    "FK_PATH_CLUSTER", "FK_PATH_TWOPHASE", "FK_PATH_SPLIT", "FkError", "SoftmaxPlan", "lib", "header_functions",
    "fk_gelu_tanh", "fk_gelu", "fk_copy", "fk_softmax_rows", "fk_softmax_rows_ex", "fk_softmax_rows_plan",
    "fk_softmax_rows_workspace", "fk_softmax_rows_ws", "fk_softmax_rows_noalloc", "fk_softmax_rows_noalloc_cap",
    "fk_softmax_rows_causal", "fk_softmax_rows_causal_ex", "softmax_causal", "FK_SOFTMAX_SKIP_MASKED",
    "fk_layernorm_rows", "fk_layernorm_rows_ex", "fk_layernorm_rows_plan", "layernorm",
    "fk_attention_fwd", "attention", "FK_EPILOGUE_NONE", "FK_EPILOGUE_GELU_TANH",
    "FK_EPILOGUE_GELU_ERF",
    "fk_status_string", "fk_last_cuda_error", "fk_version", "fk_wait_timeouts",
    "fk_wait_selftest", "make_plan", "gelu_tanh", "gelu",
    "softmax_rows", "FK_I8", "FK_E4M3",
    "fk_rmsnorm_rows", "fk_rmsnorm_rows_bwd", "fk_rmsnorm_rows_bwd_workspace", "fk_rmsnorm_rows_bwd_ws",
    "fk_quantize_rows", "fk_matmul_q8", "fk_matmul_q8_workspace", "fk_matmul_q8_ws",
    "fk_matmul_q8_wait_selftest",
    "rmsnorm", "rmsnorm_backward", "quantize_rows", "matmul_q8",
]
