"""Order of steps in the kernels of the 8-bit layer that no run on a GPU shows
reliably, read from their sources (without a GPU)."""
import os
import re

import pytest

import memory_bound_fk_b200

CSRC = os.path.join(os.path.dirname(os.path.abspath(memory_bound_fk_b200.__file__)), "csrc")
PRODUCT = ["fk_matmul_q8.cu", "fk_matmul_q8_pair.cu"]


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(name):
    """(name, body) of each __global__ function of a source file."""
    src, out = text(name), []
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", src):
        at = src.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
            if depth == 0:
                break
        out.append((m.group(1), src[at:end]))
    assert out
    return out


PRODUCT_KERNELS = [(f, k, b) for f in PRODUCT for k, b in kernels(f)]


@pytest.mark.parametrize("file,kernel,body", PRODUCT_KERNELS, ids=[k for _, k, _ in PRODUCT_KERNELS])
def test_a_pair_frees_its_tensor_memory_after_both_blocks_have_read_it(file, kernel, body):
    if "tmem_dealloc_pair" not in body:
        return
    last_read = max(m.start() for m in re.finditer(r"tmem_ld\w+\(", body))
    assert "cluster_sync();" in body[last_read:body.index("tmem_dealloc_pair")]


@pytest.mark.parametrize("file,kernel,body", PRODUCT_KERNELS, ids=[k for _, k, _ in PRODUCT_KERNELS])
def test_the_next_kernel_may_start_once_tensor_memory_is_taken(file, kernel, body):
    """A successor that starts early and takes tensor memory holds it until
    this kernel has ended: no block of this one may still be waiting for any.
    One thread's signal counts for its block, so it comes from the warp that
    allocates."""
    if "tmem_alloc" not in body:
        assert "let_next_start();" in body
        return
    assert body.count("let_next_start();") == 1
    assert re.search(r"if \(warp == [^)]*\) \{\s*(tc::)?tmem_alloc\w*\([^;]*\);\s*let_next_start\(\);\s*\}", body)


def test_early_started_kernels_read_coherently():
    """A kernel that starts while its predecessor writes may not read that
    data as constant for its life (non-coherent loads, __ldg, which the
    compiler may also move ahead of the wait)."""
    for name in sorted(os.listdir(CSRC)):
        src = text(name)
        if "after_previous()" in src or name == "fk_q8_rows.cuh":
            for banned in ("__ldg", ".nc.", "ld_stream_v4", "load1(", "__restrict__"):
                assert banned not in src, f"{banned} in {name}"


def test_every_early_started_kernel_waits_for_its_predecessor():
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu") and "launch_overlapped(" in text(name):
            for kernel, body in kernels(name):
                if "let_next_start();" in body:
                    assert body.count("after_previous();") == 1
                    seen += 1
    assert seen >= 9


def test_accumulators_are_used_after_the_wait_for_their_load():
    """A tcgen05.ld fills its registers later: in one asm statement with its
    wait, no use of them can be placed between the two."""
    for name in PRODUCT:
        assert "tmem_ld32_async" not in text(name)
    for m in re.finditer(r"__device__[^{]*\btmem_ld\w*\([^{]*\{(.*?)\n\}", text("fk_mm.cuh"), re.S):
        assert m.group(1).count("asm volatile") == 1 and "tcgen05.wait::ld" in m.group(1)
