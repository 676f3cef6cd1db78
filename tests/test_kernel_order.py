"""What is read from the kernels' sources: helpers that nothing calls, and the order of a kernel's first steps (a deadlock is not
to be tried on a GPU).

A kernel launched early holds tensor memory while it waits for the one before it.  So a kernel that allocates
tensor memory does so, on every path, before it lets the next one start."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_scaled_gemm_sm_gb300", "csrc")


def _kernels():
    for f in sorted(os.listdir(CSRC)):
        if f.endswith(".cu"):
            text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
            for part in text.split("__global__")[1:]:
                yield f, re.search(r"(\w+)\s*\(\s*(?:const|CUtensorMap|__grid)", part).group(1), part


KERNELS = [(f, name, part) for f, name, part in _kernels() if "tmem_alloc" in part]


def test_kernels_with_tensor_memory_are_found():
    assert {"prompt_kernel", "prompt_tile_kernel", "mxfp8_pair_kernel", "blockscale_pair_kernel"} <= {name for _, name, _ in KERNELS}


@pytest.mark.parametrize("f,name,part", KERNELS, ids=[k[1] for k in KERNELS])
def test_tensor_memory_is_allocated_before_the_next_kernel_may_start(f, name, part):
    alloc = re.search(r"tmem_alloc\w*\(", part).end()
    launch = part.index("grid_dep_launch()")
    assert alloc < launch
    assert "__syncthreads()" in part[alloc:launch]  # all warps know of it
    assert part.count("grid_dep_launch()") == 1


def test_every_device_helper_is_called():
    text = "".join(re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read()) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")))
    names = set(re.findall(r"__device__ __forceinline__ (?:static )?[\w:<>]+[ &*]+(\w+)\(", text))
    assert len(names) > 60
    assert sorted(n for n in names if len(re.findall(r"\b%s\b" % n, text)) == 1) == []
