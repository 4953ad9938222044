"""Dynamic shared memory begins where the static arrays end, on the alignment that its declaration asks for: kernels that
read it in vectors have to ask for 16 bytes, or round its address up.  (A misaligned vector access is a fault, so this
is shown on the source.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tile_scheduled_tensor_gb300", "csrc")
KERNEL = re.compile(r"__global__.*?\n}\n", re.S)
DECLARED = re.compile(r"extern __shared__ (?:__align__\((\d+)\) )?(\w+) (\w+)\[\];")


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))):
        for body in KERNEL.findall(open(path).read()):
            m = DECLARED.search(body)
            if m:
                name = re.search(r"(\w+)\(const", body).group(1)
                yield pytest.param(body, int(m.group(1) or 0), m.group(3), id=name)


@pytest.mark.parametrize("body,asked,array", list(_kernels()))
def test_vectors_in_dynamic_shared_memory_are_aligned(body, asked, array):
    rounded = re.search(re.escape(array) + r"\) \+ 1023\) & ~uintptr_t\(1023\)", body) is not None
    vectors = re.search(r"\b(float[24]|uint[24]|int4|longlong2)\b|alignas\(VEC", body) is not None
    assert rounded or asked >= 16 or not vectors


def test_the_kernels_are_found():
    names = [p.id for p in _kernels()]
    assert "score_rows_kernel" in names and "gemm_int8_kernel" in names and len(names) >= 8, names
