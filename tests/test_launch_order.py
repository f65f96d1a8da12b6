"""Order of tensor-memory allocation and early launch in the kernels' sources (host).

A kernel that lets its dependents start before it holds its tensor memory can wait
for ever: a dependent's CTA may take the columns first, and gives them back only
after it has waited for this kernel to end."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_linear_gb300", "csrc")


def _kernels():
    """(file:name, body) of every __global__ function, comments taken out."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        src = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        for m in re.finditer(r"__global__", src):
            name = re.search(r"\b(k_\w+)\s*\(", src[m.end():])
            at = src.index("{", m.end() + name.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                end += 1
            out.append((f"{os.path.basename(path)}:{name.group(1)}", src[at:end]))
    return out


ALLOCATING = [k for k in _kernels() if "tmem_alloc" in k[1]]


def test_allocating_kernels_are_found():
    assert {"k_attn_prefill", "k_w8a16_f8"} <= {n.split(":")[1] for n, _ in ALLOCATING}


@pytest.mark.parametrize("body", [b for _, b in ALLOCATING], ids=[n for n, _ in ALLOCATING])
def test_tensor_memory_before_dependents(body):
    alloc = max(m.start() for m in re.finditer(r"tmem_alloc(_pair)?\s*\(", body))
    barrier = body.index("__syncthreads()", alloc)
    assert body.index("pdl_trigger()") > barrier
