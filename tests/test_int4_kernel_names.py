"""The names that qlin_attn_int4_kernel_name reports are those of the kernels in the sources, and all of them (host)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_linear_gb300", "csrc")
SIZES = [(1, 16, 2, 128, 1, 37), (1, 28, 4, 128, 1, 32768), (256, 16, 2, 128, 1, 4096), (1, 28, 4, 128, 1, 131072),
         (1, 28, 4, 128, 8192, 16384), (5, 8, 8, 64, 333, 3001), (2, 14, 2, 128, 300, 9000), (1, 28, 4, 128, 1500, 16384),
         (3, 16, 2, 256, 700, 5000), (1, 4, 1, 32, 900, 5000), (2, 1600, 160, 64, 200, 6000)]


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import build
    build.build()
    from bit_quantized_linear_gb300 import capi as c
    return c


def _kernels(file):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    return set(re.findall(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(k_\w+)", text))


def test_names_are_kernels(capi):
    few, many = _kernels("attn_int4.cu"), _kernels("attn_prefill.cu")
    assert "k_attn_int4" in few and "k_attn_prefill" in many
    told = {n for s in SIZES for n in capi.qlin_attn_int4_kernel_name(*s).split("+")}
    assert few <= told, f"launched under another name: {few - told}"
    assert told <= few | many | _kernels("attn_split.cu")  # the join of the many rows' parts is there
