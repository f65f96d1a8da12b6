"""Windows as wide as an int64 can say ("no limit") are planned as what they are, wider than any context."""
import pytest
import torch

import _int4_ref as ref

WIDE = [1 << 31, 1 << 40, 1 << 61, 1 << 62, (1 << 62) + 1, (1 << 63) - 1]
SIZES = [(4, 28, 4, 128, 1, 32768), (1, 28, 4, 128, 1, 131072), (256, 16, 2, 128, 1, 4096), (1, 4, 1, 128, 1, 128),
         (19, 8, 8, 256, 1, 2777), (3, 6, 6, 64, 5, 900), (2, 28, 4, 128, 700, 9000), (1, 8, 8, 64, 2048, 8192),
         (2, 8, 2, 256, 300, 5000), (1, 8, 1, 32, 60, 70000)]


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import build
    build.build()
    from bit_quantized_linear_gb300 import capi as c
    return c


@pytest.mark.parametrize("window", WIDE)
@pytest.mark.parametrize("size", SIZES)
def test_wide_windows(capi, size, window):
    """The same workspace and kernels as under 2^30, which no context passes either; the few rows' parts and the list of
    joins are there wherever a unit has more steps than one."""
    for ws, name in ((capi.qlin_attn_int4_workspace_bytes, capi.qlin_attn_int4_kernel_name),
                     (capi.qlin_attn_mixed_workspace_bytes, capi.qlin_attn_mixed_kernel_name)):
        assert ws(*size, window) == ws(*size, 1 << 30)
        assert name(*size, window) == name(*size, 1 << 30)


@pytest.mark.parametrize("size", SIZES)
def test_wide_windows_need_what_none_needs(capi, size):
    """A window wider than max_kv takes nothing away: no less workspace than without one."""
    assert capi.qlin_attn_int4_workspace_bytes(*size, (1 << 63) - 1) >= capi.qlin_attn_int4_workspace_bytes(*size, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1 << 30, 1 << 62, (1 << 63) - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,kv,D", [([1, 1, 1], [9000, 128, 0], 128), ([1, 5], [160, 3000], 256), ([300, 1], [900, 2000], 64)])
def test_outputs(capi, nq, kv, D, causal, window):
    a = ref.Attn4(nq, kv, 2, 4, D, 16, seed=D)
    a.many = "k_attn_unpack4" in capi.qlin_attn_int4_kernel_name(len(nq), 8, 2, D, max(nq), max(kv), window)
    want, tol = a.reference(causal=causal)
    n = capi.qlin_attn_int4_workspace_bytes(len(nq), 8, 2, D, max(nq), max(kv), window)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out = capi.attn_int4(a.q.cuda(), a.q_start.cuda(), a.kv_len.cuda(), a.table.cuda(), [t.cuda() for t in a.cache()],
                         max(nq), max(kv), causal=causal, window=window, ws=ws[:n])
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    assert ((out.float().cpu().double() - want).abs() <= tol).all()
    assert (ws[n:] == 0x5A).all()
