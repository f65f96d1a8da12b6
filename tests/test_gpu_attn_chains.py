"""Attention followed at once by kernels that take tensor memory of their own (GPU)."""
import pytest
import torch

import _layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


@pytest.mark.parametrize("kv", [300, 640])
def test_few_columns_after_all_columns(capi, kv):
    """k_attn_prefill takes all of a multiprocessor's tensor memory, and at head size 64 leaves shared memory
    for a CTA of the E4M3 W8A16 linear that follows: it must hold its columns before that one starts."""
    a = ref.Attn([16], [kv], 1, 71, 64, 16, seed=kv)
    assert capi.qlin_attn_mixed_kernel_name(1, 71, 1, 64, 16, kv) == "k_attn_unpack+k_attn_prefill"
    g = torch.Generator().manual_seed(kv)
    w = capi.quantize_weight("e4m3", (torch.randn(1024, 71 * 64, generator=g) / 64).cuda())
    cache, q, qs, n, table = ([t.cuda() for t in a.cache()], a.q.cuda(), a.q_start.cuda(), a.kv_len.cuda(),
                              a.table.cuda())

    def step(between=lambda: None):
        x = capi.attn_mixed(q, qs, n, table, 16, cache, 16, kv)
        between()
        return capi.w8a16_linear("e4m3", x, *w)

    want = step(torch.cuda.synchronize).clone()
    assert torch.equal(step(), want)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(4):
            y = step()
    for _ in range(8):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and capi.qlin_get_device_status() == capi.QLIN_OK
