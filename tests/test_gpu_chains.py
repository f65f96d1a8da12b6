"""Calls that read what the call before them wrote, replayed from a graph (GPU).

In a graph, unlike in calls from the host, each kernel starts while its predecessor
runs; a read that does not wait for it sees the memory of the replay before.  So the
inputs change from replay to replay, and each result is compared, bit for bit, with
the same calls made one by one with a synchronize between them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
K, N = 768, 1024


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _weights(capi, qt, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    return capi.quantize_weight(qt, (torch.randn(n, k, generator=g) / k ** 0.5).cuda())


def _check(capi, calls, inputs):
    """calls: functions of the result so far (a tensor) -> the next; inputs: the tensors of the replays."""
    def run(x, between=lambda: None):
        for f in calls:
            x = f(x)
            between()
        return x

    want = []
    for x in inputs:
        want.append(run(x, torch.cuda.synchronize).clone())
    first = torch.zeros_like(inputs[0])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = run(first)
    for x, w in zip(inputs, want):
        first.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), w.view(torch.uint8))
    assert capi.qlin_get_device_status() == capi.QLIN_OK


def _inputs(M, n=4):
    g = torch.Generator().manual_seed(M)
    return [torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(n)]


@pytest.mark.parametrize("qt", ["e4m3", "int8"])
@pytest.mark.parametrize("M", [1, 2, 16, 32, 100, 300])
def test_weight_only_linears(capi, qt, M):
    a, b = _weights(capi, qt, 2 * N, K, 1), _weights(capi, qt, K, N, 2)
    _check(capi, [lambda x: capi.w8a16_gate_up_silu(qt, x, *a), lambda x: capi.w8a16_linear(qt, x, *b)] * 2,
           _inputs(M))


@pytest.mark.parametrize("qt", ["e4m3", "int8"])
@pytest.mark.parametrize("M", [1, 2, 16, 100, 300])
@pytest.mark.parametrize("dynamic", [True, False])
def test_quantized_linears(capi, qt, M, dynamic):
    a, b = _weights(capi, qt, N, K, 3), _weights(capi, qt, K, N, 4)
    s = torch.full((1,), 0.03, device="cuda")
    f = (lambda w: lambda x: capi.w8a8_dynamic_linear(qt, x, *w)) if dynamic else \
        (lambda w: lambda x: capi.w8a8_linear(qt, x, s, *w))
    _check(capi, [f(a), f(b)] * 2, _inputs(M))


@pytest.mark.parametrize("qt", ["e4m3", "int8"])
@pytest.mark.parametrize("M", [1, 2, 100, 300])
def test_norm_and_codes(capi, qt, M):
    a, b, u = _weights(capi, qt, N, K, 5), _weights(capi, qt, K, N, 6), torch.ones(K, device="cuda").bfloat16()

    def norm(x):
        return capi.w8a8_linear_codes(qt, *capi.rmsnorm_quant(qt, x, u, 1e-6, residual=x)[1:], *a)

    _check(capi, [norm, lambda x: capi.w8a16_linear(qt, x, *b), lambda x: capi.rmsnorm(x, u, 1e-6, residual=x)[1],
                  lambda x: capi.w8a16_linear(qt, x, *a)], _inputs(M))


@pytest.mark.parametrize("T", [1, 33, 300])
def test_projection_rotation_store_load_attention(capi, T):
    H, D = 2, 64
    a, b = _weights(capi, "e4m3", 8 * D, K, 7), _weights(capi, "e4m3", K, 4 * D, 8)
    table, pos = capi.rope_table(512, D), torch.arange(T, device="cuda")
    slots = (torch.arange(T, device="cuda") * 7) % 512
    cache = capi.kv_cache_alloc(512, H, D)
    for t in cache:
        t.zero_()
    starts, kv = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T], [512]))
    blocks = torch.arange(32, dtype=torch.int32, device="cuda").view(1, 32)

    def layer(x):
        qkv = capi.w8a16_linear("e4m3", x, *a)
        q = torch.empty(T, 4 * D, dtype=torch.bfloat16, device="cuda")
        capi.qlin_rope_kv_store_mixed("half", 4, D, table, pos, qkv[:, : 4 * D], qkv[:, 4 * D: 6 * D], qkv[:, 6 * D:],
                                      q, slots, *cache)
        y = capi.attn_mixed(q, starts, kv, blocks, 16, cache, T, 512, causal=False)
        return capi.w8a16_linear("e4m3", y, *b)

    def stored(x):
        return torch.cat([t.reshape(T, -1) for t in capi.kv_load_mixed(slots, cache)] + [x], dim=1)

    # The store runs before the load in every call, so nothing of an earlier replay's cache is seen
    _check(capi, [layer, stored], _inputs(T))
