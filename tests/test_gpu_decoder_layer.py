"""The example decoder layer: every operator's output against its restatement on the
inputs it really had, and replayed decode steps against direct ones (GPU)."""
import os
import sys

import numpy as np
import pytest
import torch

import _layer_ref as ref
from _helpers import ELEM_REL, ELEM_RMS, bf16_to_f64, check_tol, from_dev_bf16
from bit_quantized_linear_gb300 import synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu
HIDDEN, HQ, H, D, INTER, BLOCK = 512, 8, 2, 64, 768, 32


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_layer
    return decoder_layer


def _f32(t):
    return synth.bf16_bits_to_f32(from_dev_bf16(t))


def _np(t):
    return t.cpu().numpy()


def _attention(layer, batch, new, q):
    """(out, tolerance) of the attention over the layer's cache as it is now."""
    a = ref.Attn.__new__(ref.Attn)
    a.nq, a.kv = list(new), batch.kv_len.tolist()
    a.H, a.G, a.D, a.block = H, HQ // H, D, BLOCK
    a.q, a.q_start, a.kv_len, a.table = q.cpu(), batch.q_start.cpu(), batch.kv_len.cpu(), batch.blocks.cpu()
    kc, ks, vc, vs = (t.cpu() for t in layer.cache)
    a.kc, a.ks, a.vc, a.vs = kc, ks.view(torch.float16), vc, vs.view(torch.float16)
    return a.reference()


def _elements(y_bits, want, what):
    """The bar of the linears element by element.  Its Frobenius part is for many elements: rounding alone is
    1.7e-3 of it on average, and passes 2e-3 in single rows with a few large outputs."""
    rms = float(np.sqrt(np.mean(want * want)))
    assert np.all(np.abs(bf16_to_f64(y_bits) - want) <= ELEM_REL * np.abs(want) + ELEM_RMS * rms), what


def _check_layer(orc, layer, x, residual, batch, new, table, before, seen, out, check_tol=check_tol):
    """before: the cache as host arrays from before the call."""
    h, y = ref.norm(_f32(x), None if residual is None else _f32(residual), _f32(layer.norm_in), layer.eps)
    s = ref.row_scales(y, "e4m3")
    np.testing.assert_array_equal(_f32(seen["h"]), h)
    np.testing.assert_array_equal(_np(seen["scale"]), s)
    np.testing.assert_array_equal(_np(seen["codes"]), ref.codes(y, s[:, None], "e4m3"))
    E = orc.E4M3
    qw, sw = (_np(t) for t in layer.qkv)
    check_tol(from_dev_bf16(seen["qkv"]), orc.w8a8_per_token(E, _np(seen["codes"]), s, qw, sw), "qkv")

    n, m, T = HQ * D, H * D, x.shape[0]
    qkv = _f32(seen["qkv"])
    rows = _np(table)[_np(batch.positions)]
    turned = ref.rope(qkv[:, : n + m].reshape(T, HQ + H, D), rows, D, "half").reshape(T, n + m)
    np.testing.assert_array_equal(_f32(seen["q"]), turned[:, :n])
    cache = orc.KVCache(before[0].shape[0], H, D)
    cache.k_cache[:], cache.k_scale[:], cache.v_cache[:], cache.v_scale[:] = before
    orc.kv_store(cache, synth.f32_to_bf16_bits(turned[:, n:]), synth.f32_to_bf16_bits(qkv[:, n + m:]),
                 _np(batch.slots))
    for got, want in zip(_cache(layer), (cache.k_cache, cache.k_scale, cache.v_cache, cache.v_scale)):
        np.testing.assert_array_equal(got, want)

    want, tol = _attention(layer, batch, new, seen["q"])
    assert ((seen["a"].cpu().double() - want).abs() <= tol).all()
    qa, sa = orc.quantize_act_per_token(E, from_dev_bf16(seen["a"]))
    check_tol(from_dev_bf16(seen["o"]), orc.w8a8_per_token(E, qa, sa, *(_np(t) for t in layer.o)), "o")
    h2, y2 = ref.norm(_f32(seen["o"]), h, _f32(layer.norm_mlp), layer.eps)
    np.testing.assert_array_equal(_f32(seen["h2"]), h2)
    np.testing.assert_array_equal(from_dev_bf16(seen["y"]), synth.f32_to_bf16_bits(y2))
    check_tol(from_dev_bf16(seen["up"]), orc.w8a16_gate_up_silu(E, from_dev_bf16(seen["y"]),
                                                               *(_np(t) for t in layer.gate_up)), "gate_up")
    check_tol(from_dev_bf16(out), orc.w8a16(E, from_dev_bf16(seen["up"]), *(_np(t) for t in layer.down)), "down")


def _cache(layer):
    kc, ks, vc, vs = (_np(t) for t in layer.cache)
    return kc.view(np.uint8), ks.view(np.uint16), vc, vs.view(np.uint16)


def _prompt_then_token(ex, orc, prompts, check_tol):
    from bit_quantized_linear_gb300 import capi
    B, max_kv = len(prompts), max(prompts) + 1
    per = -(-max_kv // BLOCK)
    g = torch.Generator().manual_seed(sum(prompts))
    blocks = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per).cuda()
    table = capi.rope_table(max_kv, D)
    layer = ex.DecoderLayer(HIDDEN, HQ, H, D, INTER, B * per * BLOCK)
    for t in layer.cache:
        t.zero_()
    for past, new, residual in (([0] * B, list(prompts), False), (list(prompts), [1] * B, True)):
        batch = ex.Batch(past, new, blocks, BLOCK, max_kv)
        x = torch.randn(sum(new), HIDDEN, generator=g).bfloat16().cuda()
        r = (2 * torch.randn(sum(new), HIDDEN, generator=g)).bfloat16().cuda() if residual else None
        before, seen = _cache(layer), {}
        out, h2 = layer(x, r, batch, table, seen)
        assert capi.qlin_get_device_status() == capi.QLIN_OK
        _check_layer(orc, layer, x, r, batch, new, table, before, seen, out, check_tol)


@pytest.mark.parametrize("prompts", [
    pytest.param((1,), marks=pytest.mark.xfail(strict=True, reason="one row: the correctly rounded gate_up output "
                                               "misses the Frobenius bar too (2.03e-3)")),
    (3, 70, 1), (150, 40)])
def test_prompt_then_token(ex, orc, prompts):
    _prompt_then_token(ex, orc, prompts, check_tol)


@pytest.mark.parametrize("prompts", [(2,), (33,)])
def test_one_sequence(ex, orc, prompts):
    _prompt_then_token(ex, orc, prompts, _elements)


def test_replayed_steps(ex):
    """Four steps from a graph give what four direct steps give, bit for bit."""
    from bit_quantized_linear_gb300 import capi
    prompts, steps = [40, 65], 4
    blocks = torch.arange(6, dtype=torch.int32, device="cuda").flip(0).view(2, 3).contiguous()
    table = capi.rope_table(96, D)
    layer = ex.DecoderLayer(HIDDEN, HQ, H, D, INTER, 6 * BLOCK)
    x = torch.randn(sum(prompts), HIDDEN, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    layer(x, None, ex.Batch([0, 0], prompts, blocks, BLOCK, 65), table)
    cache = [t.clone() for t in layer.cache]

    def run(replay):
        for t, c in zip(layer.cache, cache):
            t.copy_(c)
        batch = ex.Batch(prompts, [1, 1], blocks, BLOCK, 96)
        token = x[:2].clone()

        def step():
            token.copy_(layer(token, None, batch, table)[0])
            batch.advance()

        if not replay:
            for _ in range(steps):
                step()
            return token
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for _ in range(steps):
            graph.replay()
        torch.cuda.synchronize()
        return token

    direct = run(False)
    assert torch.equal(run(True).view(torch.int16), direct.view(torch.int16))
    assert capi.qlin_get_device_status() == capi.QLIN_OK
