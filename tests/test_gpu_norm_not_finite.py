"""RMSNorm to codes where values are not finite (GPU): the codes are the ones the
activation quantizers of the same scale give.

Per value: a NaN is the NaN code of E4M3 (either sign) and -127 in INT8, an infinity
the largest code; a per-token scale is that of the largest value that is a number."""
import numpy as np
import pytest
import torch

import _layer_ref as ref
from bit_quantized_linear_gb300 import synth

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _dev(a):
    return torch.from_numpy(synth.f32_to_bf16_bits(a).view(np.int16)).cuda().view(torch.bfloat16)


def _rows(M, K, weights):
    rng = synth.rng_for("test-norm-not-finite", 0, f"{M}x{K}", "rows")
    x = ref.bf16_round(rng.standard_normal((M, K), dtype=np.float32))
    w = ref.bf16_round(1 + 0.2 * rng.standard_normal(K, dtype=np.float32))
    x[1, 5], x[2, K - 3], x[3, 7], x[4, 0] = np.inf, -np.inf, np.nan, -np.nan
    if weights:
        w[K // 2], w[9], w[K - 1] = np.nan, np.inf, -np.inf
    return x, w


def _codes(y, s, qtype):
    """(codes, where they are NaN)"""
    with np.errstate(all="ignore"):
        v = (y / s).astype(np.float32)
    bad = np.isnan(v)
    v = np.where(bad, np.float32(0), v)
    c = ref.codes(v, np.float32(1), qtype)
    return (np.where(bad, np.uint8(0x81), c) if qtype == "int8" else c), bad


def _check(got, y, s, qtype):
    want, bad = _codes(y, s, qtype)
    if qtype == "e4m3":
        assert ((got[bad] & 0x7F) == 0x7F).all()
        got, want = got[~bad], want[~bad]
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("M,K", [(6, 512), (2600, 512), (600, 2048), (6, 32768)])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("qtype", ["int8", "e4m3"])
@pytest.mark.parametrize("static", [True, False])
def test_codes(capi, M, K, weights, qtype, static):
    x, w = _rows(M, K, weights)
    _, y = ref.norm(x, None, w, EPS)
    if static:
        s = np.full(1, 0.03 if qtype == "int8" else 0.009, np.float32)
    else:
        top = np.fmax.reduce(np.abs(y), axis=1, initial=0).astype(np.float32)
        s = (top / np.float32(127 if qtype == "int8" else 448)).astype(np.float32)
        s = np.where(s > 0, s, np.float32(1))
    _, codes, gs = capi.rmsnorm_quant(qtype, _dev(x), _dev(w), EPS,
                                      input_scale=torch.from_numpy(s).cuda() if static else None)
    np.testing.assert_array_equal(gs.cpu().numpy(), s)
    _check(codes.cpu().numpy(), y, s if static else s[:, None], qtype)


@pytest.mark.parametrize("qtype", ["int8", "e4m3"])
def test_the_quantizers_give_these(capi, qtype):
    """The definition above is the quantizers' own: BF16 values that are not finite, through them."""
    x = np.ones((1, 64), np.float32)
    x[0, :4] = np.nan, np.inf, -np.inf, -np.nan
    s = np.full(1, 0.01, np.float32)
    got = capi.quantize_act_static(qtype, _dev(x), torch.from_numpy(s).cuda())
    _check(got.cpu().numpy(), x, s, qtype)
    x[0, 1:3] = 3.0
    s = (np.float32(3) / np.float32(127 if qtype == "int8" else 448)).astype(np.float32)
    got, gs = capi.quantize_act_dynamic(qtype, _dev(x))
    assert gs.item() == s
    _check(got.cpu().numpy(), x, s, qtype)


@pytest.mark.parametrize("qtype", ["int8", "e4m3"])
def test_the_linear_shows_it(capi, qtype):
    """A NaN in a row of the stream reaches the next linear's outputs of that row (E4M3), and no other row's."""
    K, N = 512, 64
    x, w = _rows(6, K, False)
    qw, sw = capi.quantize_weight(qtype, torch.ones(N, K, device="cuda"))
    s = torch.full((1,), 0.02, device="cuda")
    _, codes, s = capi.rmsnorm_quant(qtype, _dev(x), _dev(w), EPS, input_scale=s)
    y = capi.w8a8_linear_codes(qtype, codes, s, qw, sw).float().cpu()
    if qtype == "e4m3":
        assert torch.isnan(y[1:5]).all()
    assert torch.isfinite(y[[0, 5]]).all()
