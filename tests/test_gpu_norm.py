"""RMSNorm with the residual's addition, and the W8A8 linear on its codes, against
a 64-bit plain restatement (GPU).

Everything after the row's sum is a fixed sequence of binary32 operations, and the
sum is good to about 2^-46, so h, BF16 outputs, codes and scales are compared bit
for bit."""
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


def _rows(M, K, tag, special=True):
    """fp32 arrays of BF16 values: x, residual, weight; with rows of zeros, of values whose squares leave
    binary32 on either side, and of mixed magnitudes."""
    rng = synth.rng_for("test-norm", 0, f"{M}x{K}", tag)
    x = ref.bf16_round(rng.standard_normal((M, K), dtype=np.float32))
    r = ref.bf16_round(2 * rng.standard_normal((M, K), dtype=np.float32))
    w = ref.bf16_round(1 + 0.2 * rng.standard_normal(K, dtype=np.float32))
    w[:: max(1, K // 3)] = 0
    if special:
        for m, f in enumerate([0.0, 2.0 ** 80, 2.0 ** -80, None]):
            if m < M - 1:
                g = np.float32(2.0) ** rng.integers(-30, 30, K).astype(np.float32) if f is None else np.float32(f)
                x[m] = ref.bf16_round(x[m] * g)
                r[m] = ref.bf16_round(r[m] * g)
    return x, r, w


def _dev(a):
    return torch.from_numpy(synth.f32_to_bf16_bits(a).view(np.int16)).cuda().view(torch.bfloat16)


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


SHAPES = [(1, 16), (1, 3584), (3, 48), (7, 272), (2, 2048), (37, 1040), (5, 3584), (300, 256), (2600, 512), (5, 11008),
          (2, 32768), (2500, 2064)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_bf16_output(capi, M, K, residual):
    x, r, w = _rows(M, K, "bf16")
    h, y = ref.norm(x, r if residual else None, w, EPS)
    gh, gy = capi.rmsnorm(_dev(x), _dev(w), EPS, residual=_dev(r) if residual else None)
    np.testing.assert_array_equal(_bits(gh), synth.f32_to_bf16_bits(h))
    np.testing.assert_array_equal(_bits(gy), synth.f32_to_bf16_bits(y))


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("qtype", ["int8", "e4m3"])
@pytest.mark.parametrize("static", [False, True])
def test_codes(capi, M, K, qtype, static):
    x, r, w = _rows(M, K, qtype)
    h, y = ref.norm(x, r, w, EPS)
    s = np.full(1, 0.03 if qtype == "int8" else 0.009, np.float32) if static else ref.row_scales(y, qtype)
    gh, gq, gs = capi.rmsnorm_quant(qtype, _dev(x), _dev(w), EPS, residual=_dev(r),
                                    input_scale=torch.from_numpy(s).cuda() if static else None)
    np.testing.assert_array_equal(gs.cpu().numpy(), s)
    np.testing.assert_array_equal(_bits(gh), synth.f32_to_bf16_bits(h))
    np.testing.assert_array_equal(gq.cpu().numpy(), ref.codes(y, s if static else s[:, None], qtype))


def test_strides_and_in_place_stream(capi):
    """x a column slice, the residual stream updated in place."""
    M, K = 45, 528
    x, r, w = _rows(M, K, "strides")
    wide = torch.full((M, K + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 16: 16 + K] = _dev(x)
    stream = _dev(r)
    y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    capi.qlin_rmsnorm(wide[:, 16: 16 + K], stream, _dev(w), EPS, stream, y)
    h, want = ref.norm(x, r, w, EPS)
    np.testing.assert_array_equal(_bits(stream), synth.f32_to_bf16_bits(h))
    np.testing.assert_array_equal(_bits(y), synth.f32_to_bf16_bits(want))
    assert (wide[:, :16] == 7).all() and (wide[:, 16 + K:] == 7).all()


def test_not_finite_rows(capi):
    """An infinity makes its row's sum infinite (r = 0, inf * 0 = NaN), a NaN spreads to the row; other rows
    keep their values.  Zero rows with eps = 0 are 0 * inf."""
    x, r, w = _rows(6, 512, "inf", special=False)
    x[1, 5], x[3, 7] = np.inf, np.nan
    _, y = capi.rmsnorm(_dev(x), _dev(w), EPS)
    _, want = ref.norm(x, None, w, EPS)
    got = synth.bf16_bits_to_f32(_bits(y))
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    np.testing.assert_array_equal(got[ok], ref.bf16_round(want)[ok])
    _, y = capi.rmsnorm(torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda"), _dev(w), 0.0)
    assert torch.isnan(y).all()


def test_no_rows(capi):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    capi.qlin_rmsnorm(e, None, torch.ones(64, dtype=torch.bfloat16, device="cuda"), EPS, None, e)
    assert capi.qlin_get_device_status() == capi.QLIN_OK


@pytest.mark.parametrize("qtype", ["int8", "e4m3"])
@pytest.mark.parametrize("M", [1, 5, 130, 1024])
def test_linear_on_codes(capi, qtype, M):
    """The linear on given codes returns the bits of the linears that quantize for themselves."""
    K, N = 528, 400
    rng = synth.rng_for("test-norm", 1, f"{M}", qtype)
    w = torch.from_numpy(synth.weights(N, K, rng)).cuda()
    x = _dev(ref.bf16_round(rng.standard_normal((M, K), dtype=np.float32)))
    bias = _dev(ref.bf16_round(rng.standard_normal(N, dtype=np.float32)))
    qw, s = capi.quantize_weight(qtype, w)
    qx, sx = capi.quantize_act_dynamic(qtype, x)
    want = capi.w8a8_dynamic_linear(qtype, x, qw, s, bias)
    np.testing.assert_array_equal(_bits(capi.w8a8_linear_codes(qtype, qx, sx, qw, s, bias)), _bits(want))
    one = torch.full((1,), 0.02, device="cuda")
    want = capi.w8a8_linear(qtype, x, one, qw, s, None)
    got = capi.w8a8_linear_codes(qtype, capi.quantize_act_static(qtype, x, one), one, qw, s, None)
    np.testing.assert_array_equal(_bits(got), _bits(want))


def test_captured_and_on_another_stream(capi):
    """A captured norm replays on new inputs, on a stream that is not the default one."""
    M, K = 64, 1024
    x, r, w = _rows(M, K, "graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        tx, tr, tw = _dev(x), _dev(r), _dev(w)
        h, q, s = torch.empty_like(tx), torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda")
        capi.qlin_rmsnorm_quant("e4m3", tx, tr, tw, EPS, None, h, q, s)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            capi.qlin_rmsnorm_quant("e4m3", tx, tr, tw, EPS, None, h, q, s)
        x2, r2, _ = _rows(M, K, "graph2")
        tx.copy_(_dev(x2))
        tr.copy_(_dev(r2))
        graph.replay()
    side.synchronize()
    _, y = ref.norm(x2, r2, w, EPS)
    sc = ref.row_scales(y, "e4m3")
    np.testing.assert_array_equal(s.cpu().numpy(), sc)
    np.testing.assert_array_equal(q.cpu().numpy(), ref.codes(y, sc[:, None], "e4m3"))
