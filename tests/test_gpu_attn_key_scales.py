"""Attention over many rows with key scales far apart (GPU): the scale of a position that a
row does not see, whatever it is, leaves that row's scores within their own tolerance."""
import pytest
import torch

import _layer_ref as ref
from test_gpu_attn import _check, _run

pytestmark = pytest.mark.gpu
EXTREMES = [65504.0, float("inf"), float("nan")]


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _many(capi, a, window=0):
    name = capi.qlin_attn_mixed_kernel_name(len(a.nq), a.H * a.G, a.H, a.D, max(a.nq), max(a.kv), window)
    assert "k_attn_prefill" in name, name


def chunk(D, seed, nq=200, kv=400, up=1.0, G=4, **kw):
    """One chunk and a short second sequence; key scales near 0.025 * up, q up to the same score."""
    a = ref.Attn([nq, 150], [kv, 170], 1, G, D, 16, seed=seed, spread=0.3, q_scale=2.0 / up, **kw)
    a.ks *= up
    return a


def blind(a, position, window=0):
    """Which rows do not see a position of the first sequence (the second sequence's among them)."""
    tok = torch.arange(a.nq[0]) + a.kv[0] - a.nq[0]
    out = torch.ones(sum(a.nq), dtype=torch.bool)
    out[: a.nq[0]] = (tok < position) | ((tok >= position + window) if window else False)
    return out


def _check_blind(capi, a, position, value, window=0):
    want, tol = a.reference(window=window)
    hidden = blind(a, position, window)
    assert hidden[: a.nq[0]].any() and not hidden.all()
    a.ks[a.slots(0)[position]] = value
    _many(capi, a, window)
    out = _run(capi, a, window=window)
    assert ((out - want).abs() <= tol)[hidden].all()
    if value == 65504.0:
        _check(out, a, window=window)
    else:
        assert torch.isnan(out[~hidden]).all()


@pytest.mark.parametrize("value", EXTREMES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("up", [1.0, 0.2])
@pytest.mark.parametrize("position", [399, 341, 210])
def test_later_rows_alone_see_it(capi, D, up, position, value):
    _check_blind(capi, chunk(D, D + position, up=up), position, value)


@pytest.mark.parametrize("value", EXTREMES)
@pytest.mark.parametrize("D", [64, 128])
def test_earlier_rows_of_a_window_alone_see_it(capi, D, value):
    _check_blind(capi, chunk(D, D, nq=200, kv=600), 420, value, window=100)


@pytest.mark.parametrize("value", EXTREMES)
@pytest.mark.parametrize("D", [64, 128])
def test_split_positions(capi, D, value):
    """Positions split over CTAs: the ones before the unit, and the one that holds it."""
    a = ref.Attn([90], [6000], 1, 7, D, 64, seed=D, spread=0.3)
    want, tol = a.reference()
    a.ks[a.slots(0)[5950]] = value
    name = capi.qlin_attn_mixed_kernel_name(1, 7, 1, D, 90, 6000)
    assert "k_attn_prefill+k_attn_join" in name, name
    out = _run(capi, a)
    assert ((out - want).abs() <= tol)[:40].all()
    if value == 65504.0:
        _check(out, a)
    else:
        assert torch.isnan(out[40:]).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [0, 1])
def test_one_group_of_one_key(capi, D, value, group):
    a = chunk(D, D + group)
    want, tol = a.reference()
    a.ks[a.slots(0)[300], 0, group] = value
    _many(capi, a)
    out = _run(capi, a)
    hidden = blind(a, 300)
    assert ((out - want).abs() <= tol)[hidden].all()
    assert torch.isnan(out[~hidden]).all()


@pytest.mark.parametrize("scale", [None, -0.05, 0.0])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_over_the_range(capi, D, scale):
    """Every position its own power of two, 2^20 from the smallest to the largest, seen by all rows."""
    a = ref.Attn([130, 150], [333, 170], 2, 4, D, 16, seed=D + 3, spread=0.3, q_scale=0.01)
    e = torch.randint(-14, 7, (a.ks.shape[0], 1, 1), generator=torch.Generator().manual_seed(D))
    a.ks = (a.ks.float() * 2.0 ** e).half()
    _many(capi, a)
    kw = {} if scale is None else {"scale": scale}
    _check(_run(capi, a, **kw), a, **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_keys_and_values_far_apart_together(capi, D):
    """Units with an exponent for each position in both, and units with one in either."""
    a = ref.Attn([130, 150], [700, 170], 1, 4, D, 16, seed=D + 4, spread=0.3, q_scale=0.05)
    s = a.slots(0)
    a.ks[s[100:400:9]] *= 2.0 ** -12
    a.ks[s[250]] *= 2.0 ** 6
    a.vs[s[200:500:7]] *= 2.0 ** -12
    a.vs[s[5::50]] *= 2.0 ** 9
    _many(capi, a)
    _check(_run(capi, a), a)
