"""Attention over few rows with value scales far apart (GPU): what a row does not see, or
gives no weight, leaves its outputs within the tolerance of the others' own scales."""
import pytest
import torch

import _layer_ref as ref
from test_gpu_attn import _check, _run

pytestmark = pytest.mark.gpu
SIZES = [32, 64, 128, 256]
EXTREMES = [65504.0, float("inf"), float("nan")]


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _few(capi, a, window=0):
    name = capi.qlin_attn_mixed_kernel_name(len(a.nq), a.H * a.G, a.H, a.D, max(a.nq), max(a.kv), window)
    assert name.startswith("k_attn_split"), name


def small(D, nq, kv, seed, G=4, **kw):
    """Value scales near 2^-12: below the largest by 2^28."""
    a = ref.Attn([nq, 2], [kv, 40], 1, G, D, 16, seed=seed, spread=0.3, **kw)
    a.vs *= 2.0 ** -5
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
    a.vs[a.slots(0)[position]] = value
    _few(capi, a, window)
    out = _run(capi, a, window=window)
    assert ((out - want).abs() <= tol)[hidden].all()
    if value == 65504.0:
        _check(out, a, window=window)
    else:
        assert not torch.isfinite(out[~hidden]).all(1).any()


@pytest.mark.parametrize("value", EXTREMES)
@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("nq,kv,position", [(6, 150, 147), (2, 40, 39), (16, 520, 505)])
def test_later_rows_alone_see_it(capi, D, nq, kv, position, value):
    _check_blind(capi, small(D, nq, kv, D + nq), position, value)


@pytest.mark.parametrize("value", EXTREMES)
@pytest.mark.parametrize("D", SIZES)
def test_earlier_rows_of_a_window_alone_see_it(capi, D, value):
    """The position is in the first tile of its warp, and has left the later rows' windows."""
    _check_blind(capi, small(D, 6, 700, D), 700 - 6 - 299, value, window=300)


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("nq,kv,position", [(1, 300, 3), (1, 300, 290), (5, 9000, 4000)])
def test_a_large_value_without_weight(capi, D, nq, kv, position):
    """Every row sees it, and its score is so low that it adds nothing."""
    a = small(D, nq, kv, D + kv)
    a.q[:] = a.q[0, :D].repeat(a.G)
    s = a.slots(0)[position]
    a.vs[s] = 65504.0
    a.kc[s] = torch.where(a.q[0, :D].float() > 0, -100, 100).to(torch.int8)[None]
    a.ks[s] = 8.0
    _few(capi, a)
    _check(_run(capi, a), a)


def far_apart(D, kv=333):
    """Scales over float16's range within one sequence, rows from tiny to large, positions without a value; the
    outputs stay in bfloat16's normal range."""
    a = ref.Attn([3, 4], [kv, 300], 2, 4, D, 16, seed=D + 1, spread=2.5, q_scale=0.01)
    a.ks.clamp_(max=8.0)
    a.vs[::5] *= 2.0 ** -9
    a.vs[::7] = 2.0 ** 9
    a.vs[3::11] = 0
    a.ks[::3] *= 2.0 ** -8
    for t in range(a.q.shape[0]):
        a.q[t] *= [1.0, 2.0 ** -60, 2.0, 0.0][t % 4]
    return a


@pytest.mark.parametrize("scale", [None, -0.05, 0.0])
@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("kv", [333, 6000])
def test_scales_far_apart(capi, D, kv, scale):
    a = far_apart(D, kv)
    _few(capi, a)
    kw = {} if scale is None else {"scale": scale}
    _check(_run(capi, a, **kw), a, **kw)


def lead(D, kv, up):
    """Every eleventh position has no value, and its key, the row's own direction, outscores all others by far."""
    a = ref.Attn([2], [kv], 1, 4, D, 16, seed=D + 2, q_scale=0.05)
    a.q[:] = a.q[0, :D].repeat(a.G)
    s = a.slots(0)[3::11]
    a.vs[s] = 0
    a.kc[s] = torch.where(a.q[0, :D].float() > 0, 100, -100).to(torch.int8)[None, None]
    a.ks[s] = up
    return a


@pytest.mark.parametrize("up", [0.25, 1.0])
@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("kv", [5, 400, 5000])
def test_scores_without_a_value(capi, D, kv, up):
    """They count in the sum, and leave what the others give in place though it is small."""
    a = lead(D, kv, up)
    _few(capi, a)
    _check(_run(capi, a), a)


@pytest.mark.parametrize("D", SIZES)
def test_no_value_at_all(capi, D):
    a = ref.Attn([3, 1], [70, 9000], 1, 4, D, 16, seed=D)
    a.vs[:] = 0
    _few(capi, a)
    assert (_run(capi, a) == 0).all()


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("nq", [1, 5])
def test_scales_that_rise_and_fall(capi, D, nq):
    """From tile to tile the scales move over float16's range and back: one exponent for each tile."""
    a = ref.Attn([nq], [1200], 1, 4, D, 128, seed=D, spread=0.3)
    s = a.slots(0)
    j = torch.arange(1200)
    a.vs[s] = (a.vs[s].float() * (2.0 ** (10 * torch.sin(j / 190.0)))[:, None]).half()
    _few(capi, a)
    _check(_run(capi, a), a)
