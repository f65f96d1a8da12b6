"""Attention with scores far beyond binary32's integers (GPU).  Scores that differ, differ by
much there, and scores that are equal still share the sum: the outputs stay what they are."""
import pytest
import torch

import _layer_ref as ref
from test_gpu_attn import _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


MANY = [(D, 200, 400) for D in (64, 128)]
FEW = [(D, nq, 400) for D in (32, 64, 128, 256) for nq in (1, 4)]


def _case(capi, D, nq, kv, seed=0, **kw):
    a = ref.Attn([nq, min(nq, 40)], [kv, 60], 2, 4, D, 16, seed=D + nq + seed, **kw)
    name = capi.qlin_attn_mixed_kernel_name(2, 8, 2, D, nq, kv)
    assert ("k_attn_prefill" in name) == (nq > 100), name
    return a


def equal_keys(a, lift):
    """Every key the same, so that a row's scores are equal; returns the mean of what each row sees and the
    tolerance of that: the output's rounding, those of P and of a scaled value, and binary32 sums."""
    a.kc[:] = torch.where(torch.arange(a.D) % 3 == 0, -50, 100).to(torch.int8)
    a.ks[:] = 0.5
    a.q *= lift
    out, tol, at = [], [], 0
    for b, (n, m) in enumerate(zip(a.nq, a.kv)):
        s = a.slots(b)
        v = a.vc[s].view(ref.F8).double() * a.vs[s].double()[..., None]
        count = torch.arange(m - n + 1, m + 1, dtype=torch.float64)
        mean = [x.cumsum(0)[m - n:] / count[:, None, None] for x in (v, v.abs())]
        o, w = (x.repeat_interleave(a.G, dim=1).reshape(n, -1) for x in mean)
        out.append(o)
        tol.append(2.0 ** -8 * o.abs() + w * (2 * 2.0 ** -11 + 2.0 ** -18))
        at += n
    return torch.cat(out), torch.cat(tol)


@pytest.mark.parametrize("D,nq,kv", MANY + FEW)
@pytest.mark.parametrize("lift", [1.0, 2.0 ** 14, 2.0 ** 26, 2.0 ** 60, -2.0 ** 40])
def test_equal_scores(capi, D, nq, kv, lift):
    a = _case(capi, D, nq, kv)
    want, tol = equal_keys(a, lift)
    assert ((_run(capi, a) - want).abs() <= tol).all()


@pytest.mark.parametrize("D,nq,kv", MANY + FEW)
def test_equal_scores_of_values_far_apart(capi, D, nq, kv):
    """The forms with an exponent for each position."""
    a = _case(capi, D, nq, kv)
    a.vs[::5] *= 2.0 ** -12
    a.vs[::7] *= 2.0 ** 9
    a.vs[3::11] = 0
    want, tol = equal_keys(a, 2.0 ** 26)
    assert ((_run(capi, a) - want).abs() <= tol).all()


@pytest.mark.parametrize("D,nq,kv", MANY + FEW)
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("lift", [2.0 ** 20, 2.0 ** 24, 2.0 ** 30, 2.0 ** 50])
def test_the_largest_score_takes_all(capi, D, nq, kv, far, lift):
    """Keys of random signs: the best position of a row leads by far more than any rounding of its score."""
    a = _case(capi, D, nq, kv, seed=1, spread=0.3)
    a.ks[:] = 0.5
    a.kc[:] = torch.where(a.kc >= 0, 3, -3).to(torch.int8)
    a.q[:] = torch.where(a.q >= 0, 1.0, -1.0)  # scores are multiples of 3: ties among the best
    a.q += torch.randint(0, 2, a.q.shape, generator=torch.Generator().manual_seed(D)) * 0.5
    if far:
        a.vs[::5] *= 2.0 ** -12
        a.vs[::7] *= 2.0 ** 9
    want, _ = a.reference()
    small, _ = (a.reference(scale=4096.0))  # the limit: all weight on the best
    a.q *= lift
    out = _run(capi, a, scale=1.0)
    assert torch.isfinite(out).all()
    # ties give the mean of the tied values in both; the rounding of P and values, and of the output
    sizes = torch.cat([(a.vc[a.slots(b)].view(ref.F8).double() * a.vs[a.slots(b)].double()[..., None]).abs().amax(0)
                       .repeat_interleave(a.G, dim=0).reshape(1, -1).expand(n, -1)
                       for b, n in enumerate(a.nq)])
    tol = 2.0 ** -8 * small.abs() + sizes * (2 * 2.0 ** -11 + 2.0 ** -18)
    assert ((out - small).abs() <= tol).all()


@pytest.mark.parametrize("D,nq,kv", MANY + FEW)
def test_keys_at_the_top_of_the_range(capi, D, nq, kv):
    a = _case(capi, D, nq, kv, seed=2, spread=0.3)
    a.ks[::3] = 65504.0
    a.q *= 64.0
    _check(_run(capi, a), a)
