"""Attention over scales and query rows of all magnitudes, outputs below BF16's normal range
among them (GPU).  A rounding to BF16 is off by at most 2^-8 of the value, and by at most 2^-134,
half of the smallest subnormal, where the value is below the normal range."""
import pytest
import torch

import _layer_ref as ref
from test_gpu_attn import _run

pytestmark = pytest.mark.gpu
CASES = [(D, (200, 300), (333, 300)) for D in (64, 128)] + [(D, (3, 5), (333, 300)) for D in (32, 64, 128, 256)]


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def magnitudes(D, nq, kv):
    a = ref.Attn(nq, kv, 2, 4, D, 16, seed=100 + D, spread=2.5, q_scale=0.5)
    a.vs[::5] *= 2.0 ** -9
    a.vs[::7] = 2.0 ** 9
    a.vs[3::11] = 0
    a.ks[::3] *= 2.0 ** -8
    for t in range(a.q.shape[0]):
        a.q[t] *= [1.0, 2.0 ** -60, 2.0 ** 3, 0.0][t % 4]
    return a


@pytest.mark.parametrize("D,nq,kv", CASES)
@pytest.mark.parametrize("scale", [None, -0.05, 0.0])
def test_magnitudes(capi, D, nq, kv, scale):
    a = magnitudes(D, nq, kv)
    kw = {} if scale is None else {"scale": scale}
    want, tol = a.reference(**kw)
    out = _run(capi, a, **kw)
    assert ((out - want).abs() <= tol + 2.0 ** -134).all()
