"""Attention over many rows: tiles of the common loop and of the general one in turn (GPU)."""
import pytest
import torch

import _layer_ref as ref
from test_gpu_attn import _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _chunk(capi, D, seed, kv=2000, G=4):
    a = ref.Attn([150], [kv], 1, G, D, 16, seed=seed, spread=0.3, q_scale=0.05)
    a.q[:] = a.q[0, :D].repeat(a.G) * (1 + torch.arange(150)[:, None] % 3)  # rows of one direction
    assert capi.qlin_attn_mixed_kernel_name(1, G, 1, D, 150, kv).startswith("k_attn_unpack+k_attn_prefill")
    return a


def _lead(a, position, up, value):
    """The position's key is the rows' direction, `up` its scale: its score leads; `value`: of its scale."""
    s = a.slots(0)[position]
    a.kc[s] = torch.where(a.q[0, : a.D].float() > 0, 100, -100).to(torch.int8)[None]
    a.ks[s] = up
    a.vs[s] = value


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("positions", [(300,), (5, 1500), (1999,), (130, 131, 700, 1290)])
@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** -12, 0.0])
def test_value_scales(capi, D, positions, far):
    a = _chunk(capi, D, D + len(positions))
    for p in positions:
        a.vs[a.slots(0)[p]] *= far
    _check(_run(capi, a), a)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("up", [0.05, 0.5, 2.0])
@pytest.mark.parametrize("position", [3, 700, 1900])
def test_leads_without_a_value(capi, D, up, position):
    """Far enough ahead, the sum keeps a reference of its own to the end."""
    a = _chunk(capi, D, D + position)
    _lead(a, position, up, 0.0)
    _check(_run(capi, a), a)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("position", [3, 700, 1900])
@pytest.mark.parametrize("value", [None, 2.0 ** 4])
def test_huge_scores(capi, D, sign, position, value):
    """One key at the top of the range, for rows with a large q: its tile alone is taken as huge.  With it ahead a
    row is that position's value; with it behind it adds nothing."""
    a = _chunk(capi, D, D + position)
    a.q *= 2.0 ** 6
    s = a.slots(0)[position]
    _lead(a, position, 65504.0, a.vs[s].clone() if value is None else value)
    a.kc[s] = (sign * a.kc[s].float()).to(torch.int8)
    out = _run(capi, a)
    # the reference's tolerance would count scores of that size: rows that see a leading key are held to the
    # value itself, and others to the answer with a key whose score is just far enough behind
    sees = (torch.arange(150) + 1850 >= position) & (sign > 0)
    own = (a.vc[s].view(ref.F8).double() * a.vs[s].double()[..., None]).repeat(1, a.G).reshape(1, -1)
    assert ((out - own).abs() <= (2.0 ** -8 + 2 * 2.0 ** -11) * own.abs())[sees].all()
    a.kc[s] = (-a.kc[s].float().abs() * torch.sign(a.q[0, :D].float())).to(torch.int8)
    a.ks[s] = 4.0
    want, tol = a.reference()
    assert ((out - want).abs() <= tol)[~sees].all()


@pytest.mark.parametrize("D", [64, 128])
def test_all_in_one(capi, D):
    a = _chunk(capi, D, D)
    for p, f in ((40, 2.0 ** 12), (300, 0.0), (900, 2.0 ** -13), (1400, 2.0 ** 12)):
        a.vs[a.slots(0)[p]] *= f
    for p, f in ((600, 2.0 ** 10), (601, 2.0 ** -10), (1700, 2.0 ** -16)):
        a.ks[a.slots(0)[p]] *= f
    _lead(a, 1000, 0.3, 0.0)
    _check(_run(capi, a), a)
