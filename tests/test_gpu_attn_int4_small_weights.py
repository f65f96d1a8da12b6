"""Attention over the 4-bit cache where one position takes nearly all the weight and has no value, as the first of a
context often does: the outputs are those of the others' small weights (GPU).  Few rows and many hold them to the
same precision."""
import math

import pytest
import torch

import _int4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


@pytest.mark.parametrize("D,nq,kv,H,G", [(64, 1, 700, 2, 4), (128, 1, 3000, 2, 4), (256, 1, 700, 2, 4), (128, 6, 700, 2, 4),
                                         (32, 3, 700, 2, 4), (64, 400, 700, 2, 4), (128, 300, 700, 2, 4),
                                         (128, 600, 3000, 1, 4), (256, 400, 700, 2, 4)])
@pytest.mark.parametrize("where", ["first", "last"])
def test_a_heavy_position_without_a_value(capi, D, nq, kv, H, G, where):
    """q and keys are 0 but in one dimension, and there such that a row's other positions have equal weights from 2^-20 to
    2^-27 of the heavy one's, rounded alike if they are rounded.  Every other value is positive, 7 times a scale that
    varies, so their errors add up.

    The tolerance counts the output's rounding (2^-8), those of P and of a scaled value to float16 (2^-11 each),
    2^-18 for sums, exponentials and the binary32 score (below 20), and half of float16's smallest step beside a P of 2^8
    for each position, 2^-33.  The keys, 7 and 0, lose nothing."""
    a = ref.Attn4([nq], [kv], H, G, D, 16, seed=D + nq)
    many = "k_attn_unpack4" in capi.qlin_attn_int4_kernel_name(1, H * G, H, D, nq, kv)
    assert many == (nq > 100)
    page, off = a.place(0, torch.arange(kv))
    heavy = 0 if where == "first" else kv - nq  # seen by every row
    a.kcode[:], a.vcode[:] = 0, 7
    a.kcode[page[heavy], :, off[heavy], 5] = 7
    a.vcode[page[heavy], :, off[heavy]] = 0
    a.ks[a.ks.isfinite()] = 1.0
    g = torch.Generator().manual_seed(nq)
    lead = (20 + 7 * torch.rand(nq, H * G, generator=g)) * math.log(2.0)  # of the heavy position's score
    a.q[:] = 0
    a.q.view(nq, H * G, D)[..., 5] = (lead / 7).bfloat16()
    lead = a.q.view(nq, H * G, D)[..., 5].double() * 7
    out = capi.attn_int4(a.q.cuda(), a.q_start.cuda(), a.kv_len.cuda(), a.table.cuda(), [t.cuda() for t in a.cache()],
                         nq, kv, scale=1.0).float().cpu().double().view(nq, H, G, D)
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    v = a.vcode[page, :, off].double() * a.vs[page, :, off].double().repeat_interleave(32, dim=-1)  # [kv, H, D]
    see = (torch.arange(kv) <= torch.arange(kv - nq, kv)[:, None]).double()
    others = see.clone()
    others[:, heavy] = 0
    w = torch.exp(-lead).view(nq, H, G, 1)
    want = w * torch.einsum("nk,khd->nhd", others, v)[:, :, None] / (1 + w * others.sum(1).view(nq, 1, 1, 1))
    small = torch.einsum("nk,khd->nhd", others, v)[:, :, None] * 2.0 ** -33
    tol = want * (2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -18) + small
    over = ((out - want).abs() / tol).max()
    assert over <= 1, f"up to {float(over)} of the tolerance"
