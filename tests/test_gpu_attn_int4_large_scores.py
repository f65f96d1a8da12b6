"""Attention over the 4-bit cache with scores at and beyond the end of binary32's integers (GPU).  There a reference
cannot be moved by a few units: the weights come from differences of scores, which are exact near the largest one."""
import numpy as np
import pytest
import torch

import _int4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


# head size, new tokens, positions, sequences, kv heads: few rows in one step a warp, in several, many rows
FEW = [(D, nq, 400, 2, 2) for D in (32, 64, 128, 256) for nq in (1, 4)]
LONG = [(D, 1, 640, 32, 8) for D in (64, 256)] + [(128, 2, 640, 32, 8)]
MANY = [(D, 300, 400, 2, 2) for D in (64, 128, 256)]


def _case(capi, D, nq, kv, B, H, G=4, seed=0):
    a = ref.Attn4([nq] * B, [kv] * B, H, G, D, 16, seed=D + nq + seed)
    name = capi.qlin_attn_int4_kernel_name(B, H * G, H, D, nq, kv)
    assert ("k_attn_prefill" in name) == (nq > 100), name
    return a


def _run(capi, a, **kw):
    out = capi.attn_int4(a.q.cuda(), a.q_start.cuda(), a.kv_len.cuda(), a.table.cuda(), [t.cuda() for t in a.cache()],
                         max(a.nq), max(a.kv), **kw)
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    return out.float().cpu().double()


def _values(a, b):
    """[kv, H, D] of sequence b."""
    page, off = a.place(b, torch.arange(a.kv[b]))
    return a.vcode[page, :, off].double() * a.vs[page, :, off].double().repeat_interleave(32, dim=-1)


def _per_row(a, weights):
    """Outputs and tolerance where the row of new token i of sequence b has weights(b)[i] [kv] (which add up to 1),
    whatever its head: the output's rounding, those of P and of a scaled value (2^-11 of each term), binary32 sums
    and exponentials, and half of float16's smallest step beside a largest P of 2^8."""
    out, tol = [], []
    for b, (n, m) in enumerate(zip(a.nq, a.kv)):
        v, p = _values(a, b), weights(b)
        o, w = ((p @ x.reshape(m, -1)).view(n, a.H, 1, a.D).expand(n, a.H, a.G, a.D).reshape(n, -1)
                for x in (v, v.abs()))
        out.append(o)
        tol.append(2.0 ** -8 * o.abs() + w * (2 * 2.0 ** -11 + 2.0 ** -18) + m * 2.0 ** -33 * float(v.abs().max()))
    return torch.cat(out), torch.cat(tol)


def _seen(n, m):
    return (torch.arange(m) <= torch.arange(m - n, m)[:, None]).double()


@pytest.mark.parametrize("D,nq,kv,B,H", FEW + LONG + MANY)
@pytest.mark.parametrize("lift", [1.0] + [2.0 ** e for e in range(18, 28)] + [-2.0 ** 25, 2.0 ** 60])
def test_equal_scores(capi, D, nq, kv, B, H, lift):
    """Every key the same: a row's scores are equal, of sizes all over the band, and its output is the mean of what it
    sees."""
    a = _case(capi, D, nq, kv, B, H)
    a.kcode[:] = torch.where(torch.arange(D) % 3 == 0, -5, 6).to(torch.int8)
    a.ks[a.ks.isfinite()] = 0.5
    a.q *= lift
    want, tol = _per_row(a, lambda b: (lambda s: s / s.sum(1, keepdim=True))(_seen(nq, kv)))
    assert ((_run(capi, a) - want).abs() <= tol).all()


def _scale_of(power):
    """A softmax scale that, times log2(e), is 2^power in binary32."""
    to, log2e = np.float32(2.0 ** power), np.float32(1.44269504088896341)
    s = np.float32(to / log2e)
    for x in (s, np.nextafter(s, np.float32(0)), np.nextafter(s, np.float32(np.inf))):
        if x * log2e == to:
            return float(x)
    raise AssertionError(power)


@pytest.mark.parametrize("D,nq,kv,B,H", [c for c in FEW + LONG + MANY if c[0] > 32])
@pytest.mark.parametrize("step,base", [(1, 0), (7, 20), (9, 20), (8, 22), (8, 23), (8, 24), (8, 25), (8, 26), (16, 27)])
@pytest.mark.parametrize("order", ["up", "mixed"])
def test_steps(capi, D, nq, kv, B, H, step, base, order):
    """Scores (base 2) that are whole numbers of 2^base and more, c * step apart: c is 0 to 7 along the positions.  All
    are binary32 numbers, so the weights are powers of two that the formula gives exactly."""
    a = _case(capi, D, nq, kv, B, H, G=1 if nq == 1 else 4)
    g = torch.Generator().manual_seed(base)
    a.kcode[:], a.q[:] = 0, 0
    a.ks[a.ks.isfinite()] = 8192.0
    q = a.q.view(-1, H * a.G, D)
    if base:  # dimension 0: 7 * 8192 * q in [2^base, 2^(base + 1)), of either sign; dimension 32: c * step
        q[..., 0] = 2.0 ** (base - 22) * torch.randint(74, 147, q.shape[:2], generator=g)  # times 7: 518 to 1022
        q[::2, :, 0] *= -1
    q[..., 32] = step / 8.0
    c = torch.arange(kv) * 8 // kv
    if order == "mixed":
        c = c[torch.randperm(kv, generator=g)]
    for b in range(B):
        page, off = a.place(b, torch.arange(kv))
        a.kcode[page, :, off, 0] = 7
        a.kcode[page, :, off, 32] = c[:, None].to(torch.int8)
        a.ks[page, :, off, 1] = 8.0
    w = _seen(nq, kv) * 2.0 ** (c.double() * step)
    want, tol = _per_row(a, lambda b: w / w.sum(1, keepdim=True))
    assert ((_run(capi, a, scale=_scale_of(0)) - want).abs() <= tol).all()


def _near(out, want, a):
    """Means of values: the output's rounding, those of P and of values to float16 (2^-11 of the largest), binary32 sums."""
    sizes = torch.cat([_values(a, b).abs().amax(0).repeat_interleave(a.G, dim=0).reshape(1, -1).expand(n, -1)
                       for b, n in enumerate(a.nq)])
    assert ((out - want).abs() <= 2.0 ** -8 * want.abs() + sizes * (2 * 2.0 ** -11 + 2.0 ** -18)).all()


@pytest.mark.parametrize("D,nq,kv,B,H", FEW + MANY)
@pytest.mark.parametrize("lift", [2.0 ** 20, 2.0 ** 22, 2.0 ** 24, 2.0 ** 30, 2.0 ** 50])
def test_the_largest_score_takes_all(capi, D, nq, kv, B, H, lift):
    """Keys of random signs: the best positions of a row lead by far more than any rounding of their score."""
    a = _case(capi, D, nq, kv, B, H, seed=1)
    a.ks[a.ks.isfinite()] = 0.5
    a.kcode[:] = torch.where(a.kcode >= 0, 3, -3).to(torch.int8)
    a.q[:] = torch.where(a.q >= 0, 1.0, -1.0)  # scores are multiples of 3/4, exact sums: ties among the best
    a.q += torch.randint(0, 2, a.q.shape, generator=torch.Generator().manual_seed(D)) * 0.5
    limit, _ = a.reference(scale=4096.0)  # all weight on the best
    a.q *= lift
    _near(_run(capi, a, scale=1.0), limit, a)


@pytest.mark.parametrize("D,nq,kv,B,H", FEW + MANY)
@pytest.mark.parametrize("e", [118, 121, 124, 126])
@pytest.mark.parametrize("sign", [1, -1])
def test_largest_queries(capi, D, nq, kv, B, H, e, sign):
    """Rows of q up to the end of BF16's range beside ordinary ones, under key scales that leave their scores binary32
    numbers: the best positions take all, the first ones with keys of zeros, whose scores are 0, among them."""
    a = _case(capi, D, nq, kv, B, H, seed=2)
    a.ks[a.ks.isfinite()] = 2.0 ** -24
    a.kcode[:] = torch.where(a.kcode >= 0, 3, -3).to(torch.int8)
    for b in range(B):
        page, off = a.place(b, torch.arange(kv // 8))
        a.kcode[page, :, off] = 0
    q = torch.where(a.q >= 0, 1.0, -1.0).view(-1, H * 4, D)
    q[:, 1] = 0  # all scores 0
    small = q.clone()
    small[:, 2::4] *= 2.0 ** -60  # of nearly no score
    a.q = small.view(a.q.shape).bfloat16()
    big = (q * 2.0 ** torch.tensor([e, e, -60, e - 3.0])[torch.arange(H * 4) % 4][:, None]).view(a.q.shape).bfloat16()
    want, _ = a.reference(scale=sign * 2.0 ** 40)  # all weight on the best, or none
    a.q = big
    _near(_run(capi, a, scale=sign * D ** -0.5), want, a)
