"""Normalised query heads at the ends of the range: infinities and NaN, squares beyond and below binary32, as the
binary32 steps of the formula have them (GPU)."""
import numpy as np
import pytest
import torch

import _int4_ref as ref
from _layer_ref import bf16_round
from bit_quantized_linear_gb300 import synth

pytestmark = pytest.mark.gpu
SHAPES = [(64, 64), (64, 32), (64, 0), (80, 48), (128, 128), (128, 32), (256, 64), (512, 512), (16, 16), (32, 16)]


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _dev(a):
    return torch.from_numpy(synth.f32_to_bf16_bits(a).view(np.int16)).cuda().view(torch.bfloat16)


def _host(t):
    return synth.bf16_bits_to_f32(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def _rand(shape, seed):
    return np.random.default_rng(seed).standard_normal(shape).astype(np.float32)


def _check(capi, x, D, rot, layout, eps, store):
    """x [T, heads, D]: the outputs of q, by either entry point, against the binary32 steps: the same infinities and
    NaN, and half a BF16 step and 2^-19 of the two products apart at most (2^-134 below BF16's normal range).
    (The root mean square is off by 2^-20.4 at most, the products and their sum by four roundings of 2^-24; the
    steps themselves by three.)"""
    T, heads, _ = x.shape
    x = bf16_round(x)
    w = bf16_round(1 + np.float32(0.3) * _rand(D, 1))
    table = capi.rope_table(T, rot) if rot else None
    pos = torch.arange(T)
    q = torch.empty(T, heads * D, dtype=torch.bfloat16, device="cuda")
    args = layout, heads
    dx, dw = _dev(x.reshape(T, -1)), _dev(w)
    if store:
        cache = capi.kv_int4_alloc(1, T, 1, D)
        capi.qlin_qk_norm_rope_kv_store_int4(*args, rot, table, pos.cuda(), dx, dx[:, :D], dx[:, :D], dw, dw, eps, q,
                                             pos.cuda(), *cache)
    else:
        capi.qlin_qk_norm_rope(*args, 0, D, rot, table, pos.cuda(), dx, None, dw, None, eps, q, None)
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    with np.errstate(all="ignore"):
        y = ref.head_norm(x, w, eps).astype(np.float64)
        want, size = y.copy(), np.abs(y)
        if rot:
            t = table.cpu().numpy().astype(np.float64)
            r = rot // 2
            c, s = t[:, None, :r], t[:, None, r:]
            at = (slice(0, r), slice(r, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
            a, b = y[..., at[0]], y[..., at[1]]
            want[..., at[0]], want[..., at[1]] = a * c - b * s, b * c + a * s
            size[..., at[0]], size[..., at[1]] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
        got = _host(q).reshape(want.shape).astype(np.float64)
        top = np.float64(2.0 ** 128 - 2.0 ** 119)  # rounds to infinity from here on
        wild = ~np.isfinite(want) | (np.abs(want) > top * (1 - 2.0 ** -18))
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        far = np.isinf(want)
        np.testing.assert_array_equal(got[far], want[far])
        over = (np.abs(got - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -134))[~wild]
        assert over.size == 0 or over.max() <= 0, f"{int((over > 0).sum())} elements off, by up to {over.max()}"


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("what", [np.inf, -np.inf])
def test_one_infinity(capi, layout, D, rot, what):
    """A head's infinity makes its other elements 0, and what is turned with it NaN: past the rotation nothing."""
    for store in (False, True) if D in (32, 64, 128, 256) else (False,):
        x = _rand((D, 3, D), D + rot)
        for d in range(D):  # token d: element d of one head
            x[d, d % 3, d] = what
        _check(capi, x, D, rot, layout, 1e-6, store)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-24, 1e-30, 1.5e-38, 1e-44])
def test_all_magnitudes(capi, layout, D, rot, eps):
    """Heads from BF16's smallest numbers to its largest, alone and one large element among small ones; zeros, NaN."""
    e = np.concatenate([np.arange(-133, 127, 5), [-76, -75, -74, -63, -62, -60, -42, -41, -40, 58, 60, 61, 62, 63, 64, 126]])
    T = 2 * len(e) + 3
    x = np.empty((T, 5, D), dtype=np.float32)
    x[:] = np.clip(_rand((T, 5, D), D), -1.9, 1.9)
    with np.errstate(all="ignore"):
        for i, k in enumerate(e):
            x[i] = (x[i].astype(np.float64) * 2.0 ** float(k)).astype(np.float32)
            if i % 2:
                x[i, ::2] = x[i, ::2] * np.float32(2.0 ** -7)  # heads of other sizes beside them
            x[len(e) + i, 1, i % D] = np.float32(2.0 ** float(k))
            x[len(e) + i, 4] = np.float32(2.0 ** max(-140.0, float(k) - 9)) * np.sign(x[len(e) + i, 4])
    x[-3, 2] = 0
    x[-2] = 0
    x[-1, 3, D // 2] = np.nan
    for store in (False, True) if D in (32, 64, 128, 256) else (False,):
        _check(capi, x, D, rot, layout, eps, store)
