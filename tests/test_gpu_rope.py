"""Rotary positions, alone and with the store into the mixed KV cache (GPU).

The rotation is a fixed sequence of binary32 operations on the table's values, so
it is compared bit for bit; the table is compared with the 64-bit formula."""
import numpy as np
import pytest
import torch

import _layer_ref as ref
from bit_quantized_linear_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _dev(a):
    return torch.from_numpy(synth.f32_to_bf16_bits(a).view(np.int16)).cuda().view(torch.bfloat16)


def _host(t):
    return synth.bf16_bits_to_f32(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def _rand(shape, *tag):
    rng = synth.rng_for("test-rope", 0, str(shape), "/".join(map(str, tag)))
    return ref.bf16_round(rng.standard_normal(shape, dtype=np.float32))


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="by_parts", factor=4.0, original_context=4096.0),
            dict(scaling="by_parts", factor=32.0, original_context=2048.0, beta_fast=16.0, beta_slow=2.0)]


@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s.get("scaling", "plain"))
@pytest.mark.parametrize("rot,theta", [(16, 1e4), (64, 1e6), (128, 1e4)])
def test_table(capi, scaling, rot, theta):
    """Every value within one rounding to binary32 (2^-24 of it) and the error of a 64-bit angle of up to
    2^17 radians (its frequency is good to a few 2^-53: 2^-33 at most)."""
    n, amp = 70001, 1.1
    t = capi.rope_table(n, rot, theta, amplitude=amp, **scaling).cpu().numpy().astype(np.float64)
    f = ref.frequencies(rot, theta, **scaling)
    a = np.arange(n)[:, None] * f[None]
    want = np.concatenate([np.cos(a), np.sin(a)], axis=1) * amp
    assert np.all(np.abs(t - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -33)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 1, 1, 16, 16), (1, 28, 4, 128, 128), (5, 3, 0, 64, 32), (33, 16, 2, 128, 32),
                                           (7, 5, 2, 80, 48), (300, 4, 1, 256, 256), (2, 3, 3, 512, 496),
                                           (6000, 7, 1, 64, 64), (19, 8, 8, 32, 16), (4, 2, 1, 96, 96)])
def test_rotation(capi, layout, T, Hq, Hk, D, rot):
    n, m = Hq * D, Hk * D
    x = _rand((T, n + m + 24), layout, D, rot)
    dx = _dev(x)
    table = capi.rope_table(512, rot)
    pos = torch.randint(0, 512, (T,), generator=torch.Generator().manual_seed(T))
    rows = table.cpu().numpy()[pos.numpy()]
    want = ref.rope(x[:, : n + m].reshape(T, Hq + Hk, D), rows, rot, layout).reshape(T, n + m)
    q, k = dx[:, :n], dx[:, n: n + m] if Hk else None
    qo = torch.full((T, n + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.empty(T, m, dtype=torch.bfloat16, device="cuda") if Hk else None
    capi.qlin_rope(layout, Hq, Hk, D, rot, table, pos.cuda(), q, k, qo[:, :n], ko)
    np.testing.assert_array_equal(_host(qo[:, :n]), want[:, :n])
    assert (qo[:, n:] == 5).all()
    if Hk:
        np.testing.assert_array_equal(_host(ko), want[:, n:])
    np.testing.assert_array_equal(_host(dx), x)
    capi.qlin_rope(layout, Hq, Hk, D, rot, table, pos.cuda(), q, k, q, k)  # in place
    np.testing.assert_array_equal(_host(dx)[:, : n + m], want)
    np.testing.assert_array_equal(_host(dx)[:, n + m:], x[:, n + m:])
    assert capi.qlin_get_device_status() == capi.QLIN_OK


def test_skipped_positions(capi):
    """A negative position leaves its token; one beyond the table also sets the status."""
    T, Hq, D = 9, 2, 64
    x = _rand((T, Hq * D), "skip")
    table = capi.rope_table(100, D)
    pos = torch.arange(T) * 10
    pos[2], pos[5] = -1, -2 ** 40
    out = _dev(x * 0 + 3)
    capi.qlin_rope("half", Hq, 0, D, D, table, pos.cuda(), _dev(x), None, out, None)
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    want = ref.rope(x.reshape(T, Hq, D), table.cpu().numpy()[pos.clamp(min=0).numpy()], D, "half").reshape(T, -1)
    want[2] = want[5] = 3
    np.testing.assert_array_equal(_host(out), want)
    pos[7] = 100
    out = _dev(x * 0 + 3)
    capi.qlin_rope("half", Hq, 0, D, D, table, pos.cuda(), _dev(x), None, out, None)
    assert capi.qlin_get_device_status() == capi.QLIN_ERR_INVALID_ARG
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    want[7] = 3
    np.testing.assert_array_equal(_host(out), want)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,Hq,H,D,rot", [(1, 28, 4, 128, 128), (37, 16, 2, 128, 64), (5, 3, 1, 32, 16), (64, 8, 8, 64, 64),
                                          (21, 6, 3, 256, 112), (700, 10, 5, 32, 32), (3, 2, 2, 64, 48),
                                          (40, 4, 7, 128, 16)])
def test_store_is_rotation_then_store(capi, layout, T, Hq, H, D, rot):
    n, m = Hq * D, H * D
    x = _dev(_rand((T, n + 2 * m), layout, "store", D) * np.float32(3))
    if T > 4:
        x[2, n:] = 0
        x[3, n:] *= 1e6
    q, k, v = x.split([n, m, m], dim=1)
    S = 2 * T + 3
    table = capi.rope_table(4096, rot, scaling="linear", factor=2.0)
    g = torch.Generator().manual_seed(D + T)
    pos = torch.randint(0, 4096, (T,), generator=g).cuda()
    slots = torch.randperm(S, generator=g)[:T]
    if T > 4:
        slots[1] = -1
        pos[4] = -1
    slots = slots.cuda()
    caches = [capi.kv_cache_alloc(S, H, D) for _ in range(2)]
    for c in caches:
        for a in c:
            a.view(torch.uint8).fill_(0xA5)
    outs = [torch.full((T, n), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kr = torch.empty(T, m, dtype=torch.bfloat16, device="cuda")
    capi.qlin_rope(layout, Hq, H, D, rot, table, pos, q, k, outs[0], kr)
    both = slots.clone()
    both[pos < 0] = -1
    capi.qlin_kv_store_mixed(kr, v, both, *caches[0])
    capi.qlin_rope_kv_store_mixed(layout, Hq, rot, table, pos, q, k, v, outs[1], slots, *caches[1])
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    for a, b in zip(*caches):
        assert torch.equal(a, b)


def test_store_reports_bad_slots(capi):
    T, H, D = 6, 2, 64
    x = _dev(_rand((T, 3 * H * D), "bad"))
    q, k, v = x.split(H * D, dim=1)
    table = capi.rope_table(16, D)
    cache = capi.kv_cache_alloc(8, H, D)
    for a in cache:
        a.view(torch.uint8).fill_(0xA5)
    slots = torch.tensor([0, 1, 8, 3, 2 ** 50, 5]).cuda()
    out = torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
    capi.qlin_rope_kv_store_mixed("half", H, D, table, torch.arange(T).cuda(), q, k, v, out, slots, *cache)
    assert capi.qlin_get_device_status() == capi.QLIN_ERR_INVALID_ARG
    used = (cache[2].reshape(8, -1) != 0xA5).any(1).cpu()
    assert used.tolist() == [True, True, False, True, False, True, False, False]


def test_no_tokens(capi):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    capi.qlin_rope("half", 1, 1, 64, 64, capi.rope_table(4, 64), pos, e, e, e, e)
    assert capi.qlin_get_device_status() == capi.QLIN_OK
