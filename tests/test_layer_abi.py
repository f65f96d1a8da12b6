"""Refusals, sizes and names of the operators around the linears (RMSNorm, codes
linear, rotary positions, attention), on the host: no launch is reached."""
import ctypes

import pytest

P = ctypes.c_void_p
GOOD, ODD8, ODD2 = P(4096), P(4096 + 8), P(4096 + 2)


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import build
    build.build()
    from bit_quantized_linear_gb300 import capi as c
    return c


def _call(f, good, **change):
    args = dict(good)
    for k, v in change.items():
        assert k in args, k
        args[k] = v
    return f(*args.values())


NORM = dict(M=4, K=64, x=GOOD, ldx=64, res=GOOD, ldr=64, w=GOOD, eps=1e-6, h=GOOD, y=GOOD, stream=None)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(K=0), dict(K=24), dict(K=32784), dict(x=None), dict(x=ODD8), dict(ldx=56), dict(ldx=68),
    dict(res=None), dict(h=None), dict(ldr=32), dict(res=ODD8), dict(w=None), dict(w=ODD8), dict(h=ODD8),
    dict(y=None), dict(y=ODD2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))])
def test_rmsnorm_refusals(capi, change):
    L = capi.lib()
    assert _call(L.qlin_rmsnorm, NORM, **change) == capi.QLIN_ERR_INVALID_ARG
    quant = dict(qtype=1, **{k: v for k, v in NORM.items() if k not in ("h", "y", "stream")})
    quant.update(sx=None, h=GOOD, y=GOOD, xs=GOOD, stream=None)
    assert _call(L.qlin_rmsnorm_quant, quant, **change) == capi.QLIN_ERR_INVALID_ARG


def test_rmsnorm_quant_scale_refusals(capi):
    L, INV = capi.lib(), capi.QLIN_ERR_INVALID_ARG
    good = dict(qtype=1, M=4, K=64, x=GOOD, ldx=64, res=None, ldr=0, w=GOOD, eps=1e-6, sx=None, h=None, y=GOOD,
                xs=GOOD, stream=None)
    assert _call(L.qlin_rmsnorm_quant, good, qtype=2) == INV
    assert _call(L.qlin_rmsnorm_quant, good, xs=None) == INV             # neither scale
    assert _call(L.qlin_rmsnorm_quant, good, sx=GOOD) == INV             # both
    assert _call(L.qlin_rmsnorm_quant, good, sx=ODD2, xs=None) == INV
    assert _call(L.qlin_rmsnorm_quant, good, xs=ODD8) == INV


CODES = dict(qtype=0, M=4, K=64, N=64, qx=GOOD, xs=GOOD, per=1, qw=GOOD, ws=GOOD, bias=None, y=GOOD, work=GOOD,
             nwork=1 << 20, stream=None)


@pytest.mark.parametrize("change", [dict(qtype=5), dict(K=72), dict(N=40), dict(M=-1), dict(qx=None), dict(qx=ODD8),
                                    dict(xs=None), dict(xs=ODD2), dict(qw=None), dict(ws=None), dict(bias=ODD8),
                                    dict(y=None)])
def test_linear_codes_refusals(capi, change):
    assert _call(capi.lib().qlin_w8a8_linear_codes, CODES, **change) == capi.QLIN_ERR_INVALID_ARG


def test_linear_codes_workspace(capi):
    L = capi.lib()
    need = capi.qlin_workspace_bytes(capi.QLIN_OP_W8A8_LINEAR_CODES, "int8", 4, 64, 64)
    assert need >= 4 * 64 * 2
    assert capi.qlin_workspace_bytes(capi.QLIN_OP_W8A8_LINEAR_CODES, "e4m3", 4, 64, 64) == 0
    for change in (dict(work=None), dict(nwork=need - 1), dict(work=ODD8)):
        assert _call(L.qlin_w8a8_linear_codes, CODES, **change) == capi.QLIN_ERR_WORKSPACE


TABLE = dict(max_pos=64, rot=64, theta=1e4, scaling=3, factor=4.0, orig=4096.0, fast=32.0, slow=1.0, amp=1.0,
             table=GOOD, stream=None)


@pytest.mark.parametrize("change", [dict(max_pos=0), dict(rot=0), dict(rot=24), dict(rot=528), dict(theta=0.0),
                                    dict(theta=float("nan")), dict(scaling=4), dict(scaling=-1), dict(factor=0.0),
                                    dict(factor=float("inf")), dict(orig=0.0), dict(fast=1.0), dict(slow=-1.0),
                                    dict(amp=float("nan")), dict(table=None), dict(table=ODD8)])
def test_rope_table_refusals(capi, change):
    assert _call(capi.lib().qlin_rope_table, TABLE, **change) == capi.QLIN_ERR_INVALID_ARG


ROPE = dict(layout=0, T=4, Hq=4, Hk=2, D=64, rot=32, table=GOOD, max_pos=64, pos=GOOD, q=GOOD, ldq=256, k=GOOD,
            ldk=128, qo=P(8192), ldqo=256, ko=P(8192), ldko=128, stream=None)


@pytest.mark.parametrize("change", [
    dict(layout=2), dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(D=24), dict(D=528), dict(rot=0), dict(rot=24),
    dict(rot=80), dict(table=None), dict(table=ODD8), dict(max_pos=0), dict(pos=None), dict(pos=ODD8), dict(q=None),
    dict(q=ODD8), dict(ldq=248), dict(ldq=260), dict(k=None), dict(ldk=120), dict(qo=None), dict(ldqo=128),
    dict(ko=None), dict(ldko=64), dict(qo=GOOD, ldqo=264), dict(ko=GOOD, ldko=136)])
def test_rope_refusals(capi, change):
    assert _call(capi.lib().qlin_rope, ROPE, **change) == capi.QLIN_ERR_INVALID_ARG


STORE = dict(layout=1, T=4, Hq=4, H=2, D=64, rot=32, table=GOOD, max_pos=64, pos=GOOD, q=GOOD, ldq=256, k=GOOD,
             ldk=128, v=GOOD, ldv=128, qo=GOOD, ldqo=256, slots=GOOD, ns=64, kc=GOOD, ks=GOOD, vc=GOOD, vs=GOOD,
             stream=None)


@pytest.mark.parametrize("change", [
    dict(layout=-1), dict(D=96), dict(D=16), dict(H=0), dict(rot=72), dict(k=None), dict(ldk=64), dict(v=None),
    dict(v=ODD8), dict(ldv=132), dict(slots=None), dict(ns=-1), dict(kc=None), dict(ks=ODD8), dict(vc=None),
    dict(vs=None), dict(q=None), dict(ldqo=512)])
def test_rope_store_refusals(capi, change):
    assert _call(capi.lib().qlin_rope_kv_store_mixed, STORE, **change) == capi.QLIN_ERR_INVALID_ARG


ATTN = dict(B=2, T=2, Hq=8, H=2, D=64, q=GOOD, ldq=512, qs=GOOD, max_q=1, kv=GOOD, max_kv=64, bt=GOOD, mb=4, bs=16,
            ns=256, kc=GOOD, ks=GOOD, vc=GOOD, vs=GOOD, scale=0.125, causal=1, window=0, out=GOOD, ldo=512, ws=GOOD,
            nws=1 << 30, stream=None)


@pytest.mark.parametrize("change", [
    dict(B=-1), dict(T=-1), dict(Hq=7), dict(Hq=0), dict(H=0), dict(Hq=512, ldq=32768, ldo=32768), dict(D=96),
    dict(q=None), dict(q=ODD8), dict(ldq=504), dict(ldq=516), dict(qs=None), dict(qs=ODD2), dict(max_q=-1),
    dict(kv=None), dict(kv=ODD2), dict(max_kv=-1), dict(bt=None), dict(bt=ODD2), dict(mb=-1), dict(bs=0),
    dict(ns=250), dict(ns=-16), dict(kc=None), dict(ks=None), dict(vc=ODD8), dict(vs=None),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(window=-1), dict(out=None), dict(ldo=256)])
def test_attn_refusals(capi, change):
    assert _call(capi.lib().qlin_attn_mixed, ATTN, **change) == capi.QLIN_ERR_INVALID_ARG


def test_attn_workspace(capi):
    L = capi.lib()
    ws = capi.qlin_attn_mixed_workspace_bytes
    need = ws(1, 28, 4, 128, 1, 32768, 0)
    assert 0 < need < 1 << 26
    big = dict(ATTN, B=1, T=1, Hq=28, H=4, D=128, ldq=3584, ldo=3584, max_kv=32768, mb=2048, ns=32768)
    for change in (dict(ws=None), dict(ws=ODD8), dict(nws=need - 1)):
        assert _call(L.qlin_attn_mixed, big, **change) == capi.QLIN_ERR_WORKSPACE
    assert ws(1, 16, 2, 128, 1, 37, 0) == 0          # one part
    assert ws(0, 16, 2, 128, 1, 4096, 0) == 0
    assert ws(1, 16, 3, 128, 1, 4096, 0) == 2 ** 64 - 1
    # the partial results of any accepted sizes stay small beside the cache
    for B, q, kv in [(1, 1, 1 << 20), (256, 1, 4096), (3, 5, 100000), (1, 8192, 16384)]:
        assert ws(B, 16, 2, 128, q, kv, 0) <= max(1 << 26, B * kv * 2 * 256 // 4)


def test_attn_kernel_name(capi):
    name = capi.qlin_attn_mixed_kernel_name
    assert name(0, 16, 2, 128, 1, 4096) == "none"
    assert name(1, 16, 2, 96, 1, 4096) == "invalid"
    assert name(1, 28, 4, 128, 1, 32768) == "k_attn_split+k_attn_join"
    assert name(1, 16, 2, 128, 1, 37) == "k_attn_split"


def test_names_and_sizes(capi):
    n = capi.qlin_kernel_name
    assert n(capi.QLIN_OP_RMSNORM, 0, 5, 2048, 0) == "k_rmsnorm"
    assert n(capi.QLIN_OP_RMSNORM_QUANT, 1, 5, 2056, 0) == "invalid"
    assert n(capi.QLIN_OP_RMSNORM_QUANT, 1, 0, 2048, 0) == "none"
    assert n(capi.QLIN_OP_ROPE, 0, 5, 80, 32) == "k_rope"
    assert n(capi.QLIN_OP_ROPE_KV_STORE_MIXED, 0, 5, 128, 4) == "k_rope_kv_store<128>"
    assert n(capi.QLIN_OP_ROPE_KV_STORE_MIXED, 0, 5, 80, 4) == "invalid"
    assert n(capi.QLIN_OP_W8A8_LINEAR_CODES, 1, 5, 2048, 2048) == "k_fp8_gemm"
    for op in (capi.QLIN_OP_RMSNORM, capi.QLIN_OP_RMSNORM_QUANT, capi.QLIN_OP_ROPE, capi.QLIN_OP_ROPE_KV_STORE_MIXED):
        assert capi.qlin_workspace_bytes(op, "e4m3", 8, 128, 4) == 0


def test_binding_refusals(capi):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        capi.qlin_rmsnorm(x.t(), None, x, 1e-6, None, x)
    with pytest.raises(ValueError):
        capi.qlin_rope("half", 1, 0, 64, 64, torch.zeros(4, 32), torch.zeros(4, dtype=torch.int64), x, None, x, None)
