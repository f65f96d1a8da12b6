"""Attention over the mixed KV cache against a 64-bit restatement (GPU), with the
tolerance that tests/_layer_ref.py derives.  Whatever the sequences do not own in
the caches is NaN, infinite or extreme."""
import numpy as np
import pytest
import torch

import _layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import capi as c
    return c


def _run(capi, a, status=0, **kw):
    cache = [t.cuda() for t in a.cache()]
    out = capi.attn_mixed(a.q.cuda(), a.q_start.cuda(), a.kv_len.cuda(), a.table.cuda(), a.block, cache,
                          max(a.nq), max(a.kv), **kw)
    assert capi.qlin_get_device_status() == status
    return out.float().cpu().double()


def _check(out, a, **kw):
    want, tol = a.reference(**kw)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    ok = ~torch.isnan(want)
    over = (out - want).abs()[ok] - tol[ok]
    assert over.numel() == 0 or over.max() <= 0, f"{int((over > 0).sum())} of {over.numel()} beyond the tolerance, " \
        f"by up to {float(over.max())}"


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (4, 7), (1, 16), (3, 12)])
@pytest.mark.parametrize("block", [16, 24])
def test_decode(capi, D, H, G, block):
    a = ref.Attn([1] * 6, [1, 15, 16, 0, 67, 530], H, G, D, block, seed=D + G)
    _check(_run(capi, a), a)


@pytest.mark.parametrize("D,H,G,kv", [(128, 4, 7, 4097), (128, 2, 8, 20000), (64, 1, 1, 9999), (256, 1, 12, 5000),
                                      (32, 1, 4, 3333)])
def test_decode_long(capi, D, H, G, kv):
    """Positions split over many CTAs, beside a short and an empty sequence."""
    a = ref.Attn([1, 1, 1], [kv, 40, 0], H, G, D, 256, seed=kv)
    assert "join" in capi.qlin_attn_mixed_kernel_name(3, H * G, H, D, 1, kv)
    _check(_run(capi, a), a)


@pytest.mark.parametrize("block", [1, 3, 16, 17, 64, 1000])
def test_pages(capi, block):
    a = ref.Attn([1, 4, 1], [100, 333, 1], 2, 3, 64, block, seed=block)
    _check(_run(capi, a), a)


@pytest.mark.parametrize("D,H,G", [(128, 2, 7), (64, 8, 1), (256, 1, 2), (32, 2, 5), (128, 1, 128)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_new_tokens(capi, D, H, G, causal, window):
    """Ragged runs of new tokens over prefixes; a sequence with more rows than positions has rows that see
    nothing."""
    a = ref.Attn([5, 1, 40, 0, 9, 130], [5, 77, 129, 30, 3, 300], H, G, D, 16, seed=D + window)
    _check(_run(capi, a, causal=causal, window=window), a, causal=causal, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill(capi, D):
    a = ref.Attn([700, 257], [700, 1500], 1, 7, D, 256, seed=D)
    _check(_run(capi, a), a)


@pytest.mark.parametrize("window", [100, 128, 5000])
def test_window_decode(capi, window):
    a = ref.Attn([1, 1, 2], [4000, 90, 129], 2, 4, 128, 64, seed=window)
    _check(_run(capi, a, window=window), a, window=window)


@pytest.mark.parametrize("nq", [1, 3, 90])
def test_magnitudes(capi, nq):
    """Scales over float16's range within one sequence, q from tiny to large rows, negative softmax scale."""
    a = ref.Attn([nq, nq], [200, 300], 2, 4, 128, 16, seed=nq, spread=2.5, q_scale=0.5)
    a.vs[::5] *= 2.0 ** -9
    a.vs[::7] = 2.0 ** 9
    a.ks[::3] *= 2.0 ** -8
    for t in range(a.q.shape[0]):
        a.q[t] *= [1.0, 2.0 ** -60, 2.0 ** 3, 0.0][t % 4]
    _check(_run(capi, a), a)
    _check(_run(capi, a, scale=-0.05), a, scale=-0.05)


@pytest.mark.parametrize("nq", [1, 2, 90])
def test_largest_values(capi, nq):
    """The largest key and value the cache can hold (65504 * 127, 65504 * 448): nothing overflows."""
    a = ref.Attn([nq], [64], 1, 2, 64, 16, seed=3)
    a.ks.fill_(65504.0)
    a.vs.fill_(65504.0)
    a.q *= 2.0 ** -26
    _check(_run(capi, a), a)


@pytest.mark.parametrize("D,nq", [(128, 1), (128, 6), (64, 140), (128, 140), (256, 40)])
def test_nan_values_stay_where_they_are_seen(capi, D, nq):
    """NaN value codes in every dimension of one position: rows that see it are NaN, the others as without."""
    a = ref.Attn([nq, 3], [150, 40], 1, 4, D, 16, seed=nq)
    s = a.slots(0)[150 - 1 - nq // 2]
    a.vc[s] = 0x7F
    out = _run(capi, a)
    _check(out, a)
    assert torch.isnan(out).any() and (nq == 1 or not torch.isnan(out).all())


def test_infinite_query(capi):
    """An infinity in a query row makes that row NaN and no other."""
    a = ref.Attn([4], [50], 1, 2, 64, 16, seed=9)
    a.q[2, 5] = float("inf")
    out = _run(capi, a).view(4, 2, 64)
    assert torch.isnan(out[2, 0]).all()
    assert not torch.isnan(out[[0, 1, 3]]).any() and not torch.isnan(out[2, 1]).any()


@pytest.mark.parametrize("nq,kv", [(1, 300), (1, 9000), (100, 300)])
def test_bad_page(capi, nq, kv):
    """Positions of a page outside the cache take no part, and the status says so."""
    a = ref.Attn([nq, 1], [kv, 20], 2, 4, 128, 16, seed=nq)
    want, tol = a.reference(hole=(0, 3))
    for page in (-1, a.blocks, 2 ** 31 - 1):
        keep = int(a.table[0, 3])
        a.table[0, 3] = page
        out = _run(capi, a, status=capi.QLIN_ERR_INVALID_ARG)
        a.table[0, 3] = keep
        assert ((out - want).abs() <= tol).all()


def test_broken_counts(capi):
    """Rows, positions and table entries beyond their bounds are left out and reported; nothing is read or
    written out of range."""
    a = ref.Attn([1, 1], [100, 60], 1, 4, 64, 16, seed=1)
    cache = [t.cuda() for t in a.cache()]
    q = a.q.cuda()

    def call(q_start, kv_len, max_q=1, max_kv=100, table=a.table):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        capi.qlin_attn_mixed(q, torch.tensor(q_start, dtype=torch.int32).cuda(),
                             torch.tensor(kv_len, dtype=torch.int32).cuda(), table.cuda(), 16, *cache, max_q, max_kv,
                             0.125, True, 0, out)
        return out.float().cpu(), capi.qlin_get_device_status()

    good, status = call([0, 1, 2], [100, 60])
    assert status == capi.QLIN_OK
    bad = capi.QLIN_ERR_INVALID_ARG
    out, status = call([0, 1, 3], [100, 60])         # rows beyond q
    assert status == bad and torch.equal(out[0], good[0]) and (out[1] == 7).all()
    out, status = call([0, 1, 0], [100, 60])         # rows that run backwards
    assert status == bad and torch.equal(out[0], good[0]) and (out[1] == 7).all()
    out, status = call([-1, 1, 2], [100, 60])
    assert status == bad and (out[0] == 7).all() and torch.equal(out[1], good[1])
    out, status = call([0, 1, 2], [-5, 60])          # a negative count: no positions
    assert status == bad and (out[0] == 0).all() and torch.equal(out[1], good[1])
    out, status = call([0, 1, 2], [100, 2 ** 31 - 1], max_kv=100)
    assert status == bad and torch.equal(out[0], good[0])
    out, status = call([0, 1, 2], [100, 60], max_kv=70)
    assert status == bad and torch.equal(out[1], good[1])
    out, status = call([0, 1, 2], [100, 60], table=a.table[:, :5].contiguous())
    assert status == bad and torch.equal(out[1], good[1])
    out, status = call([0, 2, 2], [100, 60])         # more rows than max_q: the last one is left
    assert status == bad and (out[1] == 7).all()


def test_strides(capi):
    a = ref.Attn([3, 1], [30, 200], 2, 2, 64, 16, seed=4)
    T, n = a.q.shape
    q = torch.full((T, n + 48), 3.0, dtype=torch.bfloat16, device="cuda")
    q[:, 16: 16 + n] = a.q.cuda()
    out = torch.full((T, n + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    capi.attn_mixed(q[:, 16: 16 + n], a.q_start.cuda(), a.kv_len.cuda(), a.table.cuda(), 16,
                    [t.cuda() for t in a.cache()], 3, 200, out=out[:, :n])
    _check(out[:, :n].float().cpu().double(), a)
    assert (out[:, n:] == 7).all()


def test_nothing_to_do(capi):
    a = ref.Attn([1], [10], 1, 1, 64, 16)
    cache = [t.cuda() for t in a.cache()]
    n = capi.qlin_launch_count()
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    capi.attn_mixed(e, torch.zeros(2, dtype=torch.int32, device="cuda"), a.kv_len.cuda(), a.table.cuda(), 16, cache, 1, 10)
    assert capi.qlin_launch_count() == n
    out = capi.attn_mixed(a.q.cuda(), a.q_start.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                          a.table.cuda(), 16, cache, 1, 0)
    assert (out == 0).all() and capi.qlin_get_device_status() == capi.QLIN_OK


def test_offsets_beyond_32_bits(capi):
    """Pages whose codes lie beyond 2^32 bytes of the cache."""
    H, D, block = 4, 256, 256
    blocks = 2 ** 32 // (H * D * block) + 8
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 10 GB")
    a = ref.Attn([1, 2, 70], [500, 700, 300], H, 2, D, block, seed=2, extra_blocks=0)
    S = blocks * block
    big = [torch.empty((S,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda") for t in a.cache()]
    far = torch.randperm(8, generator=torch.Generator().manual_seed(1)) + blocks - 8
    far[::2] -= blocks // 2  # some below, some beyond
    for t, x in zip(big, a.cache()):
        for i in range(a.blocks):
            t[far[i] * block: (far[i] + 1) * block] = x[i * block: (i + 1) * block].cuda()
    table = torch.where(a.table >= 0, far[a.table.clamp(min=0).long()].int(), a.table)
    out = capi.attn_mixed(a.q.cuda(), a.q_start.cuda(), a.kv_len.cuda(), table.cuda(), block, big, 70, 700)
    assert capi.qlin_get_device_status() == capi.QLIN_OK
    _check(out.float().cpu().double(), a)


def test_captured_on_another_stream(capi):
    """A captured decode step replays with new lengths, tables and queries; parts and their join included."""
    a = ref.Attn([1] * 3, [900, 5000, 0], 2, 4, 128, 64, seed=11)
    b = ref.Attn([1] * 3, [5000, 0, 1234], 2, 4, 128, 64, seed=12, extra_blocks=3)
    assert a.blocks <= b.blocks + 40
    S = max(a.blocks, b.blocks) * 64
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        cache = [torch.zeros((S,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda") for t in a.cache()]
        table = torch.full((3, 79), -1, dtype=torch.int32, device="cuda")
        q, out = a.q.cuda(), torch.empty(a.q.shape, dtype=torch.bfloat16, device="cuda")
        kv, qs = a.kv_len.cuda(), a.q_start.cuda()
        ws = torch.empty(capi.qlin_attn_mixed_workspace_bytes(3, 8, 2, 128, 1, 5000), dtype=torch.uint8, device="cuda")

        def load(c):
            for t, x in zip(cache, c.cache()):
                t[: x.shape[0]] = x.cuda()
            table.fill_(-1)
            table[:, : c.table.shape[1]] = c.table.cuda()
            q.copy_(c.q)
            kv.copy_(c.kv_len)

        load(a)
        step = lambda: capi.attn_mixed(q, qs, kv, table, 64, cache, 1, 5000, out=out, ws=ws)  # noqa: E731
        step()
        side.synchronize()
        _check(out.float().cpu().double(), a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        load(b)
        graph.replay()
        side.synchronize()
        _check(out.float().cpu().double(), b)
    assert capi.qlin_get_device_status() == capi.QLIN_OK


def test_same_bits_twice(capi):
    """No order of additions depends on timing."""
    a = ref.Attn([1] * 4 + [33], [3000, 5000, 1, 0, 2000], 2, 4, 128, 64, seed=5)
    x = _run(capi, a)
    for _ in range(3):
        y = _run(capi, a)
        assert torch.equal(x, y)
