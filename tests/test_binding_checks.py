"""The binding of the operators between the linears refuses tensors that the C entry
points would misread (host; the library is stood in for, so nothing is launched)."""
import pytest
import torch

BF16, U8, F32, I32, I64 = torch.bfloat16, torch.uint8, torch.float32, torch.int32, torch.int64


class _Stream:
    cuda_stream = 0


@pytest.fixture
def capi(monkeypatch):
    from bit_quantized_linear_gb300 import build
    build.build()
    from bit_quantized_linear_gb300 import capi as c

    class Lib:
        calls = []

        def __getattr__(self, name):
            return lambda *args: self.calls.append((name, args)) or 0

    lib = Lib()
    lib.calls.clear()
    monkeypatch.setattr(c, "_lib", lib)
    c.seen = lib.calls
    return c


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def cache(S=32, H=2, D=64):
    return dict(k_cache=z(S, H, D, dtype=torch.int8), k_scale=z(S, H, D // 32, dtype=torch.int16),
                v_cache=z(S, H, D, dtype=U8), v_scale=z(S, H, dtype=torch.int16))


def norm():
    return dict(x=z(4, 64), residual=z(4, 64), weight=z(64), eps=1e-6, h_out=z(4, 64), y_out=z(4, 64))


def quant():
    return dict(qtype="e4m3", x=z(4, 64), residual=z(4, 64), weight=z(64), eps=1e-6, input_scale=None,
                h_out=z(4, 64), qx=z(4, 64, dtype=U8), x_scale=z(4, dtype=F32))


def codes():
    return dict(qtype="int8", qx=z(4, 64, dtype=U8), x_scale=z(4, dtype=F32), qw=z(32, 64, dtype=U8),
                w_scale=z(32, dtype=F32), bias=z(32), y=z(4, 32), ws=z(4096, dtype=U8))


def rope():
    return dict(layout="half", Hq=4, Hk=2, D=64, rot=32, table=z(16, 32, dtype=F32), positions=z(4, dtype=I64),
                q=z(4, 512)[:, :256], k=z(4, 512)[:, 256:384], q_out=z(4, 256), k_out=z(4, 128))


def store():
    return dict(layout="half", Hq=4, rot=32, table=z(16, 32, dtype=F32), positions=z(4, dtype=I64), q=z(4, 256),
                k=z(4, 128), v=z(4, 128), q_out=z(4, 256), slots=z(4, dtype=I64), **cache())


def attn():
    return dict(q=z(3, 256), q_start=z(3, dtype=I32), kv_len=z(2, dtype=I32), block_table=z(2, 4, dtype=I32),
                block_size=8, **cache(), max_q=2, max_kv=32, scale=0.1, causal=True, window=0, out=z(3, 256))


WRONG = [
    ("qlin_rmsnorm", norm, [
        dict(x=z(4, 64, dtype=torch.float16)), dict(residual=z(3, 64)), dict(residual=z(4, 64, dtype=F32)),
        dict(weight=z(32)), dict(weight=z(128)[::2]), dict(weight=z(64, dtype=F32)), dict(h_out=z(4, 128)[:, :64]),
        dict(h_out=z(3, 64)), dict(y_out=z(4, 128)[:, :64]), dict(y_out=z(4, 64, dtype=F32)), dict(y_out=z(2, 64))]),
    ("qlin_rmsnorm_quant", quant, [
        dict(qx=z(4, 64)), dict(qx=z(4, 32, dtype=U8)), dict(qx=z(4, 128, dtype=U8)[:, :64]),
        dict(x_scale=z(3, dtype=F32)), dict(x_scale=z(4)), dict(x_scale=z(8, dtype=F32)[::2]), dict(weight=z(65)),
        dict(input_scale=z(1), x_scale=None), dict(input_scale=z(4, dtype=F32), x_scale=None)]),
    ("qlin_w8a8_linear_codes", codes, [
        dict(x_scale=z(3, dtype=F32)), dict(x_scale=z(5, dtype=F32)), dict(x_scale=z(4)), dict(x_scale=z(1)),
        dict(qx=z(4, 128, dtype=U8)[:, :64]), dict(qx=z(4, 64)), dict(qw=z(32, 32, dtype=U8)),
        dict(qw=z(32, 128, dtype=U8)[:, :64]), dict(w_scale=z(31, dtype=F32)), dict(w_scale=z(32)),
        dict(bias=z(16)), dict(bias=z(32, dtype=F32)), dict(y=z(3, 32)), dict(y=z(4, 64)[:, :32])]),
    ("qlin_rope", rope, [
        dict(table=z(16, 64, dtype=F32)[:, :32]), dict(table=z(16, 32, dtype=torch.float64)),
        dict(positions=z(4, dtype=I32)), dict(positions=z(8, dtype=I64)[::2]), dict(q=z(3, 256)), dict(q=z(4, 128)),
        dict(q=z(4, 256, dtype=F32)), dict(k=z(5, 128)), dict(q_out=z(3, 256)), dict(q_out=z(4, 192)),
        dict(k_out=z(4, 64)), dict(k_out=z(4, 128, dtype=torch.float16))]),
    ("qlin_rope_kv_store_mixed", store, [
        dict(slots=z(4, dtype=I32)), dict(slots=z(3, dtype=I64)), dict(positions=z(4, dtype=I32)), dict(v=z(3, 128)),
        dict(k=z(4, 64)), dict(q_out=z(2, 256)), dict(k_scale=z(32, 2, 2, dtype=F32)),
        dict(v_scale=z(32, 1, dtype=torch.int16)), dict(v_cache=z(16, 2, 64, dtype=U8)),
        dict(k_cache=z(32, 4, 64, dtype=torch.int8)[:, :2])]),
    ("qlin_attn_mixed", attn, [
        dict(q_start=z(3, dtype=I64)), dict(q_start=z(2, dtype=I32)), dict(kv_len=z(2, dtype=I64)),
        dict(block_table=z(2, 4, dtype=I64)), dict(block_table=z(2, 8, dtype=I32)[:, :4]),
        dict(block_table=z(3, 4, dtype=I32)), dict(q=z(3, 256, dtype=torch.float16)), dict(q=z(3, 250)),
        dict(out=z(2, 256)), dict(out=z(3, 256, dtype=F32)), dict(out=z(3, 128)),
        dict(k_scale=z(32, 2, 1, dtype=torch.int16)), dict(v_scale=z(32, 4, dtype=torch.int16)[:, ::2])]),
]


@pytest.mark.parametrize("name,good", [w[:2] for w in WRONG], ids=[w[0] for w in WRONG])
def test_right_ones_reach_the_library(capi, name, good):
    getattr(capi, name)(**good(), stream=_Stream)
    assert [n for n, _ in capi.seen] == [name]


@pytest.mark.parametrize("name,good,change", [(n, g, c) for n, g, cs in WRONG for c in cs],
                         ids=[f"{n}-{'+'.join(c)}{i}" for n, _, cs in WRONG for i, c in enumerate(cs)])
def test_wrong_ones_do_not(capi, name, good, change):
    args = good()
    assert set(change) <= set(args)
    with pytest.raises(ValueError):
        getattr(capi, name)(**{**args, **change}, stream=_Stream)
    assert not capi.seen


def test_one_scale_or_one_a_row(capi):
    per_token = lambda: [a[6] for n, a in capi.seen]  # noqa: E731
    capi.qlin_w8a8_linear_codes(**codes(), stream=_Stream)
    capi.qlin_w8a8_linear_codes(**{**codes(), "x_scale": z(1, dtype=F32)}, stream=_Stream)
    assert per_token() == [1, 0]


def test_table_and_no_rows(capi):
    with pytest.raises(ValueError):
        capi.qlin_rope_table(z(4, 64, dtype=F32)[:, :32], 1e4, stream=_Stream)
    capi.qlin_rmsnorm(z(0, 64), None, z(64), 1e-6, None, z(0, 64), stream=_Stream)
    capi.qlin_w8a8_linear_codes(**{**codes(), "qx": z(0, 64, dtype=U8), "x_scale": z(0, dtype=F32), "y": z(0, 32)},
                                stream=_Stream)
    assert len(capi.seen) == 2
