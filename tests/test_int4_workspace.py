"""attn_int4 takes the workspace that it makes itself from the device of q, as attn_mixed does (host)."""
import pytest
import torch


@pytest.fixture(scope="module")
def capi():
    from bit_quantized_linear_gb300 import build
    build.build()
    from bit_quantized_linear_gb300 import capi as c
    return c


def test_workspace_is_where_q_is(capi, monkeypatch):
    made, calls = [], []
    storage = torch.UntypedStorage

    class Lib:
        def qlin_attn_int4_workspace_bytes(self, *sizes):
            return 4096

        def qlin_attn_int4(self, *args):
            calls.append(args)
            return 0

    monkeypatch.setattr(capi, "_lib", Lib())
    monkeypatch.setattr(capi, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch, "UntypedStorage", lambda n, device: made.append(storage(n, device=device)) or made[-1])
    q = torch.zeros(2, 256, dtype=torch.bfloat16)
    cache = [torch.zeros(2, 2, 16, n, dtype=t) for n, t in ((32, torch.uint8), (2, torch.int16)) * 2]
    i32 = dict(dtype=torch.int32)
    out = capi.attn_int4(q, torch.tensor([0, 2], **i32), torch.tensor([20], **i32), torch.zeros(1, 2, **i32), cache, 2, 32)
    assert out.device == q.device and len(calls) == 1
    assert len(made) == 1 and made[0].device == q.device and made[0].nbytes() == 4096
    assert calls[0][-3:-1] == (made[0].data_ptr(), 4096)
