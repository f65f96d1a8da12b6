"""attn_int4 takes the workspace that it makes itself as a tensor on q's device, as attn_mixed does (host)."""
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
    empty = torch.empty

    class Lib:
        def qlin_attn_int4_workspace_bytes(self, *sizes):
            return 4096

        def qlin_attn_int4(self, *args):
            calls.append(args)
            return 0

    monkeypatch.setattr(capi, "_lib", Lib())
    monkeypatch.setattr(capi, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    q = torch.zeros(2, 256, dtype=torch.bfloat16)
    cache = [torch.zeros(2, 2, 16, n, dtype=t) for n, t in ((32, torch.uint8), (2, torch.int16)) * 2]
    i32 = dict(dtype=torch.int32)
    out = capi.attn_int4(q, torch.tensor([0, 2], **i32), torch.tensor([20], **i32), torch.zeros(1, 2, **i32), cache, 2, 32)
    assert out.device == q.device and len(calls) == 1
    ws = [t for t in made if t.dtype is torch.uint8]
    assert len(ws) == 1 and ws[0].device == q.device and ws[0].numel() == 4096
    assert calls[0][-3:-1] == (ws[0].data_ptr(), 4096)
