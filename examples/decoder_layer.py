"""A decoder layer on the 8-bit linears and the mixed KV cache: prompts of several
sequences in one ragged call, then decode steps replayed from a CUDA graph.

    python examples/decoder_layer.py

Random weights at the 3B-class sizes (hidden 2048, 16 query heads over 2 KV heads of
128, intermediate 11008).  Per layer:

    h, codes = norm(x + residual) as E4M3 codes      qlin_rmsnorm_quant
    qkv      = W8A8 linear on the codes              qlin_w8a8_linear_codes
    q        = turned; k, v into their slots         qlin_rope_kv_store_mixed
    a        = attention over the cache              qlin_attn_mixed
    o        = W8A8 linear, per-token scales         qlin_w8a8_dynamic_linear
    h, y     = norm(o + h) as BF16                   qlin_rmsnorm
    x        = W8A16 gate_up with SiLU, then down    qlin_w8a16_gate_up_silu, qlin_w8a16_linear
"""
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from bit_quantized_linear_gb300 import capi  # noqa: E402

QT = "e4m3"


class DecoderLayer:
    def __init__(self, hidden, Hq, H, D, inter, num_slots, eps=1e-6, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return capi.quantize_weight(QT, torch.randn(n, k, generator=g, device="cuda") / k ** 0.5)

        self.Hq, self.H, self.D, self.eps = Hq, H, D, eps
        self.norm_in = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).bfloat16()
        self.norm_mlp = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).bfloat16()
        self.qkv, self.o = weight((Hq + 2 * H) * D, hidden), weight(hidden, Hq * D)
        self.gate_up, self.down = weight(2 * inter, hidden), weight(hidden, inter)
        self.cache = capi.kv_cache_alloc(num_slots, H, D)

    def __call__(self, x, residual, batch, table, seen=None):
        """x, residual [T, hidden] (residual None in the first layer) -> the same of the next layer.
        seen: a dict that keeps the intermediate results."""
        n, m = self.Hq * self.D, self.H * self.D
        h, codes, scale = capi.rmsnorm_quant(QT, x, self.norm_in, self.eps, residual)
        qkv = capi.w8a8_linear_codes(QT, codes, scale, *self.qkv)
        q = torch.empty(x.shape[0], n, dtype=torch.bfloat16, device=x.device)
        capi.qlin_rope_kv_store_mixed("half", self.Hq, self.D, table, batch.positions, qkv[:, :n], qkv[:, n: n + m],
                                      qkv[:, n + m:], q, batch.slots, *self.cache)
        a = capi.attn_mixed(q, batch.q_start, batch.kv_len, batch.blocks, batch.block_size, self.cache, batch.max_q,
                            batch.max_kv)
        o = capi.w8a8_dynamic_linear(QT, a, *self.o)
        h2, y = capi.rmsnorm(o, self.norm_mlp, self.eps, h)
        up = capi.w8a16_gate_up_silu(QT, y, *self.gate_up)
        out = capi.w8a16_linear(QT, up, *self.down)
        if seen is not None:
            seen.update(h=h, codes=codes, scale=scale, qkv=qkv, q=q, a=a, o=o, h2=h2, y=y, up=up)
        return out, h2


class Batch:
    """Sequences over a paged cache: `new` tokens each on top of `past`.  max_kv bounds the
    positions of every step the batch will run."""

    def __init__(self, past, new, blocks, block_size, max_kv):
        self.blocks, self.block_size, self.max_kv, self.max_q = blocks, block_size, max_kv, max(new)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([p + n for p, n in zip(past, new)], dtype=torch.int32, device="cuda")
        self.row = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(new, device="cuda"))
        self.positions = torch.cat([torch.arange(p, p + n, device="cuda") for p, n in zip(past, new)])
        self.slots = torch.empty_like(self.positions)
        self.place()

    def place(self):
        block = self.blocks[self.row, self.positions // self.block_size].long()
        torch.add(block * self.block_size, self.positions % self.block_size, out=self.slots)

    def advance(self):
        """One token further, in place (a graph's replays advance the batch)."""
        self.positions += 1
        self.kv_len += 1
        self.place()


def main(layers=4, prompts=(700, 1500, 33, 4), steps=64, hidden=2048, Hq=16, H=2, D=128, inter=11008, block_size=256):
    B, max_kv = len(prompts), max(prompts) + steps
    per = -(-max_kv // block_size)
    blocks = torch.randperm(B * per, device="cuda").to(torch.int32).view(B, per)
    table = capi.rope_table(max_kv, D)
    net = [DecoderLayer(hidden, Hq, H, D, inter, B * per * block_size, seed=i) for i in range(layers)]

    def forward(x, batch):
        residual = None
        for layer in net:
            x, residual = layer(x, residual, batch, table)
        return x

    def timed(f):
        torch.cuda.synchronize()
        t = time.perf_counter()
        r = f()
        torch.cuda.synchronize()
        return r, time.perf_counter() - t

    x = torch.randn(sum(prompts), hidden, device="cuda").bfloat16()
    prompt = Batch([0] * B, list(prompts), blocks, block_size, max(prompts))
    forward(x, prompt)
    y, t_prompt = timed(lambda: forward(x, prompt))

    # decode: the last token's output stands in for the next token's embedding
    token = y[(prompt.q_start[1:] - 1).long()].clone()
    batch = Batch(list(prompts), [1] * B, blocks, block_size, max_kv)
    start = batch.positions.clone(), batch.kv_len.clone(), batch.slots.clone(), token.clone()

    def step():
        token.copy_(forward(token, batch))
        batch.advance()

    def rewind():
        for a, b in zip((batch.positions, batch.kv_len, batch.slots, token), start):
            a.copy_(b)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    rewind()

    def decode():
        for _ in range(steps - 1):  # the batch advances after each: the last leaves it at the final position
            graph.replay()

    _, t_steps = timed(decode)
    if capi.qlin_get_device_status() != capi.QLIN_OK:
        raise RuntimeError(capi.status_string(capi.qlin_get_device_status()))
    print(f"{layers} layers, hidden {hidden}: {sum(prompts)} prompt tokens in {t_prompt * 1e3:.2f} ms; "
          f"{B} sequences decode at {t_steps / (steps - 1) * 1e6:.0f} us a step (replayed)")
    return token


if __name__ == "__main__":
    main()
