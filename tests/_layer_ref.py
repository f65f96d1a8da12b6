"""Plain 64-bit restatements of the operators around the linears (RMSNorm, rotary
positions, attention over the mixed KV cache) in numpy and CPU torch, and the
tolerance of the attention, for the tests."""
import math

import numpy as np
import torch

from bit_quantized_linear_gb300 import synth

F8 = torch.float8_e4m3fn


def bf16_round(a):
    """fp32 array -> the fp32 values of its BF16 rounding."""
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(a, np.float32)))


# ---------------------------------------------------------------------- norm
def norm(x, res, w, eps):
    """(h, y): x, res, w fp32 arrays of BF16 values.  y is the binary32 value the outputs are made from."""
    h = x if res is None else bf16_round(x + res)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        s = (h.astype(np.float64) ** 2).sum(1, keepdims=True) / h.shape[1] + float(np.float32(eps))
        r = (1.0 / np.sqrt(s)).astype(np.float32)
        return h, (h * r).astype(np.float32) * w.astype(np.float32)


def codes(y, s, qtype):
    """8-bit codes (uint8) of the binary32 quotients y / s; s broadcasts."""
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        v = (y / np.asarray(s, np.float32)).astype(np.float32)
    if qtype == "int8":
        return np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)
    return torch.from_numpy(np.clip(v, -448, 448)).to(F8).view(torch.uint8).numpy()


def row_scales(y, qtype):
    a = (np.abs(y).max(1) / np.float32(127 if qtype == "int8" else 448)).astype(np.float32)
    return np.where(a > 0, a, np.float32(1))


# ---------------------------------------------------------------------- rope
def frequencies(rot, theta, scaling="plain", factor=1.0, original_context=0.0, beta_fast=32.0, beta_slow=1.0):
    i = np.arange(rot // 2)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        keep = np.clip((original_context * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0, 1)
        f = (1 - keep) * f / factor + keep * f
    return f


def rope(x, table_rows, rot, layout):
    """x [T, heads, D] fp32 (BF16 values), table_rows [T, rot] fp32 -> fp32 values rounded to BF16, each
    product and sum one binary32 operation."""
    x = x.copy()
    c, s = table_rows[:, None, : rot // 2], table_rows[:, None, rot // 2:]
    at = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., at[0]].copy(), x[..., at[1]].copy()
    x[..., at[0]] = bf16_round(a * c - b * s)
    x[..., at[1]] = bf16_round(b * c + a * s)
    return x


# ----------------------------------------------------------------- attention
class Attn:
    """Inputs of one attention call on the host: nq and kv are the new tokens and
    positions of each sequence.  Everything of the cache that no sequence owns is
    NaN (value codes and scales) or large (key codes)."""

    def __init__(self, nq, kv, H, G, D, block, seed=0, spread=1.0, extra_blocks=3, q_scale=2.0):
        g = torch.Generator().manual_seed(seed)
        self.nq, self.kv, self.H, self.G, self.D, self.block = list(nq), list(kv), H, G, D, block
        B, T = len(nq), sum(nq)
        need = [-(-n // block) for n in kv]
        self.blocks = sum(need) + extra_blocks
        S = self.blocks * block
        self.q = (q_scale * torch.randn(T, H * G * D, generator=g)).bfloat16()
        self.kc = (torch.randn(S, H, D, generator=g) * 40).round().clamp(-127, 127).to(torch.int8)
        self.ks = (0.025 * torch.exp(spread * torch.randn(S, H, D // 32, generator=g))).half()
        self.vc = (torch.randn(S, H, D, generator=g) * 120).clamp(-448, 448).to(F8).view(torch.uint8)
        self.vs = (0.008 * torch.exp(spread * torch.randn(S, H, generator=g))).half()
        self.table = torch.full((B, max(1, max(need, default=1))), -7, dtype=torch.int32)  # unused entries: no page
        perm = torch.randperm(self.blocks, generator=g)
        owned = torch.zeros(S, dtype=torch.bool)
        at = 0
        for b, n in enumerate(kv):
            mine = perm[at: at + need[b]]
            self.table[b, : need[b]] = mine.int()
            at += need[b]
            j = torch.arange(n)
            owned[mine[j // block] * block + j % block] = True
        self.kc[~owned] = 127
        self.ks[~owned] = float("nan")
        self.vc[~owned] = 0x7F
        self.vs[~owned] = float("inf")
        self.q_start = torch.tensor([0] + list(np.cumsum(self.nq)), dtype=torch.int32)
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32)

    def cache(self):
        return self.kc, self.ks.view(torch.int16), self.vc, self.vs.view(torch.int16)

    def slots(self, b):
        j = torch.arange(self.kv[b])
        return self.table[b].long()[j // self.block] * self.block + j % self.block

    def reference(self, scale=None, causal=True, window=0, hole=None):
        """(out [T, Hq*D], tolerance) in fp64.  hole: (sequence, page index) whose positions take no part.

        The tolerance counts, per element with A = sum_j p_j |v_j| and B the row's largest
        scale * sum_d |q_d k_jd|: the output's rounding (2^-8 of the value), those of P and of a scaled value to
        float16 (2^-11 each of every term), that of a scaled key to float16 (2^-11 of every product, which moves a
        score by at most 2^-11 B and p, with the sum it is divided by, by twice that), and 2^-18 (1 + B) for fp32
        sums and exponentials."""
        scale = self.D ** -0.5 if scale is None else scale
        H, G, D = self.H, self.G, self.D
        out = torch.zeros(sum(self.nq), H * G, D, dtype=torch.float64)
        tol = torch.zeros_like(out)
        at = 0
        for b, (n, m) in enumerate(zip(self.nq, self.kv)):
            if m and n:
                sl = self.slots(b).clamp(min=0)
                k = self.kc[sl].double() * self.ks[sl].double().repeat_interleave(32, dim=2)
                v = self.vc[sl].view(F8).double() * self.vs[sl].double()[..., None]
                j = torch.arange(m)
                pos = torch.arange(m - n, m)[:, None]
                see = (j <= pos) if causal else torch.ones(n, m, dtype=torch.bool)
                if window:
                    see &= j > pos - window
                    if not causal:
                        see &= j < pos + window
                if hole and hole[0] == b:
                    see &= (j // self.block) != hole[1]
                for h in range(H):
                    v_h = v[:, h]
                    for g in range(G):
                        q = self.q[at: at + n].view(n, H * G, D)[:, h * G + g].double()
                        s = (q @ k[:, h].T) * scale
                        s[~see] = -math.inf
                        top = s.amax(1, keepdim=True)
                        p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
                        p[~see] = 0
                        den = p.sum(1, keepdim=True)
                        p = p / torch.where(den > 0, den, torch.ones_like(den))
                        # 0 * NaN of unseen positions is no contribution
                        nan = torch.isnan(v_h)
                        o = p @ torch.where(nan, torch.zeros_like(v_h), v_h)
                        hit = (see.double() @ nan.double()) > 0
                        o[hit] = math.nan
                        a = p @ torch.where(nan, torch.zeros_like(v_h), v_h.abs())
                        big = ((q.abs() @ k[:, h].abs().T) * abs(scale)).masked_fill(~see, 0).amax(1, keepdim=True)
                        out[at: at + n, h * G + g] = o
                        tol[at: at + n, h * G + g] = 2.0 ** -8 * o.abs() + a * (
                            2 * 2.0 ** -11 + 2 * 2.0 ** -11 * big + 2.0 ** -18 * (1 + big))
            at += n
        return out.reshape(at, -1), tol.reshape(at, -1)
