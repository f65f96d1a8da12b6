"""Cases and plain forms of the decoder-layer operators around the 8-bit linears.

Three operators: RMSNorm with the residual's addition and an 8-bit (or BF16)
output, rotary positions with an optional store into the mixed 8-bit KV cache,
and attention that reads that cache.  ``run`` computes each in elementary torch
operations, or, where ``own`` is set, calls the library.  ``exact`` restates the
operators in 64 bits.
"""
import math
import random

import torch

own = False

EPS = float(torch.tensor(1e-6, dtype=torch.float32))
QMAX = {"int8": 127.0, "e4m3": 448.0}
MAX_POS = 32768  # rows of the rotary table: the context the repository's KV workload serves
F8 = torch.float8_e4m3fn


def listed():
    return [
        # one token of a 7B-class decode step entering its fp8 linears
        {"name": "norm_row_e4m3", "op": "norm", "M": 1, "K": 3584, "out": "e4m3", "static": False, "residual": True},
        # an odd decode batch of a 3B-class model with dynamic INT8 activations
        {"name": "norm_batch_int8", "op": "norm", "M": 257, "K": 2048, "out": "int8", "static": False, "residual": True},
        # a prefill chunk of the 3B-class stack with a calibrated per-tensor scale
        {"name": "norm_prefill_static", "op": "norm", "M": 8192, "K": 2048, "out": "e4m3", "static": True, "residual": True},
        # the longest prefill of the repository at the 7B width, for weight-only linears (BF16 activations)
        {"name": "norm_prefill_bf16", "op": "norm", "M": 32640, "K": 3584, "out": "bf16", "static": False, "residual": True},
        # one new token of a 7B-class model: rotate q and k, store k and v
        {"name": "rope_store_token", "op": "rope", "T": 1, "Hq": 28, "H": 4, "D": 128, "rot": 128, "layout": "half", "store": True},
        # the KV workload's prefill chunk at the same heads
        {"name": "rope_store_prefill", "op": "rope", "T": 8192, "Hq": 28, "H": 4, "D": 128, "rot": 128, "layout": "half", "store": True},
        # an odd chunk, adjacent pairs, a quarter of the head rotated, kept in BF16
        {"name": "rope_partial_pairs", "op": "rope", "T": 1021, "Hq": 16, "H": 2, "D": 128, "rot": 32, "layout": "pairs", "store": False},
        # the first tokens of a chat with one user: latency
        {"name": "attn_short", "op": "attn", "kind": "decode", "B": 1, "Hq": 16, "H": 2, "D": 128, "max_q": 1, "max_kv": 37, "block": 256, "window": 0},
        # one user at the KV workload's whole context: split over the cache
        {"name": "attn_decode_long", "op": "attn", "kind": "decode", "B": 1, "Hq": 28, "H": 4, "D": 128, "max_q": 1, "max_kv": 32768, "block": 256, "window": 0},
        # a full serving batch of the 3B-class model, ragged contexts, padded rows without keys
        {"name": "attn_decode_batch", "op": "attn", "kind": "decode", "B": 256, "Hq": 16, "H": 2, "D": 128, "max_q": 1, "max_kv": 4096, "block": 256, "window": 0},
        # ragged chunks over cached prefixes, sliding window, small heads and pages
        {"name": "attn_extend_window", "op": "attn", "kind": "extend", "B": 5, "Hq": 8, "H": 8, "D": 64, "max_q": 333, "max_kv": 3001, "block": 16, "window": 1024},
        # the KV workload's prefill chunk as the second of a prompt
        {"name": "attn_prefill", "op": "attn", "kind": "extend", "B": 1, "Hq": 28, "H": 4, "D": 128, "max_q": 8192, "max_kv": 16384, "block": 256, "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn"])
    if op == "norm":
        K = 16 * _log(rng, 16, 1024)
        K = K if K != 3072 else 3088
        out = rng.choice(["e4m3", "int8", "bf16"])
        return {"op": "norm", "M": _log(rng, 1, min(32640, 32640 * 3584 // K)), "K": K, "out": out,
                "static": out != "bf16" and rng.random() < 0.4, "residual": rng.random() < 0.8}
    Hq, H = rng.choice([(28, 4), (16, 2), (8, 8), (32, 8), (12, 1), (40, 8)])
    D = rng.choice([32, 64, 128, 128, 128, 256])
    if op == "rope":
        T = _log(rng, 1, max(1, 8192 * 36 * 128 // ((Hq + 2 * H) * D)))
        return {"op": "rope", "T": T, "Hq": Hq, "H": H, "D": D, "rot": rng.choice([D, D, D // 2]),
                "layout": rng.choice(["half", "half", "pairs"]), "store": rng.random() < 0.6}
    block = rng.choice([16, 64, 256, 256, 24])
    if rng.random() < 0.6:
        B = _log(rng, 1, 256)
        return {"op": "attn", "kind": "decode", "B": B, "Hq": Hq, "H": H, "D": D, "max_q": 1,
                "max_kv": _log(rng, 1, max(1, min(32768, 256 * 4096 * 256 // (B * H * D)))), "block": block,
                "window": rng.choice([0, 0, 0, 128, 1000])}
    B = _log(rng, 1, 16)
    most = 8192 * 16384 * 28 * 128 // (B * Hq * D)  # query-key pairs of a sequence, at the largest listed cost
    q = _log(rng, 2, min(8192, int(math.sqrt(most / 2))))
    return {"op": "attn", "kind": "extend", "B": B, "Hq": Hq, "H": H, "D": D, "max_q": q,
            "max_kv": _log(rng, q, max(q, min(16384, most // q))), "block": block, "window": rng.choice([0, 0, 0, 128, 1000])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _lens(c):
    """New tokens and keys of each sequence: ragged, from the case alone.  A decode
    batch of 8 or more has two padding rows (one query, no keys)."""
    r = random.Random("%d/%d/%d" % (c["B"], c["max_q"], c["max_kv"]))
    if c["kind"] == "decode":
        kv = [c["max_kv"]] + [r.randint(max(1, c["max_kv"] // 4), c["max_kv"]) for _ in range(c["B"] - 1)]
        if c["B"] >= 8:
            kv[c["B"] // 2] = kv[-1] = 0
        return [1] * c["B"], kv
    nq = [c["max_q"]] + [r.randint(1, c["max_q"]) for _ in range(c["B"] - 1)]
    return nq, [c["max_kv"]] + [n + r.randint(0, c["max_kv"] - c["max_q"]) for n in nq[1:]]


def _cache(g, slots, H, D):
    """A mixed KV cache as the store writes it: int8 keys with float16 group-32
    scales, E4M3 values with a float16 scale per token and head."""
    kc = (_randn(g, slots, H, D) * 40).round_().clamp_(-127, 127).to(torch.int8)
    ks = (0.025 * torch.exp(0.3 * _randn(g, slots, H, D // 32))).to(torch.float16).view(torch.int16)
    vc = (_randn(g, slots, H, D) * 120).clamp_(-448, 448).to(F8).view(torch.uint8)
    vs = (0.008 * torch.exp(0.3 * _randn(g, slots, H))).to(torch.float16).view(torch.int16)
    return kc, ks, vc, vs


def _rope_table(rot):
    """[MAX_POS, rot] fp32: rot/2 cosines, then rot/2 sines, of pos * 10000^(-2i/rot)."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * (10000.0 ** (-2.0 * i / rot))[None, :]
    return torch.cat([torch.cos(a), torch.sin(a)], dim=1).float()


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c}
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        s["x"] = _randn(g, M, K).bfloat16()
        s["res"] = (2 * _randn(g, M, K)).bfloat16() if c["residual"] else None
        w = 1 + 0.2 * _randn(g, K)
        w[torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 8  # outlier channels
        s["w"] = w.bfloat16()
        s["input_scale"] = torch.full((1,), 30.0 / QMAX.get(c["out"], 1.0), device="cuda") * torch.exp(0.1 * _randn(g, 1))
        s["h"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda") if c["residual"] else None
        s["y"] = torch.empty(M, K, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.uint8, device="cuda")
        s["x_scale"] = torch.empty(M, dtype=torch.float32, device="cuda")
    elif c["op"] == "rope":
        T, Hq, H, D = c["T"], c["Hq"], c["H"], c["D"]
        s["qkv"] = _randn(g, T, (Hq + 2 * H) * D).bfloat16()  # a merged projection's rows
        s["table"] = _rope_table(c["rot"])
        start = int(torch.randint(0, MAX_POS - T + 1, (1,), generator=g, device="cuda"))
        s["pos"] = torch.arange(start, start + T, dtype=torch.int64, device="cuda")
        s["q_out"] = torch.empty(T, Hq * D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
        s["num_slots"] = 256 * (T // 256 + 2)
        s["cache"] = _cache(g, s["num_slots"], H, D) if c["store"] else None
        s["slots"] = torch.randperm(s["num_slots"], generator=g, device="cuda")[:T].contiguous()
    else:
        B, Hq, H, D, bs = c["B"], c["Hq"], c["H"], c["D"], c["block"]
        nq, kv = _lens(c)
        per = -(-c["max_kv"] // bs)
        nblocks = sum(-(-n // bs) for n in kv) + 3
        perm = torch.randperm(nblocks, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(B, per, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(kv):
            n = -(-n // bs)
            table[b, :n] = perm[at: at + n]
            at += n
        s["table"], s["cache"] = table, _cache(g, nblocks * bs, H, D)
        s["q"] = (2 * _randn(g, sum(nq), Hq * D)).bfloat16()
        start = [0]
        for n in nq:
            start.append(start[-1] + n)
        s["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(sum(nq), Hq * D, dtype=torch.bfloat16, device="cuda")
        s["scale"] = float(torch.tensor(D ** -0.5, dtype=torch.float32))
    return s


# ------------------------------------------------------------- plain forms
def _quantize(y, s, out):
    """Codes of y / s (s broadcast), as the type that holds them."""
    v = y / s
    return v.round().clamp(-127, 127).to(torch.int8) if out == "int8" else v.clamp(-448, 448).to(F8)


def _over(a, q):
    """a / q with one rounding (a division by a Python number would multiply by its reciprocal)."""
    return a / torch.full_like(a, q)


def _norm_plain(s):
    c, x, w = s["case"], s["x"], s["w"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).bfloat16()
    r = (1.0 / torch.sqrt(h.double().square().sum(1, keepdim=True) / c["K"] + EPS)).float()
    y = (h.float() * r) * w.float()
    got = {} if s["res"] is None else {"h": h}
    if c["out"] == "bf16":
        return {**got, "y": y.bfloat16()}
    if c["static"]:
        return {**got, "codes": _quantize(y, s["input_scale"], c["out"])}
    a = _over(y.abs().amax(1), QMAX[c["out"]])
    a = torch.where(a > 0, a, torch.ones_like(a))
    return {**got, "codes": _quantize(y, a[:, None], c["out"]), "scale": a}


def _rotate(x, cos, sin, c):
    """x [T, heads, D] in the type of cos and sin; the first rot dimensions are turned."""
    rot = c["rot"]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if c["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _scale16(amax, q):
    s = _over(amax, q).clamp(max=65504).half()
    return torch.where(s > 0, s, torch.ones_like(s))


def _rope_plain(s):
    c = s["case"]
    T, Hq, H, D, rot = c["T"], c["Hq"], c["H"], c["D"], c["rot"]
    t = s["table"][s["pos"]]
    qk = _rotate(s["qkv"][:, : (Hq + H) * D].float().view(T, Hq + H, D), t[:, : rot // 2], t[:, rot // 2:], c).bfloat16()
    q, k = qk[:, :Hq].reshape(T, Hq * D), qk[:, Hq:]
    if not c["store"]:
        return {"q": q, "k": k.reshape(T, H * D)}
    kc, ks, vc, vs = s["cache"]
    kg = k.float().view(T, H, D // 32, 32)
    k16 = _scale16(kg.abs().amax(-1), 127.0)
    v = s["qkv"][:, (Hq + H) * D:].float().view(T, H, D)
    v16 = _scale16(v.abs().amax(-1), 448.0)
    at = s["slots"]
    kc[at] = _quantize(kg, k16.float()[..., None], "int8").view(T, H, D)
    ks[at] = k16.view(torch.int16)
    vc[at] = _quantize(v, v16.float()[..., None], "e4m3").view(torch.uint8)
    vs[at] = v16.view(torch.int16)
    return {"q": q, **_cache_values(s["cache"])}


def _cache_values(cache):
    kc, ks, vc, vs = cache
    return {"k_codes": kc, "k_scale": ks.view(torch.float16), "v_codes": vc.view(F8), "v_scale": vs.view(torch.float16)}


def _gathered(s, real):
    """Keys and values [B, max_kv, H, D] in `real`, the visibility [B, max_q, max_kv], the padded queries
    [B, max_q, Hq, D], and the sequence and place of each query row."""
    c = s["case"]
    B, H, D, bs, Q, L = c["B"], c["H"], c["D"], c["block"], c["max_q"], c["max_kv"]
    j, i = torch.arange(L, device="cuda"), torch.arange(Q, device="cuda")
    kv, n = s["kv_len"].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    slots = s["table"].long()[:, j // bs] * bs + j % bs
    kc, ks, vc, vs = s["cache"]
    k = (kc[slots].to(real).view(B, L, H, D // 32, 32) * ks.view(torch.float16)[slots].to(real)[..., None]).view(B, L, H, D)
    v = vc.view(F8)[slots].to(real) * vs.view(torch.float16)[slots].to(real)[..., None]
    place = (kv - n)[:, None] + i  # position of query i of each sequence
    see = (j[None, None] <= place[..., None]) & (j < kv[:, None])[:, None] & (i < n[:, None])[..., None]
    if c["window"]:
        see &= j[None, None] > place[..., None] - c["window"]
    rows = torch.minimum(s["q_start"][:-1].long()[:, None] + i, s["q_start"][-1].long() - 1)
    q = s["q"].view(-1, c["Hq"], D)[rows].to(real)
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
    return k, v, see, q, b, t - s["q_start"].long()[b]


def _attend(q, k, v, see, scale):
    """Softmax attention over the last two axes; a row that sees nothing gives zeros."""
    a = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~see, -math.inf)
    m = a.amax(-1, keepdim=True)
    a = a.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    den = a.sum(-1, keepdim=True)
    return torch.matmul(a, v) / torch.where(den > 0, den, torch.ones_like(den))


def _attn_plain(s):
    c = s["case"]
    B, Hq, H, D, Q = c["B"], c["Hq"], c["H"], c["D"], c["max_q"]
    k, v, see, q, b, i = _gathered(s, torch.float32)
    q = q.view(B, Q, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * Q, D)
    see = see[:, None].expand(B, Hq // H, Q, c["max_kv"]).reshape(B, 1, Hq // H * Q, c["max_kv"])
    o = _attend(q, k.transpose(1, 2), v.transpose(1, 2), see, s["scale"])
    o = o.view(B, H, Hq // H, Q, D).permute(0, 3, 1, 2, 4)
    return o[b, i].reshape(-1, Hq * D).bfloat16()


def _run_own(s):
    from bit_quantized_linear_gb300 import capi
    c = s["case"]
    if c["op"] == "norm":
        got = {} if s["h"] is None else {"h": s["h"]}
        if c["out"] == "bf16":
            capi.qlin_rmsnorm(s["x"], s["res"], s["w"], EPS, s["h"], s["y"])
            return {**got, "y": s["y"]}
        capi.qlin_rmsnorm_quant(c["out"], s["x"], s["res"], s["w"], EPS, s["input_scale"] if c["static"] else None,
                                s["h"], s["y"], None if c["static"] else s["x_scale"])
        got["codes"] = s["y"].view(torch.int8 if c["out"] == "int8" else F8)
        return got if c["static"] else {**got, "scale": s["x_scale"]}
    if c["op"] == "rope":
        Hq, H, D = c["Hq"], c["H"], c["D"]
        q, k, v = s["qkv"].split([Hq * D, H * D, H * D], dim=1)
        if not c["store"]:
            capi.qlin_rope(c["layout"], Hq, H, D, c["rot"], s["table"], s["pos"], q, k, s["q_out"], s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        capi.qlin_rope_kv_store_mixed(c["layout"], Hq, c["rot"], s["table"], s["pos"], q, k, v, s["q_out"], s["slots"],
                                      *s["cache"])
        return {"q": s["q_out"], **_cache_values(s["cache"])}
    return capi.attn_mixed(s["q"], s["q_start"], s["kv_len"], s["table"], c["block"], s["cache"], c["max_q"],
                           c["max_kv"], scale=s["scale"], causal=True, window=c["window"], out=s["out"])


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "rope": _rope_plain, "attn": _attn_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "norm":
        el = c["M"] * c["K"]
        moved = el * (2 + (4 if c["residual"] else 0) + (2 if c["out"] == "bf16" else 1)) + 2 * c["K"]
        return {"bytes": moved + (0 if c["out"] == "bf16" or c["static"] else 4 * c["M"]), "flops": 6 * el}
    if c["op"] == "rope":
        T, Hq, H, D = c["T"], c["Hq"], c["H"], c["D"]
        moved = T * (2 * D * (2 * Hq + H) + 4 * c["rot"] + 8)  # q in and out, k in, table row, position
        moved += T * (H * (2 * D + 2 * D + D // 16 + 2) + 8) if c["store"] else T * H * D * 2
        return {"bytes": moved, "flops": 3 * T * (Hq + H) * c["rot"]}
    nq, kv = _lens(c)
    Hq, H, D, w = c["Hq"], c["H"], c["D"], c["window"]
    keys = pairs = 0
    for n, m in zip(nq, kv):
        n = min(n, m)  # rows that see a key
        first = m - n  # position of the first of them
        lo = max(0, first - w + 1) if w else 0
        keys += m - lo if n else 0
        if not w:
            pairs += n * first + n * (n + 1) // 2
        else:
            short = max(0, min(n, w - first))  # rows that still see the start
            pairs += short * first + short * (short + 1) // 2 + (n - short) * w
    return {"bytes": sum(nq) * Hq * D * 4 + keys * H * (2 * D + D // 16 + 2) + 4 * (keys // c["block"] + 2 * c["B"]),
            "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        x = s["x"].double()
        out = {}
        if c["residual"]:
            out["h"] = x + s["res"].double()
            x = out["h"].float().bfloat16().double()  # the stream the next layer reads is what is normalised
        y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w"].double()
        if c["out"] == "bf16":
            return {**out, "y": y}
        if c["static"]:
            a = s["input_scale"].double()
        else:
            out["scale"] = y.abs().amax(1) / QMAX[c["out"]]
            a = out["scale"][:, None]
        out["codes"] = None if c["out"] == "int8" else (y / a).clamp(-448, 448)
        return out
    if c["op"] == "rope":
        T, Hq, H, D, r = c["T"], c["Hq"], c["H"], c["D"], c["rot"] // 2
        t = s["table"].double()[s["pos"]]
        z = torch.complex(t[:, :r], t[:, r:])[:, None, :]
        x = s["qkv"].double().view(T, Hq + 2 * H, D)
        qk, v = x[:, : Hq + H].clone(), x[:, Hq + H:]
        if c["layout"] == "half":
            y = torch.complex(qk[..., :r].clone(), qk[..., r: 2 * r].clone()) * z
            qk[..., :r], qk[..., r: 2 * r] = y.real, y.imag
        else:
            y = torch.complex(qk[..., 0: 2 * r: 2].clone(), qk[..., 1: 2 * r: 2].clone()) * z
            qk[..., 0: 2 * r: 2], qk[..., 1: 2 * r: 2] = y.real, y.imag
        q, k = qk[:, :Hq].reshape(T, Hq * D), qk[:, Hq:]
        if not c["store"]:
            return {"q": q, "k": k.reshape(T, H * D)}
        _, ks, vc, vs = s["cache"]
        ks, vc, vs = ks.view(torch.float16).double(), vc.view(F8).double(), vs.view(torch.float16).double()
        ks[s["slots"]] = k.reshape(T, H, D // 32, 32).abs().amax(-1) / 127
        top = v.abs().amax(-1)
        vs[s["slots"]] = top / 448
        vc[s["slots"]] = v / (top / 448).half().double()[..., None]
        return {"q": q, "k_codes": None, "k_scale": ks, "v_codes": vc, "v_scale": vs}
    nq, kv = _lens(c)
    Hq, H, D, bs, w = c["Hq"], c["H"], c["D"], c["block"], c["window"]
    G, at = Hq // H, 0
    kc, ks, vc, vs = s["cache"]
    out = torch.zeros(sum(nq), Hq, D, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(nq, kv)):
        t = torch.arange(m, device="cuda")
        slots = s["table"][b].long()[t // bs] * bs + t % bs
        q = s["q"][at: at + n].view(n, H, G, D).double()
        dead = None
        if m:
            p = torch.arange(m - n, m, device="cuda")[:, None]
            dead = t > p
            if w:
                dead = dead | (t <= p - w)
        for h in range(H if m else 0):
            k = kc[slots, h].double() * ks.view(torch.float16)[slots, h].double().repeat_interleave(32, dim=1)
            v = vc.view(F8)[slots, h].double() * vs.view(torch.float16)[slots, h].double()[:, None]
            for g in range(G):
                a = torch.mm(q[:, h, g], k.t()) * s["scale"]
                a[dead] = -math.inf
                out[at: at + n, h * G + g] = torch.nan_to_num(torch.softmax(a, 1)) @ v
        at += n
    return out.reshape(-1, Hq * D)
