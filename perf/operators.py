"""Timed cases of the prompt and 4-bit-cache operators.

Four groups of cases, each with a plain form (elementary torch operations in 32 bits) and the
library's calls:

* ``decode``: one gated decode step over a 4-bit KV cache (``decode_ex`` with ``kv_scales``);
* ``cache``:  K and V rows quantised into the 4-bit cache and read back as BF16 rows
              (``kv_write_fp4``, ``kv_gather_fp4``);
* ``mrope``:  Q/K RMSNorm, rotary positions with several axes and the cache write
              (``qk_norm_mrope_kv_write``);
* ``packed``: gated causal attention over packed prompts (``prefill_packed``).
"""
import math
import random

import torch

own = False

D = 256
BLK = 16                     # head dimensions per scale of the 4-bit cache
ROW4 = D // 2 + D // 2 + 2 * (D // BLK)   # bytes of one (slot, KV head): K and V codes, both rows' scales
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a chat with one user, the shortest step: latency
        {"name": "decode_b1_l512", "op": "decode", "batch": 1, "lo": 512, "hi": 512, "hq": 16, "hkv": 2, "window": 0,
         "sinks": False, "draw": 1},
        # the bandwidth workload: 64 users at 4096 positions
        {"name": "decode_b64_l4096", "op": "decode", "batch": 64, "lo": 4096, "hi": 4096, "hq": 16, "hkv": 2, "window": 0,
         "sinks": False, "draw": 2},
        # a server under load: 224 users, every length from 1 on
        {"name": "decode_b224_ragged", "op": "decode", "batch": 224, "lo": 1, "hi": 6142, "hq": 16, "hkv": 2, "window": 0,
         "sinks": False, "draw": 3},
        # few long documents, sixteen query heads to a KV head, attention sinks
        {"name": "decode_b8_l32769_g16", "op": "decode", "batch": 8, "lo": 32769, "hi": 32769, "hq": 32, "hkv": 2,
         "window": 0, "sinks": True, "draw": 4},
        # the new tokens of a decode step go into the cache
        {"name": "cache_t64", "op": "cache", "tokens": 64, "hkv": 2, "spare": 1024},
        # a whole prompt's rows
        {"name": "cache_t16384", "op": "cache", "tokens": 16384, "hkv": 2, "spare": 4096},
        # one decode token with the gate copied out and its rows written to a BF16 cache
        {"name": "mrope_t1", "op": "mrope", "tokens": 1, "hq": 16, "hkv": 2, "rope": 64, "axes": 3, "kv": "bf16",
         "gate": True, "norm": True, "far": 200000, "spare": 64},
        # a decode step of 224 users into a 4-bit cache
        {"name": "mrope_t224_fp4", "op": "mrope", "tokens": 224, "hq": 16, "hkv": 2, "rope": 64, "axes": 3, "kv": "fp4",
         "gate": True, "norm": True, "far": 200000, "spare": 64},
        # a prompt with images: queries and keys for the prompt attention, rows into a BF16 cache
        {"name": "mrope_t16383", "op": "mrope", "tokens": 16383, "hq": 16, "hkv": 2, "rope": 64, "axes": 3, "kv": "bf16",
         "gate": False, "norm": True, "far": 40000, "spare": 257},
        # a few short questions in one batch: latency
        {"name": "packed_b4_t300", "op": "packed", "seqs": 4, "tokens": 300, "hq": 16, "hkv": 2, "prefix": 0, "draw": 1},
        # an ordinary batch of prompts, every length
        {"name": "packed_b9_t6001", "op": "packed", "seqs": 9, "tokens": 6001, "hq": 32, "hkv": 2, "prefix": 0, "draw": 2},
        # long prompts, two of them continued after a cached prefix
        {"name": "packed_b3_t12288", "op": "packed", "seqs": 3, "tokens": 12288, "hq": 16, "hkv": 2, "prefix": 1000, "draw": 3},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "packed", "packed", "mrope", "cache"])
    if op == "decode":
        batch = _log_int(rng, 1, 224)
        hi = _log_int(rng, 1, min(131072, 1000000 // batch))
        hq, hkv = rng.choice([(16, 2), (16, 2), (32, 2), (8, 1), (12, 4), (8, 8)])
        # a KV head more costs as much as a position more
        hi = max(1, hi * 2 // max(2, hkv))
        return {"op": op, "batch": batch, "lo": rng.choice([0, 1, hi]), "hi": hi, "hq": hq, "hkv": hkv,
                "window": rng.choice([0, 0, max(1, hi // 3)]), "sinks": rng.random() < 0.3, "draw": rng.randrange(1 << 30)}
    if op == "packed":
        tokens = _log_int(rng, 1, 9000)
        hq, hkv = rng.choice([(16, 2), (32, 2), (8, 1), (12, 4)]) if tokens < 6000 else (16, 2)
        seqs = _log_int(rng, 1, max(1, min(64, tokens)))
        return {"op": op, "seqs": seqs, "tokens": tokens, "hq": hq, "hkv": hkv,
                "prefix": rng.choice([0, 0, rng.randrange(1, 3000 // seqs)]), "draw": rng.randrange(1 << 30)}
    if op == "mrope":
        hq, hkv = rng.choice([(16, 2), (8, 1), (12, 4)])
        return {"op": op, "tokens": _log_int(rng, 1, 16000), "hq": hq, "hkv": hkv, "rope": rng.choice([16, 64, 128, 256]),
                "axes": rng.choice([1, 3, 3, 4]), "kv": rng.choice(["none", "bf16", "fp4"]), "gate": rng.random() < 0.5,
                "norm": rng.random() < 0.8, "far": _log_int(rng, 100, 1000000), "spare": rng.randrange(1, 300)}
    hkv = rng.choice([1, 2, 4])
    return {"op": op, "tokens": _log_int(rng, 1, 32768 // hkv), "hkv": hkv, "spare": rng.randrange(1, 2000)}


def _lengths(case):
    """A decode batch's lengths: they follow from the case."""
    r = random.Random(case["draw"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    return [max(1, n[0])] + n[1:]


def _splits(case):
    """A packed batch's query lengths and key lengths: they follow from the case."""
    r = random.Random(case["draw"])
    n, t = case["seqs"], case["tokens"]
    share = [r.expovariate(1.0) + 0.02 for _ in range(n)]
    lens = [max(1, int(t * x / sum(share))) for x in share]
    while sum(lens) > t:
        lens[lens.index(max(lens))] -= 1
    lens[r.randrange(n)] += t - sum(lens)
    more = [case["prefix"] if case["prefix"] and i % 2 == 0 else 0 for i in range(n)]
    return lens, [a + b for a, b in zip(lens, more)]


def _seen(case):
    """Visible (query, key) pairs of a packed batch."""
    return sum(nq * (nk - nq) + nq * (nq + 1) // 2 for nq, nk in zip(*_splits(case)))


def work(case):
    op = case["op"]
    if op == "decode":
        w = case["window"]
        n = sum(min(x, w) if w else x for x in _lengths(case))
        b = case["batch"] * case["hq"]
        return {"bytes": n * (case["hkv"] * ROW4 + 4) + b * (3 * 2 * D + 4), "flops": 4 * D * (case["hq"] * n)}
    if op == "cache":
        return {"bytes": case["tokens"] * (case["hkv"] * 2 * (2 * 2 * D + ROW4) + 8), "flops": 0}
    if op == "mrope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        rows = 2 * (hq + hkv)                                    # q and k in and out
        rows += 2 * hq if case["gate"] else 0
        b = t * (rows * 2 * D + 4 * case["axes"])
        if case["kv"] == "bf16":
            b += t * (hkv * 2 * D * 3 + 4)                       # k again, v in and out
        if case["kv"] == "fp4":
            b += t * (hkv * (2 * D + ROW4) + 4) + t * hkv * (ROW4 + 2 * 2 * D)   # written, then read back
        return {"bytes": b, "flops": 0}
    nq, nk = _splits(case)
    return {"bytes": 2 * D * (3 * case["tokens"] * case["hq"] + 2 * sum(nk) * case["hkv"]) + 4 * case["tokens"] * case["hq"],
            "flops": 4 * D * case["hq"] * _seen(case)}


# ---------------------------------------------------------------- the 4-bit format, plainly

def _e2m1_codes(x):
    """Codes of values already divided by their scale: nearest, ties to the even code, beyond 6 to 6."""
    a = x.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8))
    return code | ((x < 0).to(torch.uint8) << 3)


def _quantise(x, descale):
    """[..., D] values to (codes of one byte each [..., D], e4m3 scales [..., D / 16])."""
    y = (x / descale).unflatten(-1, (D // BLK, BLK))
    s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.to(y.dtype).unsqueeze(-1)
    z = torch.where(sf == 0, torch.zeros_like(y), y / torch.where(sf == 0, torch.ones_like(sf), sf))
    return _e2m1_codes(z).flatten(-2), s


def _pack(codes):
    """Two codes a byte, the even dimension in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _table(device, dtype):
    v = torch.tensor(E2M1, dtype=dtype, device=device)
    v = torch.cat([v, -v])
    b = torch.arange(256, device=device)
    return torch.stack([v[b & 15], v[b >> 4]], -1)      # byte -> (even dimension, odd dimension)


def _values(packed, scales, descale, dtype):
    """Packed codes [..., D / 2] and e4m3 scale bytes [..., D / 16] to values [..., D]."""
    v = _table(packed.device, dtype)[packed.long()].flatten(-2).unflatten(-1, (D // BLK, BLK))
    s = scales.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1)
    return (v * s * descale).flatten(-2)


# ---------------------------------------------------------------- inputs

def _randn(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _pages(gen, lengths, page=16):
    """Slots of every position: each sequence's pages are anywhere in the pool."""
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(need) + 8, generator=gen, device="cuda")
    parts, at = [], 0
    for n, k in zip(lengths, need):
        s = (order[at:at + k, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
        parts.append(s)
        at += k
    return torch.cat(parts).to(torch.int32), int(order.numel()) * page


def _cumulative(lengths):
    c = [0]
    for n in lengths:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "decode":
        lengths = _lengths(case)
        hq, hkv, b = case["hq"], case["hkv"], case["batch"]
        s["lengths"] = lengths
        s["indices"], slots = _pages(gen, lengths)
        s["indptr"] = _cumulative(lengths)
        s["kd"], s["vd"] = 1.0, 1.0
        s["k_pool"] = torch.empty(slots, hkv, D // 2, dtype=torch.uint8, device="cuda")
        s["v_pool"] = torch.empty_like(s["k_pool"])
        s["scales"] = torch.empty(slots, hkv, 2, D // BLK, dtype=torch.uint8, device="cuda")
        for at in range(0, slots, 1 << 17):
            for i, pool in enumerate((s["k_pool"], s["v_pool"])):
                x = _randn(gen, min(1 << 17, slots - at), hkv, D)
                codes, sc = _quantise(x.float(), 1.0)
                pool[at:at + (1 << 17)] = _pack(codes)
                s["scales"][at:at + (1 << 17), :, i] = sc.view(torch.uint8)
        s["q"], s["gate"] = _randn(gen, b, hq, D), _randn(gen, b, hq, D, std=2.0)
        s["sinks"] = torch.randn(hq, generator=gen, device="cuda") if case["sinks"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(b, hq, device="cuda")
        s["ws"] = torch.zeros(48 << 20, dtype=torch.uint8, device="cuda")   # a decode program's scratch
    elif op == "cache":
        t, hkv = case["tokens"], case["hkv"]
        slots = t + case["spare"]
        # K and V as the projection leaves them: parts of one row
        s["kv"] = _randn(gen, t, 2 * hkv * D)
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:t].to(torch.int32)
        s["k_pool"] = torch.zeros(slots, hkv, D // 2, dtype=torch.uint8, device="cuda")
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        s["scales"] = torch.zeros(slots, hkv, 2, D // BLK, dtype=torch.uint8, device="cuda")
        s["kd"], s["vd"] = 0.5, 0.25
    elif op == "mrope":
        t, hq, hkv, rope = case["tokens"], case["hq"], case["hkv"], case["rope"]
        slots = t + case["spare"]
        s["qgkv"] = _randn(gen, t, (2 * hq + 2 * hkv) * D)
        s["positions"] = torch.randint(0, case["far"], (case["axes"], t), generator=gen, device="cuda", dtype=torch.int32)
        s["inv_freq"] = (1e6 ** (-torch.arange(0, rope, 2, device="cuda", dtype=torch.float64) / rope)).float()
        s["axis"] = [i % case["axes"] for i in range(rope // 2)]
        s["wq"] = _randn(gen, D, std=0.1) + 1 if case["norm"] else None
        s["wk"] = _randn(gen, D, std=0.1) + 1 if case["norm"] else None
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:t].to(torch.int32)
        if case["kv"] == "bf16":
            s["k_pool"] = torch.zeros(slots, hkv, D, dtype=torch.bfloat16, device="cuda")
            s["v_pool"] = torch.zeros_like(s["k_pool"])
        elif case["kv"] == "fp4":
            s["k_pool"] = torch.zeros(slots, hkv, D // 2, dtype=torch.uint8, device="cuda")
            s["v_pool"] = torch.zeros_like(s["k_pool"])
            s["scales"] = torch.zeros(slots, hkv, 2, D // BLK, dtype=torch.uint8, device="cuda")
    else:
        nq, nk = _splits(case)
        hq, hkv = case["hq"], case["hkv"]
        s["nq"], s["nk"] = nq, nk
        s["cu_q"], s["cu_k"] = _cumulative(nq), _cumulative(nk)
        # queries and gate as two parts of the projection's rows
        rows = _randn(gen, sum(nq), 2, hq, D)
        s["q"], s["gate"] = rows[:, 0], rows[:, 1]
        s["gate"].mul_(2.0)
        s["k"], s["v"] = _randn(gen, sum(nk), hkv, D), _randn(gen, sum(nk), hkv, D)
        s["out"] = torch.empty(sum(nq), hq, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(hq, sum(nq), device="cuda")
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"decode": _decode, "cache": _cache, "mrope": _mrope, "packed": _packed}[op](s)


def _own(s, op):
    import gated_gqa_attention_gb300 as gda
    c = s["case"]
    if op == "decode":
        gda.decode_ex(s["q"], s["gate"], s["k_pool"], s["v_pool"], s["indptr"], s["indices"], out=s["out"], lse=s["lse"],
                      workspace=s["ws"], scale=1.0 / 16.0, window=c["window"], sinks=s["sinks"], kv_scales=s["scales"],
                      k_descale=s["kd"], v_descale=s["vd"], max_len=max(s["lengths"]), total_len=sum(s["lengths"]))
        return s["out"], s["lse"]
    if op == "cache":
        t, hkv = c["tokens"], c["hkv"]
        k, v = s["kv"][:, :hkv * D].view(t, hkv, D), s["kv"][:, hkv * D:].view(t, hkv, D)
        gda.kv_write_fp4(k, v, s["slots"], s["k_pool"], s["v_pool"], s["scales"], k_descale=s["kd"], v_descale=s["vd"])
        return gda.kv_gather_fp4(s["k_pool"], s["v_pool"], s["scales"], s["slots"], k_descale=s["kd"], v_descale=s["vd"])
    if op == "mrope":
        t, hq, hkv = c["tokens"], c["hq"], c["hkv"]
        gate = torch.empty(t, hq, D, dtype=torch.bfloat16, device="cuda") if c["gate"] else None
        kv = {} if c["kv"] == "none" else {"slots": s["slots"], "k_pool": s["k_pool"], "v_pool": s["v_pool"],
                                           "kv_scales": s.get("scales")}
        q, k = gda.qk_norm_mrope_kv_write(s["qgkv"], s["positions"], s["inv_freq"], s["axis"], hq, hkv, w_q_norm=s["wq"],
                                          w_k_norm=s["wk"], eps=1e-6, gate_out=gate, **kv)
        out = {"q": q, "k": k}
        if gate is not None:
            out["gate"] = gate
        if c["kv"] == "bf16":
            out["k_pool"], out["v_pool"] = s["k_pool"], s["v_pool"]
        if c["kv"] == "fp4":
            out["k4"], out["v4"] = gda.kv_gather_fp4(s["k_pool"], s["v_pool"], s["scales"], s["slots"])
        return out
    gda.prefill_packed(s["q"], s["gate"], s["k"], s["v"], s["cu_q"], cu_seqlens_k=s["cu_k"], out=s["out"], lse=s["lse"],
                       scale=1.0 / 16.0, causal=True)
    return s["out"], s["lse"]


def _gated(o, gate):
    """The gate is defined on BF16 operands: the attention result and the sigmoid are rounded, then their product,
    so that a fused call equals attention followed by the standalone gate."""
    return (o.to(torch.bfloat16).float() * torch.sigmoid(gate.float()).to(torch.bfloat16).float()).to(torch.bfloat16)


def _decode(s):
    c = s["case"]
    b, hq, hkv = c["batch"], c["hq"], c["hkv"]
    start, end = s["indptr"][:-1].long(), s["indptr"][1:].long()
    if c["window"]:
        start = torch.maximum(start, end - c["window"])
    most = max(min(x, c["window"]) if c["window"] else x for x in s["lengths"])
    pos = start[:, None] + torch.arange(most, device="cuda")
    valid = pos < end[:, None]                                                   # [B, L]
    slot = s["indices"].long()[pos.clamp(max=s["indices"].numel() - 1)]
    slot = torch.where(valid, slot, torch.zeros_like(slot))
    # [B, L, Hkv, D] -> [B, Hkv, L, D]
    k = _values(s["k_pool"][slot], s["scales"][:, :, 0][slot], s["kd"], torch.float32).transpose(1, 2)
    q = s["q"].float().view(b, hkv, hq // hkv, D)
    score = (q @ k.transpose(2, 3)) * (1.0 / 16.0)                               # [B, Hkv, G, L]
    del k
    score = score.masked_fill(~valid[:, None, None, :], -math.inf)
    top = score.amax(-1)
    if s["sinks"] is not None:
        top = torch.maximum(top, s["sinks"].view(hkv, -1))
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - safe[..., None])
    total = p.sum(-1)
    if s["sinks"] is not None:
        total = total + torch.exp(s["sinks"].view(hkv, -1) - safe)
    v = _values(s["v_pool"][slot], s["scales"][:, :, 1][slot], s["vd"], torch.float32).transpose(1, 2)
    o = p @ v
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o)).view(b, hq, D)
    lse = (safe + torch.log(total)).view(b, hq)
    return _gated(o, s["gate"]), lse


def _cache(s):
    c = s["case"]
    t, hkv = c["tokens"], c["hkv"]
    slot = s["slots"].long()
    kv = s["kv"].float().view(t, 2, hkv, D)
    for i, (pool, d) in enumerate(((s["k_pool"], s["kd"]), (s["v_pool"], s["vd"]))):
        codes, sc = _quantise(kv[:, i], d)
        pool[slot] = _pack(codes)
        s["scales"][slot, :, i] = sc.view(torch.uint8)
    return (_values(s["k_pool"][slot], s["scales"][slot][:, :, 0], s["kd"], torch.float32).to(torch.bfloat16),
            _values(s["v_pool"][slot], s["scales"][slot][:, :, 1], s["vd"], torch.float32).to(torch.bfloat16))


def _norm_rotate(x, w, cos, sin, rope, eps=1e-6):
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.to(x.dtype)
    a, b, rest = x[..., :rope // 2], x[..., rope // 2:rope], x[..., rope:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _mrope(s):
    c = s["case"]
    t, hq, hkv, rope = c["tokens"], c["hq"], c["hkv"], c["rope"]
    x = s["qgkv"].float().view(t, 2 * hq + 2 * hkv, D)
    # far positions times a frequency lose the angle in 32 bits
    angle = s["positions"].double()[s["axis"]].t() * s["inv_freq"].double()      # [T, rope / 2]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _norm_rotate(x[:, :hq], s["wq"], cos, sin, rope).to(torch.bfloat16)
    k = _norm_rotate(x[:, 2 * hq:2 * hq + hkv], s["wk"], cos, sin, rope).to(torch.bfloat16)
    v = s["qgkv"].view(t, 2 * hq + 2 * hkv, D)[:, 2 * hq + hkv:]
    out = {"q": q, "k": k}
    if c["gate"]:
        out["gate"] = s["qgkv"].view(t, 2 * hq + 2 * hkv, D)[:, hq:2 * hq].contiguous()
    slot = s["slots"].long()
    if c["kv"] == "bf16":
        s["k_pool"][slot], s["v_pool"][slot] = k, v
        out["k_pool"], out["v_pool"] = s["k_pool"], s["v_pool"]
    if c["kv"] == "fp4":
        for i, (name, pool, rows) in enumerate((("k4", s["k_pool"], k), ("v4", s["v_pool"], v))):
            codes, sc = _quantise(rows.float(), 1.0)
            pool[slot] = _pack(codes)
            s["scales"][slot, :, i] = sc.view(torch.uint8)
            out[name] = _values(pool[slot], s["scales"][slot][:, :, i], 1.0, torch.float32).to(torch.bfloat16)
    return out


def _packed(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    tq, tk = s["q"].shape[0], s["k"].shape[0]
    iq, ik = torch.arange(tq, device="cuda"), torch.arange(tk, device="cuda")
    seq_q = torch.bucketize(iq, s["cu_q"][1:].long(), right=True)
    seq_k = torch.bucketize(ik, s["cu_k"][1:].long(), right=True)
    # positions counted from each sequence's end: query i sees the keys that are not nearer to it
    left_q, left_k = s["cu_q"][1:].long()[seq_q] - iq, s["cu_k"][1:].long()[seq_k] - ik
    hidden = (seq_q[:, None] != seq_k[None]) | (left_k[None] < left_q[:, None])  # [Tq, Tk]
    q = s["q"].float().view(tq, hkv, hq // hkv, D).permute(1, 2, 0, 3)           # [Hkv, G, Tq, D]
    k, v = s["k"].float().permute(1, 0, 2)[:, None], s["v"].float().permute(1, 0, 2)[:, None]
    score = (q @ k.transpose(2, 3)).mul_(1.0 / 16.0).masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = ((p @ v) / total).permute(2, 0, 1, 3).reshape(tq, hq, D)
    lse = (top + torch.log(total)).view(hq, tq)
    return _gated(o, s["gate"]), lse


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "cache": _exact_cache, "mrope": _exact_mrope, "packed": _exact_packed}[case["op"]](s)


def _nibbles64(packed, scales, descale):
    """Values of packed rows in 64 bits, one half byte after the other."""
    mag = torch.tensor(E2M1, dtype=torch.float64, device=packed.device)
    out = torch.empty(*packed.shape[:-1], D, dtype=torch.float64, device=packed.device)
    for half in (0, 1):
        n = (packed >> (4 * half)) & 15
        out[..., half::2] = mag[(n & 7).long()] * (1.0 - 2.0 * (n >> 3).double())
    return out * scales.view(torch.float8_e4m3fn).double().repeat_interleave(BLK, -1) * descale


def _exact_decode(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    out = torch.zeros(c["batch"], hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(s["lengths"]):
        first = at + (max(0, n - c["window"]) if c["window"] else 0)
        slot = s["indices"][first:at + n].long()
        at += n
        k = _nibbles64(s["k_pool"][slot], s["scales"][slot, :, 0], s["kd"])
        v = _nibbles64(s["v_pool"][slot], s["scales"][slot, :, 1], s["vd"])
        for h in range(hkv):
            rows = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            score = s["q"][b, rows].double() @ k[:, h].t() / 16.0
            if s["sinks"] is not None:
                score = torch.cat([score, s["sinks"][rows].double()[:, None]], 1)
            if score.shape[1] == 0:
                continue
            lse[b, rows] = torch.logsumexp(score, 1)
            out[b, rows] = torch.softmax(score, 1)[:, :k.shape[0]] @ v[:, h]
    return out / (1.0 + torch.exp(-s["gate"].double())), lse


def _quantised64(x, descale):
    """Each value of x as the 4-bit cache holds it, from the format's definition."""
    y = x.double().unflatten(-1, (D // BLK, BLK)) / descale
    scale = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0)
    # nearest e4m3 value: three bits after the leading one, steps of 2^-9 below 2^-6, ties to even
    step = torch.exp2(torch.floor(torch.log2(scale.clamp(min=2.0 ** -6))) - 3)
    scale = torch.round(scale / step) * step
    z = torch.where(scale > 0, y / scale.clamp(min=2.0 ** -9), torch.zeros_like(y))
    a = z.abs().clamp(max=6.0)
    # nearest e2m1 value: steps of 1/2 below 2, 1 below 4, 2 up to 6, ties to even
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    return (torch.round(a / step) * step * torch.sign(z) * scale * descale).flatten(-2)


def _exact_cache(s):
    kv = s["kv"].view(s["case"]["tokens"], 2, s["case"]["hkv"], D)
    return _quantised64(kv[:, 0], s["kd"]), _quantised64(kv[:, 1], s["vd"])


def _exact_mrope(s):
    c = s["case"]
    t, hq, hkv, half = c["tokens"], c["hq"], c["hkv"], c["rope"] // 2
    x = s["qgkv"].double().view(t, 2 * hq + 2 * hkv, D)
    pos = torch.stack([s["positions"][a] for a in s["axis"]], 1).double()
    turn = torch.polar(torch.ones_like(pos), pos * s["inv_freq"].double())[:, None]
    res = {}
    for name, rows, w in (("q", x[:, :hq], s["wq"]), ("k", x[:, 2 * hq:2 * hq + hkv], s["wk"])):
        if w is not None:
            rows = rows / torch.sqrt(rows.pow(2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        z = torch.complex(rows[..., :half], rows[..., half:2 * half]) * turn
        res[name] = torch.cat([z.real, z.imag, rows[..., 2 * half:]], -1)
    v = x[:, 2 * hq + hkv:]
    slot = s["slots"].long()
    if c["gate"]:
        res["gate"] = x[:, hq:2 * hq].contiguous()
    if c["kv"] == "bf16":
        for name, rows in (("k_pool", res["k"]), ("v_pool", v)):
            res[name] = s[name].double()
            res[name][slot] = rows
    if c["kv"] == "fp4":
        # the cache takes the BF16 key; its quantised value jumps where the key is next to a border
        res["k4"], res["v4"] = None, _quantised64(v, 1.0)
    return res


def _exact_packed(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(hq, s["q"].shape[0], dtype=torch.float64, device="cuda")
    aq = ak = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        seen = torch.ones(nq, nk, dtype=torch.bool, device="cuda").tril(nk - nq)
        for h in range(hq):
            g = h // (hq // hkv)
            score = s["q"][aq:aq + nq, h].double() @ s["k"][ak:ak + nk, g].double().t() / 16.0
            score.masked_fill_(~seen, -math.inf)
            lse[h, aq:aq + nq] = torch.logsumexp(score, 1)
            out[aq:aq + nq, h] = torch.softmax(score, 1) @ s["v"][ak:ak + nk, g].double()
        aq, ak = aq + nq, ak + nk
    return out / (1.0 + torch.exp(-s["gate"].double())), lse
