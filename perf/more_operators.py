"""Timed cases of attention over a paged cache for chunks of new tokens, and of the 8-bit cache's writes.

Three groups of cases, each with a plain form (elementary torch operations in 32 bits) and the
library's calls:

* ``paged``:  gated causal attention of each sequence's newest tokens over its cache rows
              (``prefill_paged``), for BF16, 8-bit (e4m3) and 4-bit caches;
* ``window``: the same with a sliding window and a few first tokens that stay visible;
* ``cache``:  K and V rows quantised into an 8-bit cache and read back as BF16 rows
              (``kv_write_e4m3``, ``kv_gather_e4m3``).
"""
import math
import random

import torch

own = False

D = 256
BLK = 16                     # head dimensions per scale of the 4-bit cache
ROW = {"bf16": 2 * 2 * D, "e4m3": 2 * D, "fp4": D + 2 * (D // BLK)}   # bytes of one (slot, KV head), K and V
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def _case(name, op, batch, t, before, hq=16, hkv=2, kv="bf16", window=0, first=0, sinks=False, seed=1):
    """``t`` and ``before``: ranges of a sequence's new tokens and of the positions in the cache before them."""
    return {"name": name, "op": op, "batch": batch, "t_lo": t[0], "t_hi": t[1], "p_lo": before[0], "p_hi": before[1],
            "hq": hq, "hkv": hkv, "kv": kv, "window": window, "first": first, "sinks": sinks, "draw": seed}


def listed():
    return [
        # one user's next token, the shortest call: latency
        _case("paged_b1_t1_l512", "paged", 1, (1, 1), (511, 511)),
        # 32 users, each with a token and four drafted ones to be checked
        _case("paged_b32_t5", "paged", 32, (5, 5), (2000, 4096), seed=2),
        # the same for more users of every length, with an 8-bit cache
        _case("paged_b64_t4_e4m3", "paged", 64, (4, 4), (0, 8192), kv="e4m3", seed=3),
        # a server's mixed step: chunks of prompts beside users' next tokens, 16 query heads to a KV head, 4-bit cache
        _case("paged_b9_mix_fp4", "paged", 9, (1, 1500), (0, 6000), hq=32, kv="fp4", seed=4),
        # chunks of four documents with an 8-bit cache
        _case("paged_b4_t512_e4m3", "paged", 4, (512, 512), (7000, 8192), kv="e4m3", seed=5),
        # one chunk of a long document
        _case("paged_b1_t2048_l34816", "paged", 1, (2048, 2048), (32768, 32768), seed=6),
        # a decode step of 64 long chats that keep a window and the first four tokens
        _case("window_b64_t1_l16384", "window", 64, (1, 1), (16383, 16383), window=4096, first=4, seed=7),
        # drafted tokens over an odd window, every length, one query head to a KV head, sink logits, 8-bit cache
        _case("window_b16_t3_e4m3", "window", 16, (1, 3), (500, 20000), hq=8, hkv=8, kv="e4m3", window=2047, first=5,
              sinks=True, seed=8),
        # two new prompts under a window: the band of the score matrix is all there is to do
        _case("window_b2_t4097", "window", 2, (4097, 4097), (0, 0), window=1024, first=16, seed=9),
        # the new tokens of a decode step go into the cache
        {"name": "cache_t64", "op": "cache", "tokens": 64, "hkv": 2, "spare": 1024},
        # a chunk's rows, four KV heads
        {"name": "cache_t2047", "op": "cache", "tokens": 2047, "hkv": 4, "spare": 333},
        # a whole prompt's rows
        {"name": "cache_t16384", "op": "cache", "tokens": 16384, "hkv": 2, "spare": 4096},
    ]


_MOST_PAIRS = 16 * 2048 * 32768      # query heads times visible (query, key) pairs: the largest listed case's
_MOST_ROWS = 64 * 16384 * 2          # (position, KV head) rows of BF16 pools: likewise


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["paged", "paged", "paged", "window", "window", "cache"])
    if op == "cache":
        hkv = rng.choice([1, 2, 4])
        return {"op": op, "tokens": _log_int(rng, 1, 32768 // hkv), "hkv": hkv, "spare": rng.randrange(1, 2000)}
    hq, hkv = rng.choice([(16, 2), (16, 2), (32, 2), (8, 1), (12, 4), (8, 8)])
    if rng.random() < 0.5:           # steps: few tokens of many users
        batch = _log_int(rng, 1, 224)
        t_hi = rng.choice([1, 2, 4, 5, 8, 16])
    else:                            # chunks of prompts
        batch = _log_int(rng, 1, 8)
        t_hi = _log_int(rng, 16, 4096 // batch)
    p_hi = _log_int(rng, 1, max(1, min(65536, _MOST_ROWS // (2 * batch * hkv), _MOST_PAIRS // (batch * t_hi * hq) - t_hi)))
    window, first = 0, 0
    if op == "window":
        window = _log_int(rng, 1, p_hi + t_hi)
        first = rng.choice([0, 1, 4, 64, 130])
    return {"op": op, "batch": batch, "t_lo": rng.choice([0, 1, t_hi]), "t_hi": t_hi, "p_lo": rng.choice([0, p_hi // 2, p_hi]),
            "p_hi": p_hi, "hq": hq, "hkv": hkv, "kv": rng.choice(["bf16", "e4m3", "fp4"]), "window": window, "first": first,
            "sinks": rng.random() < 0.3, "draw": rng.randrange(1 << 30)}


def _lengths(case):
    """Each sequence's new tokens and positions in all: they follow from the case."""
    r = random.Random(case["draw"])
    nq = [r.randint(case["t_lo"], case["t_hi"]) for _ in range(case["batch"])]
    nq[0] = max(1, nq[0])
    return nq, [n + r.randint(case["p_lo"], case["p_hi"]) for n in nq]


def _seen(p, window, first):
    """Keys that the query at position p sees."""
    if not window:
        return p + 1
    return min(p + 1, window) + min(first, max(0, p + 1 - window))


def _band(n, total, window, first):
    """Positions that any of the last n of `total` positions sees."""
    if not n:
        return 0
    low = max(0, total - n + 1 - window) if window else 0
    return total - low + min(first, low)


def work(case):
    if case["op"] == "cache":
        return {"bytes": case["tokens"] * (case["hkv"] * 2 * (2 * 2 * D + D + D) + 8), "flops": 0}
    w, f = case["window"], case["first"]
    pairs = rows = 0
    for n, total in zip(*_lengths(case)):
        pairs += sum(_seen(p, w, f) for p in range(total - n, total))
        rows += _band(n, total, w, f)
    t = sum(_lengths(case)[0]) * case["hq"]
    return {"bytes": rows * (case["hkv"] * ROW[case["kv"]] + 4) + t * (3 * 2 * D + 4), "flops": 4 * D * case["hq"] * pairs}


# ---------------------------------------------------------------- the caches' formats, plainly

def _quantise8(x, descale):
    """Values as e4m3 codes: nearest, ties to even, beyond 448 to 448."""
    return (x / descale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _e2m1_codes(x):
    """Codes of values already divided by their scale: nearest, ties to the even code, beyond 6 to 6."""
    a = x.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8))
    return code | ((x < 0).to(torch.uint8) << 3)


def _quantise4(x, descale):
    """[..., D] values to (packed codes [..., D / 2], e4m3 scale bytes [..., D / 16])."""
    y = (x / descale).unflatten(-1, (D // BLK, BLK))
    s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.to(y.dtype).unsqueeze(-1)
    z = torch.where(sf == 0, torch.zeros_like(y), y / torch.where(sf == 0, torch.ones_like(sf), sf))
    codes = _e2m1_codes(z).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), s.view(torch.uint8)


def _values4(packed, scales, descale):
    """Packed codes [..., D / 2] and e4m3 scale bytes [..., D / 16] to values [..., D]."""
    v = torch.tensor(E2M1, device=packed.device)
    v = torch.cat([v, -v])
    b = torch.arange(256, device=packed.device)
    table = torch.stack([v[b & 15], v[b >> 4]], -1)      # byte -> (even dimension, odd dimension)
    x = table[packed.long()].flatten(-2).unflatten(-1, (D // BLK, BLK))
    return (x * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1) * descale).flatten(-2)


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
    s = {"case": case}
    hkv = case["hkv"]
    if case["op"] == "cache":
        t = case["tokens"]
        slots = t + case["spare"]
        # K and V as the projection leaves them: parts of one row
        s["kv"] = _randn(gen, t, 2 * hkv * D)
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:t].to(torch.int32)
        s["k_pool"] = torch.zeros(slots, hkv, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        s["kd"], s["vd"] = 0.03125, 0.011
        return s
    nq, nk = _lengths(case)
    hq, kv = case["hq"], case["kv"]
    s["nq"], s["nk"] = nq, nk
    s["cu"], s["indptr"] = _cumulative(nq), _cumulative(nk)
    s["indices"], slots = _pages(gen, nk)
    # queries and gate as two parts of the projection's rows
    rows = _randn(gen, sum(nq), 2, hq, D)
    s["q"], s["gate"] = rows[:, 0], rows[:, 1]
    s["gate"].mul_(2.0)
    s["kd"], s["vd"], s["scales"] = (1.0, 1.0, None) if kv == "bf16" else (0.5, 0.25, None)
    if kv == "fp4":
        s["scales"] = torch.empty(slots, hkv, 2, D // BLK, dtype=torch.uint8, device="cuda")
    width, dtype = {"bf16": (D, torch.bfloat16), "e4m3": (D, torch.float8_e4m3fn), "fp4": (D // 2, torch.uint8)}[kv]
    for i, (name, d) in enumerate((("k_pool", s["kd"]), ("v_pool", s["vd"]))):
        pool = s[name] = torch.empty(slots, hkv, width, dtype=dtype, device="cuda")
        for at in range(0, slots, 1 << 18):
            x = _randn(gen, min(1 << 18, slots - at), hkv, D)
            end = at + x.shape[0]
            if kv == "bf16":
                pool[at:end] = x
            elif kv == "e4m3":
                pool[at:end] = _quantise8(x.float(), d)
            else:
                pool[at:end], s["scales"][at:end, :, i] = _quantise4(x.float(), d)
    s["sinks"] = torch.randn(hq, generator=gen, device="cuda") if case["sinks"] else None
    s["out"] = torch.empty(sum(nq), hq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(hq, sum(nq), device="cuda")
    s["ws"] = None
    if own:
        import gated_gqa_attention_gb300 as gda
        # a serving program's scratch for this call
        n = gda.prefill_paged_workspace_bytes(sum(nq), case["batch"], hq, hkv, D)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    if own:
        return _own(s)
    return _cache(s) if s["case"]["op"] == "cache" else _paged(s)


def _own(s):
    import gated_gqa_attention_gb300 as gda
    c = s["case"]
    if c["op"] == "cache":
        t, hkv = c["tokens"], c["hkv"]
        k, v = s["kv"][:, :hkv * D].view(t, hkv, D), s["kv"][:, hkv * D:].view(t, hkv, D)
        gda.kv_write_e4m3(k, v, s["slots"], s["k_pool"], s["v_pool"], k_descale=s["kd"], v_descale=s["vd"])
        return gda.kv_gather_e4m3(s["k_pool"], s["v_pool"], s["slots"], k_descale=s["kd"], v_descale=s["vd"])
    gda.prefill_paged(s["q"], s["gate"], s["k_pool"], s["v_pool"], s["cu"], s["indptr"], s["indices"], out=s["out"],
                      lse=s["lse"], scale=1.0 / 16.0, window=c["window"], keep_first=c["first"], sinks=s["sinks"],
                      kv_scales=s["scales"], k_descale=s["kd"], v_descale=s["vd"], workspace=s["ws"])
    return s["out"], s["lse"]


def _gated(o, gate):
    """The gate is defined on BF16 operands: the attention result and the sigmoid are rounded, then their product,
    so that a fused call equals attention followed by the standalone gate."""
    return (o.to(torch.bfloat16).float() * torch.sigmoid(gate.float()).to(torch.bfloat16).float()).to(torch.bfloat16)


def _rows(s, slot, i):
    """The K (i = 0) or V (i = 1) rows of the slots: [Hkv, L, D] in 32 bits."""
    pool, d = (s["k_pool"], s["kd"]) if i == 0 else (s["v_pool"], s["vd"])
    kv = s["case"]["kv"]
    if kv == "fp4":
        x = _values4(pool[slot], s["scales"][slot, :, i], d)
    elif kv == "e4m3":
        x = pool.view(torch.uint8)[slot].view(torch.float8_e4m3fn).float() * d
    else:
        x = pool[slot].float()
    return x.transpose(0, 1)


def _paged(s):
    c = s["case"]
    hq, hkv, window, first = c["hq"], c["hkv"], c["window"], c["first"]
    g = hq // hkv
    o = torch.zeros(sum(s["nq"]), hq, D, device="cuda")
    lse = torch.full((hq, sum(s["nq"])), -math.inf, device="cuda")
    aq = ak = 0
    for n, total in zip(s["nq"], s["nk"]):
        slot = s["indices"][ak:ak + total].long()
        rows = slice(aq, aq + n)
        aq, ak = aq + n, ak + total
        if n == 0:
            continue
        k, v = _rows(s, slot, 0), _rows(s, slot, 1)
        p = torch.arange(total - n, total, device="cuda")[:, None]
        j = torch.arange(total, device="cuda")[None]
        hidden = j > p
        if window:
            hidden |= (j <= p - window) & (j >= first)
        for h in range(hkv):
            heads = slice(h * g, (h + 1) * g)
            q = s["q"][rows, heads].float().transpose(0, 1)                          # [G, n, D]
            score = (q @ k[h].t()).mul_(1.0 / 16.0).masked_fill_(hidden, -math.inf)  # [G, n, L]
            top = score.amax(-1, keepdim=True)
            if s["sinks"] is not None:
                top = torch.maximum(top, s["sinks"][heads].view(g, 1, 1))
            e = score.sub_(top).exp_()
            sum_e = e.sum(-1, keepdim=True)
            if s["sinks"] is not None:
                sum_e = sum_e + torch.exp(s["sinks"][heads].view(g, 1, 1) - top)
            o[rows, heads] = ((e @ v[h]) / sum_e).transpose(0, 1)
            lse[heads, rows] = (top + torch.log(sum_e)).squeeze(-1)
    return _gated(o, s["gate"]), lse


def _cache(s):
    c = s["case"]
    slot = s["slots"].long()
    kv = s["kv"].float().view(c["tokens"], 2, c["hkv"], D)
    out = []
    for i, (pool, d) in enumerate(((s["k_pool"], s["kd"]), (s["v_pool"], s["vd"]))):
        raw = pool.view(torch.uint8)
        raw[slot] = _quantise8(kv[:, i], d).view(torch.uint8)
        out.append((raw[slot].view(torch.float8_e4m3fn).float() * d).to(torch.bfloat16))
    return tuple(out)


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_cache(s) if case["op"] == "cache" else _exact_paged(s)


def _exact_cache(s):
    """Each value as the 8-bit cache holds it: three bits after the leading one, steps of 2^-9 below 2^-6."""
    kv = s["kv"].view(s["case"]["tokens"], 2, s["case"]["hkv"], D)
    res = []
    for i, d in enumerate((s["kd"], s["vd"])):
        d = float(torch.tensor(d, dtype=torch.float32))      # the descale is a 32-bit argument
        y = kv[:, i].double() / d
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        res.append((torch.round(y / step) * step).clamp(-448.0, 448.0) * d)
    return tuple(res)


def _exact_rows(s, slot, i, h):
    pool, d = (s["k_pool"], s["kd"]) if i == 0 else (s["v_pool"], s["vd"])
    kv = s["case"]["kv"]
    if kv == "bf16":
        return pool[slot, h].double()
    raw = pool.view(torch.uint8)[slot, h]
    if kv == "e4m3":
        return raw.view(torch.float8_e4m3fn).double() * d
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    x = torch.empty(slot.numel(), D, dtype=torch.float64, device="cuda")
    for half in (0, 1):
        n = (raw >> (4 * half)) & 15
        x[:, half::2] = mag[(n & 7).long()] * (1.0 - 2.0 * (n >> 3).double())
    return x * s["scales"][slot, h, i].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(BLK, -1) * d


def _exact_paged(s):
    c = s["case"]
    hq, g, window, first = c["hq"], c["hq"] // c["hkv"], c["window"], c["first"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, total) in enumerate(zip(s["nq"], s["nk"])):
        at = sum(s["nk"][:b])
        if n == 0:
            continue
        seen = torch.ones(n, total, dtype=torch.bool, device="cuda").tril(total - n)
        if window:
            seen &= torch.ones_like(seen).triu(total - n - window + 1) | (torch.arange(total, device="cuda") < first)
        # positions that no query sees are left out
        some = seen.any(0)
        slot, seen = s["indices"][at:at + total].long()[some], seen[:, some]
        for h in range(hq):
            if h % g == 0:
                k, v = _exact_rows(s, slot, 0, h // g), _exact_rows(s, slot, 1, h // g)
            score = (s["q"][start:start + n, h].double() @ k.t() / 16.0).masked_fill_(~seen, -math.inf)
            if s["sinks"] is not None:
                score = torch.cat([score, s["sinks"][h].double().expand(n, 1)], 1)
            lse[h, start:start + n] = torch.logsumexp(score, 1)
            out[start:start + n, h] = torch.softmax(score, 1)[:, :v.shape[0]] @ v
        start += n
    return out / (1.0 + torch.exp(-s["gate"].double())), lse
