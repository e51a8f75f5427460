"""Attention over a paged cache and the 8-bit cache's format in float64 from their formulas (torch, any
device), written apart from the kernels: what the tests compare with."""
import math

import torch

import plain64
from plain64 import D, E4M3


def quantise8(x, descale=1.0):
    """e4m3 codes of x / descale (the quotient in float32, IEEE): nearest, ties to even, beyond 448 to 448."""
    y = x.float().cpu() / torch.tensor(descale, dtype=torch.float32)
    code = plain64.nearest(y.double(), E4M3).to(torch.uint8) + 128 * torch.signbit(y).to(torch.uint8)
    return torch.where(torch.isnan(y), torch.full_like(code, 0x7F) | (code & 0x80), code)


def values8(codes, descale=1.0):
    c = codes.cpu().view(torch.uint8)
    v = torch.cat([E4M3, torch.tensor([math.nan], dtype=torch.float64)])[(c & 127).long()]
    return v * (1.0 - 2.0 * (c >> 7).double()) * float(torch.tensor(descale, dtype=torch.float32))


def paged(q, gate, k_rows, v_rows, cu, indptr, indices, scale, window=0, keep_first=0, sinks=None, fill=math.nan):
    """k_rows, v_rows: float64 [slots, Hkv, D] (descales applied) on q's device; a slot outside them is a row of
    zeros.  Rows of no sequence: ``fill``."""
    Tq, Hq, _ = q.shape
    dev = q.device
    n_slots, Hkv, _ = k_rows.shape
    G = Hq // Hkv
    a = plain64.Attn(Tq, Hq, device=dev, fill=fill)
    cu, ip = cu.tolist(), indptr.tolist()
    zero = torch.zeros(1, Hkv, D, dtype=torch.float64, device=dev)
    for b in range(len(cu) - 1):
        n, L = cu[b + 1] - cu[b], ip[b + 1] - ip[b]
        if n <= 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        p = torch.arange(L - n, L, device=dev)[:, None]
        j = torch.arange(L, device=dev)[None]
        seen = j <= p
        if window:
            seen = seen & ((j > p - window) | (j < keep_first))
        slot = indices[ip[b]:ip[b + 1]].long().to(dev)
        bad = (slot < 0) | (slot >= n_slots)
        slot = torch.where(bad, torch.full_like(slot, n_slots), slot)
        # only what some query sees (other rows may hold anything)
        some = seen.any(0)
        slot, seen = slot[some], seen[:, some]
        for h in range(Hq):
            k = torch.cat([k_rows[:, h // G], zero[:, 0]])[slot]
            v = torch.cat([v_rows[:, h // G], zero[:, 0]])[slot]
            qh = q[rows, h].double()
            s = (scale * (qh @ k.t())).masked_fill(~seen, -math.inf)
            top = s.amax(1) if s.shape[1] else torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
            if sinks is not None:
                top = torch.maximum(top, sinks[h].double().to(dev))
            base = torch.where(top == -math.inf, torch.zeros_like(top), top)
            e = torch.exp(s - base[:, None])
            total = e.sum(1)
            if sinks is not None:
                total = total + torch.exp(sinks[h].double().to(dev) - base)
            w = torch.where(total[:, None] > 0, e / total[:, None], torch.zeros_like(e))
            a.out[rows, h], a.pv[rows, h] = w @ v, w @ v.abs()
            a.lse[rows, h] = base + torch.log(total)
            if s.shape[1]:
                a.sabs[rows, h] = scale * (qh.abs() @ k.abs().t()).masked_fill(~seen, 0.0).amax(1)
    return a.gated(gate)
