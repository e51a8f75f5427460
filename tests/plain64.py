"""The prompt and 4-bit-cache operators in float64 from their formulas (torch, any device),
written apart from the kernels: what the tests compare with."""
import math

import torch

D, BLK = 256, 16
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# the 127 finite values of e4m3 from 0 up (torch's own decoding of the 8-bit codes)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def nearest(x, table):
    """Index of the table value (ascending from 0) nearest to each |x|, ties to the even index; beyond the
    last value the last.  Even indexes are the codes whose last bit is 0."""
    a = x.abs().clamp(max=float(table[-1]))
    hi = torch.searchsorted(table, a).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - table[lo], table[hi] - a
    return torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))


def quantise(x, descale=1.0):
    """[..., D] values -> (code bytes [..., D/2], scale bytes [..., D/16]).  The formula divides in
    float32; y / s and max / 6 are taken in float32 here too (IEEE division of float32 operands)."""
    y = (x.float().cpu() / torch.tensor(descale, dtype=torch.float32)).unflatten(-1, (D // BLK, BLK))
    nan = torch.isnan(y).any(-1)
    top = torch.where(torch.isnan(y), torch.zeros_like(y), y.abs()).amax(-1)
    s = nearest((top / torch.tensor(6.0)).double(), E4M3)
    sf = E4M3[s].float()[..., None]
    z = torch.where(sf > 0, y / torch.where(sf > 0, sf, torch.ones_like(sf)), torch.zeros_like(y))
    z = torch.where(nan[..., None], torch.zeros_like(z), z)
    c = nearest(z.double(), E2M1) + 8 * ((z < 0) | ((z == 0) & torch.signbit(z))).long()
    c = c.flatten(-2).to(torch.uint8)
    s = torch.where(nan, torch.full_like(s, 0x7F), s).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def values(codes, scales, descale=1.0):
    """Code bytes [..., D/2] and scale bytes [..., D/16] -> float64 [..., D]."""
    codes, scales = codes.cpu(), scales.cpu()
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = E2M1[c & 7] * (1.0 - 2.0 * (c >> 3).double())
    s = scales.contiguous().view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(BLK, -1) * float(torch.tensor(descale, dtype=torch.float32))


def sigmoid(g):
    return 1.0 / (1.0 + torch.exp(-g.double()))


class Attn:
    """What an attention call is compared with, in float64: out (gated if there is a gate), lse, and the
    two sums that the bounds below need -- pv = sum_j p_j |v_j| (times the gate's sigmoid) and
    sabs = the largest scale * sum_d |q_d k_d| over the visible keys."""

    def __init__(self, *shape, device="cpu", fill=0.0):
        f = dict(dtype=torch.float64, device=device)
        self.out = torch.full((*shape, D), fill, **f)
        self.pv = torch.full((*shape, D), fill, **f)
        self.lse = torch.full(shape, -math.inf if fill == 0.0 else fill, **f)
        self.sabs = torch.zeros(shape, **f)

    def gated(self, gate):
        if gate is not None:
            s = sigmoid(gate.to(self.out.device))
            self.out, self.pv = self.out * s, self.pv * s
        return self


def bound_out(a: Attn, p_step, n):
    """Largest |error| of an output.  Probabilities are rounded to p_step relative (FP16 2^-11, BF16 2^-8; below
    FP16's normal range 2^-25 absolute, n of them against a sum of at least 1); scores carry 16 FP32 accumulations
    and a few FP32 steps, 2^-19 of sabs, which move a probability and the sum by that much each (twice: 2^-18), plus
    the FP32 exponentials and sums, 2^-18; then O, the sigmoid and the product are rounded to BF16, half a step
    (2^-8) each, plus the second-order terms (0.02 of it)."""
    rel = p_step + 2.0 ** -18 * (1 + a.sabs[..., None])
    vmax = a.pv.abs().amax() if a.pv.numel() else 0.0
    return rel * a.pv + n * 2.0 ** -25 * vmax + 3.06 * 2.0 ** -8 * a.out.abs() + 1e-30


def bound_lse(a: Attn):
    """Scores as above (2^-19 of sabs), the sum's relative error 2^-18 and the final FP32 steps."""
    return 2.0 ** -19 * a.sabs + 2.0 ** -18 + 2.0 ** -21 * torch.where(a.lse.isfinite(), a.lse.abs(), 0.0)


def check(out, lse, a: Attn, p_step, n, what=""):
    got, want = out.to(a.out.device).double(), a.out
    err, tol = (got - want).abs(), bound_out(a, p_step, n)
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d outputs off, worst %.3g of the bound" % (what, int(bad.sum()), float((err / tol).max()))
    if lse is None:
        return
    got = lse.to(a.lse.device).double()
    dead = a.lse == -math.inf
    assert torch.equal(got == -math.inf, dead), "%s: dead rows" % what
    err = (got - a.lse).abs()[~dead]
    bad = ~(err <= bound_lse(a)[~dead])
    assert not bad.any(), "%s: %d lse off, worst %.3g" % (what, int(bad.sum()), float(err.max()))


def decode(q, gate, k_rows, v_rows, indptr, indices, scale, window=0, sinks=None):
    """k_rows, v_rows: float64 [slots, Hkv, D] (descales applied); all on the CPU."""
    B, Hq, _ = q.shape
    G = Hq // k_rows.shape[1]
    a = Attn(B, Hq)
    ip = indptr.tolist()
    for b in range(B):
        i0, i1 = ip[b], ip[b + 1]
        if window:
            i0 = max(i0, i1 - window)
        rows = indices[i0:i1].long()
        for h in range(Hq):
            k, v = k_rows[rows, h // G], v_rows[rows, h // G]
            s = scale * (k @ q[b, h].double())
            if sinks is not None:
                s = torch.cat([s, sinks[h:h + 1].double()])
            if s.numel() == 0:
                continue
            a.lse[b, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - a.lse[b, h])[:i1 - i0]
            a.out[b, h], a.pv[b, h] = p @ v, p @ v.abs()
            if i1 > i0:
                a.sabs[b, h] = scale * (k.abs() @ q[b, h].double().abs()).max()
    return a.gated(gate)


def packed(q, gate, k, v, cu_q, cu_k, scale, causal):
    """Rows of no sequence: NaN."""
    Tq, Hq, _ = q.shape
    G = Hq // k.shape[1]
    a = Attn(Tq, Hq, device=q.device, fill=math.nan)
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cq) - 1):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        seen = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
        if causal:
            seen = seen.tril(nk - nq)
        for h in range(Hq):
            if nk == 0:
                a.out[rq, h] = a.pv[rq, h] = 0.0
                a.lse[rq, h] = -math.inf
                continue
            qh, kh, vh = q[rq, h].double(), k[rk, h // G].double(), v[rk, h // G].double()
            s = (scale * (qh @ kh.t())).masked_fill(~seen, -math.inf)
            l = torch.logsumexp(s, 1)
            p = torch.exp(s - torch.where(l == -math.inf, torch.zeros_like(l), l)[:, None])
            a.out[rq, h], a.pv[rq, h], a.lse[rq, h] = p @ vh, p @ vh.abs(), l
            a.sabs[rq, h] = scale * (qh.abs() @ kh.abs().t()).masked_fill(~seen, 0.0).amax(1)
    return a.gated(gate)


def norm_rope(x, w, eps, angle):
    """x: [T, H, D]; angle: [T, rope_dim/2] in float64 (None: no rotation)."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    if angle is None or angle.shape[1] == 0:
        return x
    r = angle.shape[1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :r], x[..., r:2 * r]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * r:]], -1)
