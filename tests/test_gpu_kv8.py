"""Writing the 8-bit KV cache and reading it back on the GPU.  Stored codes follow from the formula bit
for bit (an IEEE division, a rounding to nearest even), and so do the rows read back."""
import pytest
import torch

import paged64
from canary import Guarded, check_all

pytestmark = pytest.mark.gpu
D = 256


def cache(slots, Hkv, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)
    return r(slots, Hkv, D), r(slots, Hkv, D)


def rows(kind, T, Hkv, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "normal":
        return torch.randn(T, Hkv, D, generator=g).bfloat16()
    if kind == "bits":      # every kind of bf16: NaN, infinities, subnormals, both zeros
        return torch.randint(-32768, 32768, (T, Hkv, D), generator=g, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    if kind == "ties":      # halfway between codes, normal and subnormal, the largest and what rounds to it
        t = torch.cat([(paged64.E4M3[1:] + paged64.E4M3[:-1]) / 2, paged64.E4M3, torch.tensor([463.0, 464.0, 465.0, 480.0])])
        t = torch.cat([t, -t])
        return t[torch.randint(0, len(t), (T, Hkv, D), generator=g)].bfloat16()
    e = torch.randint(-24, 16, (T, Hkv, 1), generator=g)
    return torch.randn(T, Hkv, D, generator=g).mul(torch.exp2(e.float())).bfloat16()


def same_codes(got, want):
    # the sign of a NaN is free
    got, want = got.cpu().view(torch.uint8), want.view(torch.uint8)
    nan = (want & 0x7F) == 0x7F
    return torch.equal((got & 0x7F) == 0x7F, nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn])
@pytest.mark.parametrize("T,Hkv,kind,kd,vd", [
    (1, 1, "normal", 1.0, 1.0), (33, 2, "normal", 0.37, 2.5), (200, 3, "bits", 1.0, 1.0), (64, 2, "ties", 1.0, 1.0),
    (64, 2, "ties", 0.75, 0.5), (257, 8, "range", 1.0, 3e-3), (5, 4, "bits", 1.7e30, 1e-30), (7, 1, "bits", 2.0 ** -130, 1.0)])
def test_write_is_the_formula(gda, T, Hkv, kind, kd, vd, dtype):
    slots_n = T + 9
    kp, vp = cache(slots_n, Hkv)
    k, v = rows(kind, T, Hkv, 1), rows(kind, T, Hkv, 2)
    if kind == "ties":
        k, v = (k.float() * kd).bfloat16(), (v.float() * vd).bfloat16()   # (exact: 3 and 5 significant bits)
    slots = torch.randperm(slots_n, generator=torch.Generator().manual_seed(3))[:T].to(torch.int32)
    # k and v as two parts of one projection row (a row of 2 Hkv D + 8 elements)
    proj = torch.zeros(T, 2 * Hkv * D + 8, dtype=torch.bfloat16)
    proj[:, :Hkv * D], proj[:, Hkv * D:2 * Hkv * D] = k.flatten(1), v.flatten(1)
    proj = proj.cuda()
    gk, gv = Guarded.copy_of(kp.cuda()), Guarded.copy_of(vp.cuda())
    gda.kv_write_e4m3(proj[:, :Hkv * D].unflatten(1, (Hkv, D)), proj[:, Hkv * D:2 * Hkv * D].unflatten(1, (Hkv, D)),
                      slots.cuda(), gk.t.view(dtype), gv.t.view(dtype), k_descale=kd, v_descale=vd)
    check_all(k_pool=gk, v_pool=gv)
    want_k, want_v = kp.clone(), vp.clone()
    want_k[slots.long()], want_v[slots.long()] = paged64.quantise8(k, kd), paged64.quantise8(v, vd)
    rest = torch.ones(slots_n, dtype=torch.bool)
    rest[slots.long()] = False
    for got, want in ((gk.t, want_k), (gv.t, want_v)):
        assert same_codes(got[slots.long().cuda()], want[slots.long()])
        assert torch.equal(got.cpu()[rest], want[rest])              # other slots untouched


def test_write_skips_slots_outside_the_pool(gda):
    kp, vp = cache(10, 2)
    k = rows("normal", 5, 2, 1)
    slots = torch.tensor([-1, 10, 3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    dk, dv = kp.cuda(), vp.cuda()
    gda.kv_write_e4m3(k.cuda(), k.cuda(), slots.cuda(), dk, dv)
    keep = [i for i in range(10) if i != 3]
    assert torch.equal(dk.cpu()[keep], kp[keep]) and torch.equal(dv.cpu()[keep], vp[keep])
    assert torch.equal(dk.cpu()[3], paged64.quantise8(k[2])) and torch.equal(dv.cpu()[3], paged64.quantise8(k[2]))


@pytest.mark.parametrize("N,Hkv,kd,vd", [(1, 2, 1.0, 1.0), (37, 1, 0.37, -2.0), (1000, 3, 1.0, 1e-3)])
def test_gather_reads_the_values(gda, N, Hkv, kd, vd):
    kp, vp = cache(50, Hkv, seed=N)                 # (NaN codes among them)
    idx = torch.randint(-3, 53, (N,), generator=torch.Generator().manual_seed(4)).to(torch.int32)   # some outside, some twice
    gk, gv = Guarded((N, Hkv, D), torch.bfloat16), Guarded((N, Hkv, D), torch.bfloat16)
    gda.kv_gather_e4m3(kp.cuda(), vp.cuda(), idx.cuda(), k_descale=kd, v_descale=vd, k_out=gk.t, v_out=gv.t)
    check_all(k=gk, v=gv)
    inside = (idx >= 0) & (idx < 50)
    for got, pool, d in ((gk.t, kp, kd), (gv.t, vp, vd)):
        # a code is exact in FP32; the descale is one FP32 rounding, then BF16
        x = paged64.values8(pool).float() * torch.tensor(d, dtype=torch.float32)
        want = torch.where(inside[:, None, None], x[idx.clamp(0, 49).long()], torch.zeros(())).bfloat16()
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


def test_all_codes_round_trip(gda):
    """Every code read back and written again is the same code (NaNs as NaNs, -0 as -0)."""
    kp = torch.arange(256, dtype=torch.uint8).view(1, 1, D).contiguous().cuda()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = gda.kv_gather_e4m3(kp, kp.flip(-1).contiguous(), zero)
    ko, vo = torch.zeros_like(kp), torch.zeros_like(kp)
    gda.kv_write_e4m3(k, v, zero, ko, vo)
    assert same_codes(ko, kp.cpu()) and same_codes(vo, kp.flip(-1).cpu())


def test_write_then_gather_in_a_graph(gda):
    k = rows("normal", 40, 2, 1).cuda()
    kp, vp = (t.cuda() for t in cache(64, 2))
    slots = torch.randperm(64)[:40].to(torch.int32).cuda()
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gda.kv_write_e4m3(k, k, slots, kp, vp, k_descale=0.25, v_descale=0.3)
            gda.kv_gather_e4m3(kp, vp, slots, k_descale=0.25, v_descale=0.3, k_out=ko, v_out=vo)
    k.mul_(3.0)
    g.replay()
    torch.cuda.synchronize()
    for got, d in ((ko, 0.25), (vo, 0.3)):
        # (both roundings of the value as the kernel makes them: FP32, then BF16)
        want = (paged64.values8(paged64.quantise8(k, d)).float() * torch.tensor(d)).bfloat16()
        assert torch.equal(got.cpu(), want)


def test_what_is_written_is_what_decode_reads(gda):
    """Rows written here, attended over by the 8-bit decode and by the BF16 decode on the rows read back: descales are
    powers of two, so that both caches stand for the same values."""
    B, L, hkv = 3, 150, 2
    k, v = rows("normal", B * L, hkv, 5).cuda(), rows("normal", B * L, hkv, 6).cuda()
    kp, vp = (torch.zeros(B * L, hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.randperm(B * L).to(torch.int32).cuda()
    gda.kv_write_e4m3(k, v, slots, kp, vp, k_descale=0.125, v_descale=0.0625)
    kb, vb = gda.kv_gather_e4m3(kp, vp, slots, k_descale=0.125, v_descale=0.0625)
    q, gate = rows("normal", B, 16, 7).cuda(), rows("normal", B, 16, 8).cuda()
    ptr = torch.tensor([0, L, 2 * L, 3 * L], dtype=torch.int32).cuda()
    a = gda.decode(q, gate, kp, vp, ptr, slots, k_descale=0.125, v_descale=0.0625)
    b = gda.decode(q, gate, kb, vb, ptr, torch.arange(B * L, dtype=torch.int32).cuda())
    # probabilities in FP16 there, BF16 here: 2^-8 + 2^-11 of what they weigh, three BF16 roundings of each result
    tol = (2.0 ** -8 + 2.0 ** -11 + 6.1 * 2.0 ** -8) * (vb.float().abs().max() * torch.sigmoid(gate.float()))
    assert bool(((a.float() - b.float()).abs() <= tol).all())
