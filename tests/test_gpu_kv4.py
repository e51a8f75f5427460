"""Writing the 4-bit KV cache and reading it back on the GPU.  Stored codes and scales follow
from the formula bit for bit (IEEE divisions, roundings to nearest even), and so do the
rows read back."""
import pytest
import torch

import plain64
from canary import Guarded, check_all

pytestmark = pytest.mark.gpu
D = 256


def cache(slots, Hkv, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)
    return r(slots, Hkv, D // 2), r(slots, Hkv, D // 2), r(slots, Hkv, 2, D // 16) & 0x7E


def rows(kind, T, Hkv, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "normal":
        return torch.randn(T, Hkv, D, generator=g).bfloat16()
    if kind == "bits":      # every kind of bf16: NaN, infinities, subnormals, both zeros
        return torch.randint(-32768, 32768, (T, Hkv, D), generator=g, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    if kind == "ties":      # quotients on the borders between codes, and maxima on those between scales
        v = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.25, -0.75, -5.0, -0.0, 0.125, 7.0, 6.375])
        return v[torch.randint(0, 16, (T, Hkv, D), generator=g)].bfloat16() * 2.0 ** float(seed % 5 - 2)
    e = torch.randint(-24, 16, (T, Hkv, 1), generator=g)   # from scales that round to 0 to saturated ones
    return torch.randn(T, Hkv, D, generator=g).mul(torch.exp2(e.float())).bfloat16()


@pytest.mark.parametrize("T,Hkv,kind,kd,vd", [
    (1, 1, "normal", 1.0, 1.0), (33, 2, "normal", 0.37, 2.5), (200, 3, "bits", 1.0, 1.0), (64, 2, "ties", 1.0, 0.5),
    (257, 8, "range", 1.0, 3e-3), (5, 4, "bits", 1.7e30, 1e-30)])
def test_write_is_the_formula(gda, T, Hkv, kind, kd, vd):
    slots_n = T + 9
    kp, vp, sc = cache(slots_n, Hkv)
    k, v = rows(kind, T, Hkv, 1), rows(kind, T, Hkv, 2)
    slots = torch.randperm(slots_n, generator=torch.Generator().manual_seed(3))[:T].to(torch.int32)
    # k and v as two parts of one projection row (a row of 2 Hkv D + 8 elements)
    proj = torch.zeros(T, 2 * Hkv * D + 8, dtype=torch.bfloat16)
    proj[:, :Hkv * D], proj[:, Hkv * D:2 * Hkv * D] = k.flatten(1), v.flatten(1)
    proj = proj.cuda()
    gk, gv, gs = Guarded.copy_of(kp.cuda()), Guarded.copy_of(vp.cuda()), Guarded.copy_of(sc.cuda())
    gda.kv_write_fp4(proj[:, :Hkv * D].unflatten(1, (Hkv, D)), proj[:, Hkv * D:2 * Hkv * D].unflatten(1, (Hkv, D)),
                     slots.cuda(), gk.t, gv.t, gs.t, k_descale=kd, v_descale=vd)
    check_all(k_pool=gk, v_pool=gv, scales=gs)
    want_k, want_v, want_s = kp.clone(), vp.clone(), sc.clone()
    want_k[slots.long()], want_s[slots.long(), :, 0] = plain64.quantise(k, kd)
    want_v[slots.long()], want_s[slots.long(), :, 1] = plain64.quantise(v, vd)
    assert torch.equal(gs.t.cpu(), want_s)
    assert torch.equal(gk.t.cpu(), want_k) and torch.equal(gv.t.cpu(), want_v)   # other slots untouched


def test_write_skips_slots_outside_the_pool(gda):
    kp, vp, sc = cache(10, 2)
    k = rows("normal", 4, 2, 1)
    slots = torch.tensor([-1, 10, 3, 2 ** 31 - 1], dtype=torch.int32)
    dk, dv, ds = kp.cuda(), vp.cuda(), sc.cuda()
    gda.kv_write_fp4(k.cuda(), k.cuda(), slots.cuda(), dk, dv, ds)
    keep = [i for i in range(10) if i != 3]
    assert torch.equal(dk.cpu()[keep], kp[keep]) and torch.equal(dv.cpu()[keep], vp[keep])
    assert torch.equal(ds.cpu()[keep], sc[keep])
    assert torch.equal(dk.cpu()[3], plain64.quantise(k[2])[0])


@pytest.mark.parametrize("N,Hkv,kd,vd", [(1, 2, 1.0, 1.0), (37, 1, 0.37, -2.0), (1000, 3, 1.0, 1e-3)])
def test_gather_reads_the_values(gda, N, Hkv, kd, vd):
    kp, vp, sc = cache(50, Hkv, seed=N)
    sc[7] = 0x7F                                    # NaN scales
    idx = torch.randint(-3, 53, (N,), generator=torch.Generator().manual_seed(4)).to(torch.int32)   # some outside, some twice
    gk, gv = Guarded((N, Hkv, D), torch.bfloat16), Guarded((N, Hkv, D), torch.bfloat16)
    gda.kv_gather_fp4(kp.cuda(), vp.cuda(), sc.cuda(), idx.cuda(), k_descale=kd, v_descale=vd, k_out=gk.t, v_out=gv.t)
    check_all(k=gk, v=gv)
    inside = (idx >= 0) & (idx < 50)
    for got, pool, i, d in ((gk.t, kp, 0, kd), (gv.t, vp, 1, vd)):
        # code * scale is exact; the descale is one FP32 rounding, then BF16
        x = plain64.values(pool, sc[:, :, i]).float() * torch.tensor(d, dtype=torch.float32)
        want = torch.where(inside[:, None, None], x[idx.clamp(0, 49).long()], torch.zeros(())).bfloat16()
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


def test_all_codes_and_scales(gda):
    """Every code under every scale byte through the read path."""
    kp = torch.arange(256, dtype=torch.uint8)[:, None, None].expand(256, 1, D // 2).contiguous()
    sc = torch.zeros(256, 1, 2, D // 16, dtype=torch.uint8)
    idx = torch.arange(256, dtype=torch.int32).cuda()
    for base in range(0, 256, 16):
        sc[:, 0, 0] = torch.arange(base, base + 16, dtype=torch.uint8)
        sc[:, 0, 1] = sc[:, 0, 0].flip(-1)
        k, v = gda.kv_gather_fp4(kp.cuda(), kp.cuda(), sc.cuda(), idx)
        for got, i in ((k, 0), (v, 1)):
            want = plain64.values(kp, sc[:, :, i]).bfloat16()
            assert torch.equal(got.cpu().nan_to_num(7e4), want.nan_to_num(7e4))


def test_write_then_gather_in_a_graph(gda):
    k = rows("normal", 40, 2, 1).cuda()
    kp, vp, sc = (t.cuda() for t in cache(64, 2))
    slots = torch.randperm(64)[:40].to(torch.int32).cuda()
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gda.kv_write_fp4(k, k, slots, kp, vp, sc)
            gda.kv_gather_fp4(kp, vp, sc, slots, k_out=ko, v_out=vo)
    k.mul_(3.0)
    g.replay()
    torch.cuda.synchronize()
    want = plain64.values(*plain64.quantise(k)).bfloat16()
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want)
