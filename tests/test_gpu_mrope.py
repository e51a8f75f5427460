"""The step before attention with positions on several axes, on the GPU against float64."""
import pytest
import torch

import plain64
from canary import Guarded, check_all

pytestmark = pytest.mark.gpu
D = 256


def make(T, Hq, Hkv, rope, axes, seed, far=5000, extra=0):
    g = torch.Generator().manual_seed(seed)
    width = (2 * Hq + 2 * Hkv) * D
    qgkv = torch.randn(T, width + extra, generator=g).bfloat16()[:, :width]
    pos = torch.randint(0, far, (axes, T), generator=g).to(torch.int32)
    inv = (1e6 ** (-torch.arange(0, max(rope, 1), 2, dtype=torch.float64) / max(rope, 1))).float()[:rope // 2]
    axis = [int(x) for x in torch.randint(0, axes, (rope // 2,), generator=g)]
    wq, wk = (torch.rand(D, generator=g) + 0.5).bfloat16(), (torch.rand(D, generator=g) + 0.5).bfloat16()
    return qgkv, pos, inv, axis, wq, wk


def reference(qgkv, pos, inv, axis, Hq, Hkv, wq, wk):
    x = qgkv.reshape(qgkv.shape[0], 2 * Hq + 2 * Hkv, D)
    angle = pos.double()[axis].t() * inv.double() if axis else None
    return (plain64.norm_rope(x[:, :Hq], wq, 1e-6, angle), x[:, Hq:2 * Hq],
            plain64.norm_rope(x[:, 2 * Hq:2 * Hq + Hkv], wk, 1e-6, angle), x[:, 2 * Hq + Hkv:])


def near(got, want, rope):
    """BF16's half step of the value, and 2^-20 of the two rotated inputs for the FP32 steps before it: the norm's
    256-term sum, the angle's cos and sin (2^-23 each) and the rotation."""
    got = got.cpu().double()
    big = want.abs()
    if rope:
        a, b = want[..., :rope // 2], want[..., rope // 2:rope]
        n = torch.sqrt(a * a + b * b)
        big = torch.cat([n, n, want[..., rope:].abs()], -1)
    bad = (got - want).abs() > 2.0 ** -8 * want.abs() + 2.0 ** -20 * big + 1e-38
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("T,Hq,Hkv,rope,axes,norm,pool", [
    (1, 16, 2, 64, 3, True, "bf16"), (7, 16, 2, 0, 1, True, "none"), (50, 4, 4, 256, 4, False, "fp4"),
    (224, 16, 2, 64, 3, True, "fp4"), (33, 3, 1, 16, 1, True, "bf16"), (3000, 5, 1, 128, 2, True, "none"),
    (1300, 1, 1, 64, 3, True, "bf16")])
def test_matches_float64(gda, T, Hq, Hkv, rope, axes, norm, pool):
    qgkv, pos, inv, axis, wq, wk = make(T, Hq, Hkv, rope, axes, seed=T + rope, extra=24)
    if not norm:
        wq = wk = None
    slots_n = T + 11
    slots = torch.randperm(slots_n, generator=torch.Generator().manual_seed(1))[:T].to(torch.int32)
    gq, gk, gg = (Guarded((T, h, D), torch.bfloat16) for h in (Hq, Hkv, Hq))
    kw, pools = {}, []
    if pool == "bf16":
        pools = [Guarded((slots_n, Hkv, D), torch.bfloat16, fill=3.0) for _ in range(2)]
    elif pool == "fp4":
        pools = [Guarded((slots_n, Hkv, D // 2), torch.uint8, fill=9) for _ in range(2)]
        pools.append(Guarded((slots_n, Hkv, 2, D // 16), torch.uint8, fill=5))
        kw = dict(kv_scales=pools[2].t, k_descale=0.5, v_descale=0.25)
    if pools:
        kw.update(slots=slots.cuda(), k_pool=pools[0].t, v_pool=pools[1].t)
    c = lambda t: None if t is None else t.cuda()
    padded = torch.zeros(T, qgkv.shape[1] + 24, dtype=torch.bfloat16, device="cuda")   # rows further apart
    padded[:, :qgkv.shape[1]] = qgkv.cuda()
    q, k = gda.qk_norm_mrope_kv_write(padded[:, :qgkv.shape[1]], pos.cuda(), inv.cuda(), axis, Hq, Hkv, w_q_norm=c(wq),
                                      w_k_norm=c(wk), q_out=gq.t, k_out=gk.t, gate_out=gg.t, **kw)
    check_all(q=gq, k=gk, gate=gg, **{"pool%d" % i: p for i, p in enumerate(pools)})
    rq, rg, rk, rv = reference(qgkv, pos, inv, axis, Hq, Hkv, wq, wk)
    near(q, rq, rope)
    near(k, rk, rope)
    assert torch.equal(gg.t.cpu(), rg)
    s = slots.long()
    rest = torch.ones(slots_n, dtype=torch.bool)
    rest[s] = False
    if pool == "bf16":
        kp, vp = pools[0].t.cpu(), pools[1].t.cpu()
        assert torch.equal(kp[s], k.cpu()) and torch.equal(vp[s], rv)
        assert (kp[rest] == 3.0).all() and (vp[rest] == 3.0).all()
    elif pool == "fp4":
        kp, vp, sc = (p.t.cpu() for p in pools)
        kc, ks = plain64.quantise(k, 0.5)
        vc, vs = plain64.quantise(rv, 0.25)
        assert torch.equal(kp[s], kc) and torch.equal(vp[s], vc) and torch.equal(sc[s], torch.stack([ks, vs], 2))
        assert (kp[rest] == 9).all() and (vp[rest] == 9).all() and (sc[rest] == 5).all()


def test_far_and_negative_positions(gda):
    """The angle keeps its accuracy over all of int32."""
    qgkv, _, inv, axis, wq, wk = make(8, 2, 1, 256, 2, seed=1)
    pos = torch.tensor([[0, -1, 1000003, -(2 ** 31), 2 ** 31 - 1, 7, 123456789, -99999],
                        [5, 2 ** 30, -1, 0, 1, 2 ** 31 - 1, -(2 ** 31), 3]], dtype=torch.int32)
    q, k = gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), axis, 2, 1)
    rq, _, rk, _ = reference(qgkv, pos, inv, axis, 2, 1, None, None)
    near(q, rq, 256)
    near(k, rk, 256)


def test_one_axis_is_the_plain_rotation(gda):
    """With one axis and no far positions: the same as gda.qk_norm_rope_kv_write within its BF16 tables."""
    qgkv, pos, inv, axis, wq, wk = make(20, 4, 2, 64, 1, seed=2)
    q, k = gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), axis, 4, 2, w_q_norm=wq.cuda(), w_k_norm=wk.cuda())
    ang = pos[0].double()[:, None] * inv.double()
    tab = lambda f: torch.cat([f(ang), f(ang)], 1).bfloat16().cuda()
    kp, vp = (torch.zeros(20, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q2, _ = gda.qk_norm_rope_kv_write(qgkv.cuda(), torch.arange(20, dtype=torch.int32).cuda(), kp, vp, 4, w_q_norm=wq.cuda(),
                                      w_k_norm=wk.cuda(), cos=tab(torch.cos), sin=tab(torch.sin), rope_dim=64)
    # the tables' cos and sin are rounded to BF16: half a step (2^-8) of each product, and both results' own
    lim = lambda x: 2 * 2.0 ** -8 * torch.cat([x[..., :32].abs() + x[..., 32:64].abs()] * 2 + [x[..., 64:].abs()], -1) * 1.5
    assert ((q.double() - q2.double()).abs() <= lim(q2.double())).all()
    assert ((k.double() - kp.double()).abs() <= lim(kp.double())).all()


def test_slots_outside_the_pool(gda):
    qgkv, pos, inv, axis, _, _ = make(4, 2, 2, 64, 1, seed=3)
    slots = torch.tensor([-1, 6, 2, -(2 ** 31)], dtype=torch.int32)
    kp, vp = (torch.full((6, 2, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _, k = gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), axis, 2, 2, slots=slots.cuda(), k_pool=kp, v_pool=vp)
    rest = [0, 1, 3, 4, 5]
    assert (kp[rest] == 3.0).all() and (vp[rest] == 3.0).all() and torch.equal(kp[2], k[2])


def test_captured(gda):
    qgkv, pos, inv, axis, _, _ = make(9, 2, 2, 64, 3, seed=4)
    x, p, f = qgkv.cuda(), pos.cuda(), inv.cuda()
    q, k = torch.empty(9, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(9, 2, D, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gda.qk_norm_mrope_kv_write(x, p, f, axis, 2, 2, q_out=q, k_out=k)
    p.add_(17)
    g.replay()
    torch.cuda.synchronize()
    rq, _, rk, _ = reference(qgkv, pos + 17, inv, axis, 2, 2, None, None)
    near(q, rq, 64)
    near(k, rk, 64)


@pytest.mark.parametrize("T,Hq,Hkv,pool", [(4864, 2, 1, "none"), (4865, 1, 1, "bf16"), (7290, 2, 1, "fp4"), (14599, 1, 1, "none")])
def test_more_tokens_than_warps(gda, T, Hq, Hkv, pool):
    """Several passes of the grid; in the last one the warps share the tokens that are left."""
    test_matches_float64(gda, T, Hq, Hkv, 64, 3, True, pool)


@pytest.mark.parametrize("side", ["q", "k"])
def test_one_norm_and_more_kv_heads_than_query_heads(gda, side):
    T, Hq, Hkv = 37, 2, 5
    qgkv, pos, inv, axis, wq, wk = make(T, Hq, Hkv, 32, 2, seed=6)
    wq, wk = (wq, None) if side == "q" else (None, wk)
    c = lambda t: None if t is None else t.cuda()
    gate = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    q, k = gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), axis, Hq, Hkv, w_q_norm=c(wq), w_k_norm=c(wk),
                                      gate_out=gate)
    rq, rg, rk, _ = reference(qgkv, pos, inv, axis, Hq, Hkv, wq, wk)
    near(q, rq, 32)
    near(k, rk, 32)
    assert torch.equal(gate.cpu(), rg)


def test_many_axes(gda):
    """Every pair on an axis of its own, the last of 128 axes among them."""
    T, Hq, Hkv = 9, 1, 1
    qgkv, _, _, _, wq, wk = make(T, Hq, Hkv, 256, 2, seed=8)
    g = torch.Generator().manual_seed(9)
    pos = torch.randint(-1000, 100000, (128, T), generator=g, dtype=torch.int32)
    inv = (1e4 ** (-torch.arange(0, 256, 2) / 256)).float()
    axis = list(range(127, -1, -1))
    q, k = gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), axis, Hq, Hkv, w_q_norm=wq.cuda(), w_k_norm=wk.cuda())
    rq, _, rk, _ = reference(qgkv, pos, inv, axis, Hq, Hkv, wq, wk)
    near(q, rq, 256)
    near(k, rk, 256)
