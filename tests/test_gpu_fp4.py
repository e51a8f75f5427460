"""Gated decode over a 4-bit KV cache on the GPU against float64 (plain64): the split path and
the one-kernel path, group sizes, windows, sinks, empty sequences, bad indices, captures."""
import math

import pytest
import torch

import plain64
from canary import Guarded, check_all

pytestmark = pytest.mark.gpu
D = 256
FP16 = 2.0 ** -11


def batch(lens, Hq=16, Hkv=2, seed=0, spare=7, kd=1.0, vd=1.0, k_std=1.0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    slots = n + spare
    k = (torch.randn(slots, Hkv, D, generator=g) * k_std * kd).bfloat16()
    v = (torch.randn(slots, Hkv, D, generator=g) * vd).bfloat16()
    kp, ks = plain64.quantise(k, kd)
    vp, vs = plain64.quantise(v, vd)
    idx = torch.randperm(slots, generator=g)[:n].to(torch.int32)
    ip = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    q = torch.randn(len(lens), Hq, D, generator=g).bfloat16()
    gate = (2 * torch.randn(len(lens), Hq, D, generator=g)).bfloat16()
    return dict(q=q, gate=gate, kp=kp, vp=vp, sc=torch.stack([ks, vs], 2), ip=ip, idx=idx, kd=kd, vd=vd, lens=lens,
                k=plain64.values(kp, ks, kd), v=plain64.values(vp, vs, vd))


def run(gda, b, **kw):
    go, gl = Guarded((*b["q"].shape,), torch.bfloat16), Guarded(b["q"].shape[:2], torch.float32)
    idx = b["idx"].cuda() if b["idx"].numel() else torch.zeros(1, dtype=torch.int32, device="cuda")
    gda.decode_ex(b["q"].cuda(), b["gate"].cuda() if kw.get("fuse_gate", True) else None, b["kp"].cuda(), b["vp"].cuda(),
                  b["ip"].cuda(), idx, out=go.t, lse=gl.t, scale=1 / 16, kv_scales=b["sc"].cuda(), k_descale=b["kd"],
                  v_descale=b["vd"], **kw)
    check_all(out=go, lse=gl)
    return go.t.cpu(), gl.t.cpu()


def want(b, gate=True, **kw):
    return plain64.decode(b["q"], b["gate"] if gate else None, b["k"], b["v"], b["ip"], b["idx"], 1 / 16, **kw)


CASES = [
    ([1], 16, 2), ([0], 16, 2), ([31, 32, 33, 0, 1, 64], 16, 2), ([512], 16, 2), ([300, 7, 1000], 8, 8), ([257], 3, 1),
    ([700, 65], 12, 4), ([129, 2048], 32, 2), ([95, 96, 97], 40, 2), ([5000], 16, 2), ([1] * 70 + [513], 16, 2),
]


@pytest.mark.parametrize("lens,Hq,Hkv", CASES)
@pytest.mark.parametrize("path", ["auto", "bound", "splits"])
def test_matches_float64(gda, lens, Hq, Hkv, path):
    b = batch(lens, Hq, Hkv, seed=len(lens) + Hq, kd=0.5 if Hq > 8 else 0.3, vd=1.5)
    kw = {"auto": {}, "bound": dict(max_len=max(1, max(lens)), total_len=sum(lens)), "splits": dict(num_splits=5)}[path]
    out, lse = run(gda, b, **kw)
    plain64.check(out, lse, want(b), FP16, max(lens), path)


@pytest.mark.parametrize("window,sinks,max_len", [(0, True, 0), (50, False, 0), (50, True, 0), (1, True, 0), (0, True, 700),
                                                  (100, True, 700), (5000, False, 0)])
def test_window_and_sinks(gda, window, sinks, max_len):
    b = batch([0, 1, 49, 50, 51, 700, 333], seed=5)
    s = torch.linspace(-3, 6, 16) if sinks else None
    out, lse = run(gda, b, window=window, sinks=s.cuda() if sinks else None, max_len=max_len)
    plain64.check(out, lse, want(b, window=window, sinks=s), FP16, 700)


def test_many_sequences_take_the_stream_schedule(gda):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 400, (224,), generator=g).tolist()
    b = batch(lens, seed=8)
    out, lse = run(gda, b)
    plain64.check(out, lse, want(b), FP16, 400)


@pytest.mark.parametrize("max_len", [0, 600])
def test_peaked_scores_and_ungated(gda, max_len):
    """Scores up to several hundred (one position takes nearly all the weight) and the ungated form."""
    b = batch([600, 77], seed=11, k_std=8.0)
    out, lse = run(gda, b, fuse_gate=False, max_len=max_len)
    plain64.check(out, lse, want(b, gate=False), FP16, 600)


def test_entry_points_agree(gda):
    b = batch([400, 3, 90], seed=12, kd=0.25, vd=4.0)
    d = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in b.items()}
    kw = dict(scale=1 / 16, k_descale=0.25, v_descale=4.0)
    o1 = gda.decode(d["q"], d["gate"], d["kp"], d["vp"], d["ip"], d["idx"], kv_scales=d["sc"], **kw)
    o2 = gda.decode_ex(d["q"], d["gate"], d["kp"], d["vp"], d["ip"], d["idx"], kv_scales=d["sc"].view(torch.float8_e4m3fn), **kw)
    o3 = gda.decode_ex(d["q"], None, d["kp"], d["vp"], d["ip"], d["idx"], kv_scales=d["sc"], fuse_gate=False, **kw)
    assert torch.equal(o1, o2) and torch.equal(gda.gate(o3, d["gate"]), o1)


@pytest.mark.parametrize("max_len", [0, 512])
def test_nan_rows(gda, max_len):
    """A NaN block in a named row reaches the query heads of its KV head and no others; NaN rows that
    no sequence names reach nothing."""
    b = batch([512, 100, 64], seed=13)
    ip, idx = b["ip"].tolist(), b["idx"]
    unused = torch.ones(b["kp"].shape[0], dtype=torch.bool)
    unused[idx.long()] = False
    b["sc"][unused] = 0x7F
    out, lse = run(gda, b, max_len=max_len)
    plain64.check(out, lse, want(b), FP16, 512)
    b["sc"][int(idx[ip[1] + 40]), 1, 0, 3] = 0x7F      # sequence 1, KV head 1, a K block
    b["sc"][int(idx[ip[2] + 63]), 0, 1, 15] = 0xFF     # sequence 2, KV head 0, the last V block
    out2, lse2 = run(gda, b, max_len=max_len)
    assert torch.isnan(out2[1, 8:].float()).all() and torch.isnan(lse2[1, 8:]).all()
    assert torch.isnan(out2[2, :8, 240:].float()).all()
    assert torch.equal(out2[0], out[0]) and torch.equal(out2[1, :8], out[1, :8])
    assert torch.equal(out2[2, 8:], out[2, 8:]) and torch.equal(out2[2, :8, :240], out[2, :8, :240])


def test_check_indices(gda):
    b = batch([100, 40], seed=14)
    b["idx"][17], b["idx"][120] = -5, b["kp"].shape[0]
    ws = torch.empty(gda.workspace_bytes(2, 16, 2, D), dtype=torch.uint8, device="cuda")
    gda.workspace_init(ws)
    out, lse = run(gda, b, check_indices=True, workspace=ws)
    assert gda.read_error(ws) == 1
    zero = b["kp"].shape[0] - 1                          # the bad rows read as zeros
    free = next(i for i in range(zero + 1) if i not in set(b["idx"].tolist()))
    b["k"][free], b["v"][free] = 0.0, 0.0
    b["idx"][17] = b["idx"][120] = free
    plain64.check(out, lse, want(b), FP16, 100)


def test_rows_beyond_two_gigabytes(gda):
    """Slots whose byte offsets pass 2^31 (codes) in a pool of 18 million rows."""
    slots, Hkv = 9_000_000, 2
    b = batch([150, 20], seed=15)
    far = torch.randperm(slots - 8_500_000, generator=torch.Generator().manual_seed(1))[:b["kp"].shape[0]] + 8_500_000
    kp = torch.zeros(slots, Hkv, D // 2, dtype=torch.uint8, device="cuda")
    vp, sc = torch.zeros_like(kp), torch.zeros(slots, Hkv, 2, D // 16, dtype=torch.uint8, device="cuda")
    kp[far.cuda()], vp[far.cuda()], sc[far.cuda()] = b["kp"].cuda(), b["vp"].cuda(), b["sc"].cuda()
    idx = far[b["idx"].long()].to(torch.int32).cuda()
    for kw in ({}, dict(max_len=150)):
        lse = torch.empty(2, 16, device="cuda")
        out = gda.decode_ex(b["q"].cuda(), b["gate"].cuda(), kp, vp, b["ip"].cuda(), idx, scale=1 / 16, lse=lse, kv_scales=sc, **kw)
        plain64.check(out.cpu(), lse.cpu(), want(b), FP16, 150)


def test_repeatable_and_on_two_streams(gda):
    """The same bits every time, and two calls at once on their own workspaces."""
    a, b = batch([3000, 10, 900], seed=16), batch([50] * 40, seed=17)
    refs = [run(gda, x)[0] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    dev = [{k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in y.items()} for y in (a, b)]
    ws = [torch.zeros(gda.workspace_bytes(x["q"].shape[0], 16, 2, D), dtype=torch.uint8, device="cuda") for x in dev]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                x = dev[i]
                outs[i].append(gda.decode_ex(x["q"], x["gate"], x["kp"], x["vp"], x["ip"], x["idx"], workspace=ws[i], scale=1 / 16,
                                             kv_scales=x["sc"]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o.cpu(), refs[i]) for o in outs[i])


def test_captured_and_replayed(gda):
    """A captured call follows the cache and the lengths as they are at replay."""
    b = batch([600, 40], seed=18)
    d = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in b.items()}
    ws = torch.zeros(gda.workspace_bytes(2, 16, 2, D), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(d["q"]), torch.empty(2, 16, device="cuda")
    call = lambda: gda.decode_ex(d["q"], d["gate"], d["kp"], d["vp"], d["ip"], d["idx"], out=out, lse=lse, workspace=ws,
                                 scale=1 / 16, kv_scales=d["sc"])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    b["ip"] = torch.tensor([0, 33, 640], dtype=torch.int32)
    d["ip"].copy_(b["ip"])
    b["k"], b["v"] = b["v"], b["k"]
    t = d["kp"].clone()
    d["kp"].copy_(d["vp"])
    d["vp"].copy_(t)
    d["sc"].copy_(d["sc"].flip(2))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    plain64.check(out.cpu(), lse.cpu(), want(b), FP16, 640)


def test_a_decode_step_from_projection_to_output(gda):
    """qk_norm_mrope_kv_write into the cache, then decode over it, against the same two steps in float64."""
    B, Hq, Hkv = 5, 16, 2
    b = batch([1, 40, 300, 77, 512], seed=19)
    g = torch.Generator().manual_seed(20)
    qgkv = torch.randn(B, (2 * Hq + 2 * Hkv) * D, generator=g).bfloat16()
    pos = torch.randint(0, 5000, (3, B), generator=g, dtype=torch.int32)
    inv = 1e4 ** (-torch.arange(0, 64, 2) / 64)
    axis = gda.mrope_pair_axis([12, 10, 10], interleaved=True)
    slots = torch.stack([b["idx"][i - 1] for i in b["ip"][1:].tolist()])
    d = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in b.items()}
    gate = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    q, k = gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), axis, Hq, Hkv, gate_out=gate, slots=slots.cuda(),
                                      k_pool=d["kp"], v_pool=d["vp"], kv_scales=d["sc"])
    out = gda.decode(q, gate, d["kp"], d["vp"], d["ip"], d["idx"], scale=1 / 16, kv_scales=d["sc"])
    x = qgkv.view(B, 2 * Hq + 2 * Hkv, D)
    assert torch.equal(gate.cpu(), x[:, Hq:2 * Hq])
    # the cache's new rows are k_out and v quantised; the others are as they were
    kc, ks = plain64.quantise(k.cpu())
    vc, vs = plain64.quantise(x[:, 2 * Hq + Hkv:])
    b["kp"][slots.long()], b["vp"][slots.long()] = kc, vc
    b["sc"][slots.long()] = torch.stack([ks, vs], 2)
    assert torch.equal(d["kp"].cpu(), b["kp"]) and torch.equal(d["vp"].cpu(), b["vp"]) and torch.equal(d["sc"].cpu(), b["sc"])
    b["k"], b["v"] = plain64.values(b["kp"], b["sc"][:, :, 0]), plain64.values(b["vp"], b["sc"][:, :, 1])
    b["q"], b["gate"] = q.cpu(), gate.cpu()
    plain64.check(out.cpu(), None, want(b), FP16, 512)


@pytest.mark.parametrize("Hq,max_len", [(16, 0), (16, 512), (32, 0), (40, 0)])
@pytest.mark.parametrize("value", [math.inf, math.nan, 1e30])
def test_one_query_head_with_extreme_values(gda, Hq, max_len, value):
    """An infinite, NaN or huge element of one query head leaves every other head as it was."""
    b = batch([300, 65], Hq, 2, seed=19)
    out, lse = run(gda, b, max_len=max_len)
    head = Hq // 2 - 3
    b["q"][1, head, 100] = value
    out2, lse2 = run(gda, b, max_len=max_len)
    others = [h for h in range(Hq) if h != head]
    assert torch.equal(out2[0], out[0]) and torch.equal(out2[1, others], out[1, others])
    assert torch.equal(lse2[1, others], lse[1, others])
    if math.isnan(value):
        assert torch.isnan(out2[1, head].float()).all() and torch.isnan(lse2[1, head])


@pytest.mark.parametrize("max_len,total_len", [(10, 0), (10, 765), (1, 1), (700, 3), (5000, 10 ** 6)])
def test_wrong_bounds_change_only_the_speed(gda, max_len, total_len):
    b = batch([700, 65], seed=20)
    out, lse = run(gda, b, max_len=max_len, total_len=total_len)
    plain64.check(out, lse, want(b), FP16, 700)
