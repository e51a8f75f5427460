"""Attention of new tokens over a paged cache against float64 (the bounds are derived in plain64):
every cache type, head layout and chunk shape, windows with visible first tokens, sinks, rows that see
nothing, strides, streams, graphs and what must stay untouched."""
import math

import pytest
import torch

import paged64
import plain64
from canary import Guarded

pytestmark = pytest.mark.gpu
D = 256
# rounding of a probability: BF16 for a BF16 cache, FP16 for codes
P_STEP = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11, "fp4": 2.0 ** -11}


def cum(n):
    return torch.tensor([0] + list(torch.tensor(n, dtype=torch.int64).cumsum(0)), dtype=torch.int32)


class Batch:
    """Inputs of one call on the GPU, and the rows that its cache stands for in float64."""

    def __init__(self, lens, hq=16, hkv=2, kv="bf16", seed=0, spare=37, kd=0.5, vd=0.25, gate=True, sinks=False):
        g = torch.Generator().manual_seed(seed)
        nq, nk = [n for n, _ in lens], [n for _, n in lens]
        self.hq, self.hkv, self.kv = hq, hkv, kv
        Tq, Tk = sum(nq), sum(nk)
        slots = Tk + spare
        self.cu, self.indptr = cum(nq).cuda(), cum(nk).cuda()
        self.indices = torch.randperm(slots, generator=g)[:Tk].to(torch.int32).cuda()
        rows = torch.randn(Tq, 2, hq, D, generator=g).bfloat16()
        rows[:, 1] *= 2
        rows = rows.cuda()
        self.q, self.gate = rows[:, 0], (rows[:, 1] if gate else None)
        k, v = (torch.randn(slots, hkv, D, generator=g).bfloat16() for _ in range(2))
        self.kw = {}
        if kv == "bf16":
            self.k_pool, self.v_pool = k.cuda(), v.cuda()
            self.k64, self.v64 = k.double().cuda(), v.double().cuda()
        elif kv == "e4m3":
            ck, cv = paged64.quantise8(k, kd), paged64.quantise8(v, vd)
            self.k_pool, self.v_pool = ck.cuda().view(torch.float8_e4m3fn), cv.cuda().view(torch.float8_e4m3fn)
            self.k64, self.v64 = paged64.values8(ck, kd).cuda(), paged64.values8(cv, vd).cuda()
            self.kw = dict(k_descale=kd, v_descale=vd)
        else:
            (ck, sk), (cv, sv) = plain64.quantise(k, kd), plain64.quantise(v, vd)
            self.k_pool, self.v_pool = ck.cuda(), cv.cuda()
            self.kw = dict(kv_scales=torch.stack([sk, sv], 2).contiguous().cuda(), k_descale=kd, v_descale=vd)
            self.k64, self.v64 = plain64.values(ck, sk, kd).cuda(), plain64.values(cv, sv, vd).cuda()
        self.sinks = (torch.randn(hq, generator=g) * 2).cuda() if sinks else None
        self.longest = max(nk) if nk else 0

    def call(self, gda, window=0, keep_first=0, scale=1.0 / 16.0, lse=True, **kw):
        out = kw.pop("out", None)
        lse_t = torch.empty(self.hq, self.q.shape[0], device="cuda") if lse else None
        o = gda.prefill_paged(self.q, self.gate, self.k_pool, self.v_pool, self.cu, self.indptr, self.indices, out=out,
                              lse=lse_t, scale=scale, window=window, keep_first=keep_first, sinks=self.sinks,
                              **{**self.kw, **kw})
        return o, lse_t

    def want(self, window=0, keep_first=0, scale=1.0 / 16.0, fill=math.nan):
        return paged64.paged(self.q, self.gate, self.k64, self.v64, self.cu, self.indptr, self.indices, scale, window,
                             keep_first, self.sinks, fill)

    def check(self, gda, window=0, keep_first=0, scale=1.0 / 16.0, what="", **kw):
        o, lse = self.call(gda, window, keep_first, scale, **kw)
        torch.cuda.synchronize()
        assert gda.prefill_read_error() == 0
        plain64.check(o, lse.t(), self.want(window, keep_first, scale), P_STEP[self.kv], self.longest, what)
        return o, lse


KV = ["bf16", "e4m3", "fp4"]
HEADS = [(16, 2), (8, 8), (12, 4), (32, 2), (5, 1), (24, 1)]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("lens", [
    [(1, 1)], [(1, 128)], [(1, 129)], [(2, 2)], [(17, 17)], [(5, 300), (1, 77), (1, 1)], [(128, 128)], [(130, 515)],
    [(1, 4000)], [(300, 2000), (3, 2500)], [(0, 0), (1, 5), (0, 70), (7, 7), (0, 0)]], ids=str)
def test_lengths(gda, kv, lens):
    Batch(lens, kv=kv, seed=len(lens)).check(gda)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_heads(gda, kv, heads):
    Batch([(3, 200), (40, 700), (1, 1300)], *heads, kv=kv, seed=3).check(gda)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window, first", [(1, 0), (1, 1), (64, 4), (127, 0), (128, 130), (129, 1), (500, 16), (3000, 5)])
def test_windows(gda, kv, window, first):
    Batch([(3, 200), (150, 900), (1, 2300), (1, 1), (20, 20)], kv=kv, seed=5).check(gda, window, first)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window, first", [(0, 0), (70, 3)])
def test_sinks(gda, kv, window, first):
    b = Batch([(5, 5), (90, 333), (1, 1000), (4, 0), (9, 3)], kv=kv, sinks=True, seed=6)
    b.check(gda, window, first)
    b.sinks += torch.where(torch.arange(16, device="cuda") % 3 == 0, 90.0, -90.0)   # far above and far below the scores
    b.check(gda, window, first)
    b.sinks[::2] = -math.inf                                                        # no sink
    o, lse = b.check(gda, window, first)
    # a sink that is no number, or infinite: its head alone
    b.sinks[5], b.sinks[6] = math.nan, math.inf
    o2, lse2 = b.call(gda, window, first)
    rest = [h for h in range(16) if h not in (5, 6)]
    seen = b.want(window, first).sabs > 0                                           # rows with keys
    assert bool(o2[:, 5][seen[:, 5]].isnan().all()) and bool((o2[:, 6] == 0).all())
    assert torch.equal(o[:, rest], o2[:, rest]) and torch.equal(lse[rest], lse2[rest])


@pytest.mark.parametrize("kv", KV)
def test_rows_that_see_nothing(gda, kv):
    """More tokens than positions: the first rows have no key; a sequence without positions has none at all."""
    b = Batch([(9, 3), (140, 20), (3, 0), (1, 0), (20, 19)], kv=kv, seed=7)
    o, lse = b.check(gda)
    assert bool((o[:6] == 0).all()) and bool((lse[:, :6] == -math.inf).all())
    assert bool((o[9:9 + 120] == 0).all()) and bool((o[149:153] == 0).all())
    b.check(gda, window=2, keep_first=1)


@pytest.mark.parametrize("kv", KV)
def test_no_positions_and_no_tokens(gda, kv):
    b = Batch([(3, 0), (2, 0)], kv=kv, seed=8)
    o, lse = b.call(gda)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    b = Batch([(0, 5), (0, 2)], kv=kv, seed=8)
    o, lse = b.call(gda)
    assert o.shape == (0, 16, D)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("scale", [1.0, 1e-3])
def test_scales_and_no_gate(gda, kv, scale):
    b = Batch([(70, 700), (2, 3000)], kv=kv, gate=False, seed=9)
    o, lse = b.check(gda, scale=scale)
    # without lse: the same outputs
    o2, _ = b.call(gda, scale=scale, lse=False)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("kv", ["e4m3", "fp4"])
def test_queries_of_any_size(gda, kv):
    """Query rows from 2^-120 to 2^100 beside ordinary ones over a cache of codes."""
    b = Batch([(40, 300)], kv=kv, seed=10)
    e = torch.randint(-120, 100, (40, 16, 1), generator=torch.Generator().manual_seed(1)).cuda()
    # (small scores: the bound on them is relative to sabs, and far above 1 a score's own rounding moves a probability)
    b.q = (b.q.float() * torch.exp2(torch.minimum(e, torch.full_like(e, 2)).float())).bfloat16()
    b.check(gda)
    b.q[3:5] = 0
    b.check(gda)
    # a huge element makes its head's softmax one-hot; other heads and tokens keep their bits
    o, _ = b.call(gda)
    b.q[7, 4, 100] = 3e38
    o2, _ = b.call(gda)
    b.q[7, 4, 100] = math.inf
    o3, _ = b.call(gda)
    rest = torch.ones(40, 16, dtype=torch.bool, device="cuda")
    rest[7, 4] = False
    assert bool(o2.isfinite().all()) and torch.equal(o[rest], o2[rest]) and torch.equal(o[rest], o3[rest])


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window, first", [(0, 0), (200, 4)])
def test_bytes_around_the_outputs(gda, kv, window, first):
    """Rows of no sequence, and everything around the outputs and the workspace, stay as they are."""
    b = Batch([(3, 400), (200, 1000), (0, 9), (30, 30)], kv=kv, seed=11)
    Tq = b.q.shape[0]
    lead, tail = 5, 7
    big = torch.full((lead + Tq + tail, 2, 16, D), math.nan, dtype=torch.bfloat16, device="cuda")
    big[lead:lead + Tq, 0], big[lead:lead + Tq, 1] = b.q, b.gate
    b.q, b.gate = big[:, 0], big[:, 1]
    b.cu = b.cu + lead
    ws = Guarded((gda.prefill_paged_workspace_bytes(Tq, 4, 16, 2, D),), torch.uint8)
    out = Guarded(b.q.shape, torch.bfloat16, fill=7.0)
    lse = Guarded((16, lead + Tq + tail), torch.float32, fill=7.0)
    gda.prefill_paged(b.q, b.gate, b.k_pool, b.v_pool, b.cu, b.indptr, b.indices, out=out.t, lse=lse.t, scale=1 / 16,
                      window=window, keep_first=first, workspace=ws.t, **b.kw)
    for g in (ws, out, lse):
        g.check()
    a = b.want(window, first, fill=7.0)
    live = slice(lead, lead + Tq)
    for t in (out.t, lse.t.t()):
        assert bool((t[:lead] == 7.0).all()) and bool((t[lead + Tq:] == 7.0).all())
    a.out, a.pv, a.lse, a.sabs = a.out[live], a.pv[live], a.lse[live], a.sabs[live]
    plain64.check(out.t[live], lse.t.t()[live], a, P_STEP[kv], b.longest)


@pytest.mark.parametrize("kv", KV)
def test_rows_that_no_query_sees_may_hold_anything(gda, kv):
    """NaN rows behind each sequence's positions, in slots that nobody names, and in positions that have left the
    window of every token in the batch: the outputs are those of clean pools."""
    lens, window, first = [(3, 700), (1, 400), (20, 500)], 100, 4
    b = Batch(lens, kv=kv, seed=12)
    want, _ = b.call(gda, window, first)
    ip, named = b.indptr.tolist(), torch.zeros(b.k_pool.shape[0], dtype=torch.bool, device="cuda")
    for i, (n, L) in enumerate(lens):
        slot = b.indices[ip[i]:ip[i + 1]].long()
        named[slot[L - n - window + 1:]] = True
        named[slot[:first]] = True
    for name in ("k_pool", "v_pool"):
        raw = getattr(b, name).clone()
        raw.view(torch.uint8)[~named] = 0x7F if kv != "bf16" else 0xFF
        setattr(b, name, raw)
    if kv == "fp4":
        b.kw["kv_scales"] = b.kw["kv_scales"].clone()
        b.kw["kv_scales"][~named] = 0x7F
    got, _ = b.call(gda, window, first)
    assert torch.equal(got, want)


@pytest.mark.parametrize("kv", KV)
def test_slots_outside_the_pools(gda, kv):
    """Read as zeros and reported; a slot that no query sees is not looked at."""
    b = Batch([(4, 300), (1, 200)], kv=kv, seed=13)
    b.indices[10], b.indices[299], b.indices[420] = -1, b.k_pool.shape[0], 2 ** 31 - 1
    o, lse = b.call(gda)
    torch.cuda.synchronize()
    assert gda.prefill_read_error() == gda.DEVERR_INDEX
    assert gda.prefill_read_error() == 0
    plain64.check(o, lse.t(), b.want(), P_STEP[kv], b.longest)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.call(gda, error_word=word)
    assert int(word.item()) == gda.DEVERR_INDEX and gda.prefill_read_error() == 0
    b = Batch([(4, 300)], kv=kv, seed=13)
    b.indices[10] = -1
    b.check(gda, window=100)                       # (asserts that the error word stays 0)


@pytest.mark.parametrize("kv", KV)
def test_shared_and_repeated_slots(gda, kv):
    """Sequences with a common prefix, and one slot named many times."""
    b = Batch([(3, 400), (5, 400), (1, 300)], kv=kv, seed=14)
    b.indices[400:800 - 5] = b.indices[:395]
    b.indices[800:1100] = b.indices[800]
    b.check(gda)


@pytest.mark.parametrize("kv", KV)
def test_single_tokens_are_a_decode_step(gda, kv):
    """Against the decode kernels on the same cache: both are within the derived bounds of float64."""
    lens = [(1, L) for L in (1, 700, 128, 4000, 33)]
    b = Batch(lens, kv=kv, sinks=True, seed=15)
    o, lse = b.check(gda, window=500)
    d = gda.decode_ex(b.q.contiguous(), b.gate.contiguous(), b.k_pool, b.v_pool, b.indptr, b.indices, scale=1 / 16,
                      window=500, sinks=b.sinks, **b.kw)
    a = b.want(window=500)
    assert bool(((o.double() - d.double()).abs() <= 2 * plain64.bound_out(a, 2.0 ** -8, b.longest)).all())


def test_a_chunk_is_its_tokens_one_by_one(gda):
    """A prompt in one call, in chunks and token by token gives the same results within twice the bounds."""
    b = Batch([(150, 150)], seed=16)
    whole, _ = b.check(gda)
    a = b.want()
    for step in (1, 64):
        for i0 in range(0, 150, step):
            n = min(step, 150 - i0)
            cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            ip = torch.tensor([0, i0 + n], dtype=torch.int32, device="cuda")
            o = gda.prefill_paged(b.q[i0:i0 + n], b.gate[i0:i0 + n], b.k_pool, b.v_pool, cu, ip, b.indices, scale=1 / 16)
            tol = 2 * plain64.bound_out(a, 2.0 ** -8, 150)[i0:i0 + n]
            assert bool(((o.double() - whole[i0:i0 + n].double()).abs() <= tol).all())


@pytest.mark.parametrize("kv", KV)
def test_the_same_call_gives_the_same_bits(gda, kv):
    b = Batch([(5, 3000), (70, 2500), (1, 6000), (300, 300)], kv=kv, seed=17)
    o, lse = b.call(gda)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(12):
        cold.fill_(i)
        o2, lse2 = b.call(gda)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", KV)
def test_graph_follows_the_lengths(gda, kv):
    """Captured once, replayed with other lengths, slots and rows; two graphs share a workspace in turn."""
    b = Batch([(6, 900), (40, 333), (0, 0)], kv=kv, seed=18)
    ws = torch.empty(gda.prefill_paged_workspace_bytes(46, 3, 16, 2, D), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros(46, 16, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(16, 46, device="cuda")
    call = lambda w: gda.prefill_paged(b.q, b.gate, b.k_pool, b.v_pool, b.cu, b.indptr, b.indices, out=out, lse=lse,
                                       scale=1 / 16, window=w, keep_first=2, workspace=ws, **b.kw)
    call(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for w in (0, 100):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(w)
        graphs.append((w, g))
    for cu, ip in (([0, 6, 46, 46], [0, 900, 1233, 1233]), ([0, 1, 2, 46], [0, 1, 500, 1233]), ([0, 0, 46, 46], [0, 0, 1233, 1233])):
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        b.indptr.copy_(torch.tensor(ip, dtype=torch.int32))
        b.indices.copy_(b.indices[torch.randperm(1233, generator=torch.Generator().manual_seed(len(cu)))])
        for w, g in graphs:
            g.replay()
            torch.cuda.synchronize()
            plain64.check(out, lse.t(), b.want(w, 2), P_STEP[kv], 1233)
    assert gda.prefill_read_error() == 0


def test_streams(gda):
    """Two streams at once with their own workspaces; a side stream whose outputs belong to it."""
    bs = [Batch([(5, 2000), (64, 700)], seed=19), Batch([(1, 300)] * 20, kv="e4m3", seed=20)]
    refs = [b.call(gda, lse=False)[0] for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (s, b) in enumerate(zip(streams, bs)):
            if _ % 2:
                with torch.cuda.stream(s):
                    outs[i].append(b.call(gda, lse=False)[0])
            else:
                outs[i].append(b.call(gda, lse=False, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, refs[i]) for i in range(2) for o in outs[i])


def test_wait_limit_gives_a_typed_timeout(gda):
    b = Batch([(30, 2000), (1, 500), (0, 3), (200, 700)], seed=21)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kv in KV:
        b = Batch([(30, 2000), (1, 500), (0, 3), (200, 700)], kv=kv, seed=21)
        want, _ = b.call(gda, error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        try:
            gda.debug_wait_limit(200)           # SM cycles: below the latency of a first load
            b.call(gda, error_word=err)
            torch.cuda.synchronize()            # the call returns
        finally:
            gda.debug_wait_limit(0)
        assert int(err.item()) & gda.DEVERR_TIMEOUT
        err.zero_()
        got, _ = b.call(gda, error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.equal(got, want)


def test_every_gate_code(gda):
    """All 65 536 gate values through both epilogues (whole items, joined parts): bit for bit the standalone gate on
    the ungated output."""
    codes = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    for lens, hq in (([(256, 256)], 1), ([(1, 5000)] * 16, 16)):
        b = Batch(lens, hq, 1, seed=22)
        g = codes.view(sum(n for n, _ in lens), hq, D)
        b.gate = None
        o, _ = b.call(gda)
        b.gate = g
        out, _ = b.call(gda)
        w = gda.gate(o, g)
        nan = torch.isnan(w.float())
        assert torch.equal(torch.isnan(out.float()), nan)
        assert torch.equal(out.view(torch.int16)[~nan], w.view(torch.int16)[~nan])


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads", [(16, 2), (24, 1), (12, 4)], ids=str)
@pytest.mark.parametrize("empty", [0, 80])
def test_long_and_short_by_either_kernel(gda, kv, heads, empty):
    """The same sequences, alone and with so many empty ones that the batch goes by a CTA to an item: blocks of 256
    and of 128 rows, tiles of 128 and of 64 keys, parts joined."""
    b = Batch([(150, 900), (1, 2300), (40, 40), (9, 3), (17, 4097)] + [(0, 0)] * empty, *heads, kv=kv, sinks=True, seed=31)
    for window, first in ((0, 0), (100, 70), (64, 0), (1, 1)):
        o, lse = b.check(gda, window, first)
        o2, lse2 = b.call(gda, window, first)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("tokens, positions", [(1, 500), (1, 30000), (4, 20000), (9, 5000), (16, 9000), (20, 12000)])
def test_one_sequence_in_many_parts(gda, kv, tokens, positions):
    b = Batch([(tokens, positions)], kv=kv, seed=32)
    o, lse = b.check(gda)
    o2, lse2 = b.call(gda)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["e4m3", "fp4"])
@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("spike", [0, 59900])
def test_many_small_weights_beside_a_large_one(gda, kv, tokens, spike):
    """One key's weight is 1, all others' 2^-24.6 (4 bits hold 1 as 1.03: 2^-25.4): their sum, 2.4e-3 (1.4e-3), is the
    whole of O.  FP16 probabilities are held 2^7 higher than that, so each is within 2^-11 relative, or 2^-32 of
    the largest."""
    b = Batch([(tokens, 60000)], kv=kv, seed=34, kd=1.0, vd=1.0, gate=False)
    slots = b.k64.shape[0]
    k, v = torch.zeros(slots, 2, D), torch.ones(slots, 2, D)
    at = int(b.indices[spike])
    k[at, :, 0], v[at] = 1.0, 0.0
    k, v = k.bfloat16(), v.bfloat16()
    if kv == "e4m3":
        b.k_pool, b.v_pool = (paged64.quantise8(x, 1.0).cuda().view(torch.float8_e4m3fn) for x in (k, v))
    else:
        (ck, sk), (cv, sv) = plain64.quantise(k, 1.0), plain64.quantise(v, 1.0)
        b.k_pool, b.v_pool = ck.cuda(), cv.cuda()
        b.kw = dict(kv_scales=torch.stack([sk, sv], 2).contiguous().cuda(), k_descale=1.0, v_descale=1.0)
        k, v = plain64.values(ck, sk, 1.0), plain64.values(cv, sv, 1.0)
    b.k64, b.v64 = k.double().cuda(), v.double().cuda()
    b.q[:] = 0
    b.q[..., 0] = 273.0
    o, lse = b.call(gda)
    want = b.want()
    tol = plain64.bound_out(want, 2.0 ** -11, 0) + 60000 * 2.0 ** -32
    assert bool((want.out > 1e-3).all()) and bool(((o.double() - want.out).abs() <= tol).all())


@pytest.mark.parametrize("heads", [(144, 1), (300, 1), (260, 2)], ids=str)
@pytest.mark.parametrize("lens", [[(1, 700)], [(3, 200), (1, 129), (0, 4)], [(9, 9), (1, 500)]], ids=str)
def test_a_token_in_several_blocks(gda, heads, lens):
    """More query heads to a KV head than a block has rows."""
    for kv in ("bf16", "e4m3"):
        Batch(lens, *heads, kv=kv, sinks=True, seed=35).check(gda, 100, 3)


@pytest.mark.parametrize("kv", KV)
def test_strides_of_q_and_gate_apart(gda, kv):
    b = Batch([(3, 200), (40, 700), (1, 1300)], kv=kv, seed=36)
    o, lse = b.check(gda)
    wide = torch.full((44, 16 * D + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :16 * D] = b.gate.reshape(44, 16 * D)
    b.q, b.gate = b.q.contiguous(), wide[:, :16 * D].unflatten(1, (16, D))
    o2, lse2 = b.call(gda)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    b.q, b.gate = b.gate, b.q                      # and the other way round
    b.check(gda)


def test_wait_limit_with_few_rows(gda):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kv in KV:
        b = Batch([(1, 3000), (2, 500), (0, 3), (1, 700)], kv=kv, seed=33)
        want, _ = b.call(gda, error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        try:
            gda.debug_wait_limit(200)           # SM cycles: below the latency of a first load
            b.call(gda, error_word=err)
            torch.cuda.synchronize()            # the call returns
        finally:
            gda.debug_wait_limit(0)
        assert int(err.item()) & gda.DEVERR_TIMEOUT
        err.zero_()
        got, _ = b.call(gda, error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.equal(got, want)


def test_many_short_sequences(gda):
    import random
    r = random.Random(5)
    lens = [(n, n + r.choice([0, 0, 1, 5, 140])) for n in (r.choice([0, 1, 1, 2, 3]) for _ in range(3000))]
    for kv in ("bf16", "fp4"):
        Batch(lens, 2, 1, kv=kv, seed=23).check(gda)
    # and a long one among them: its share of the CTAs is cut over many of them
    Batch(lens[:700] + [(2, 60000)] + lens[700:1400], 2, 1, seed=24).check(gda, window=50000, keep_first=3)


def test_offsets_past_32_bits(gda):
    """Queries, gate, output and pool rows more than 2^32 bytes from the first."""
    T, Hq, n, L = 270000, 32, 130, 300
    rows = torch.zeros(T, 2, Hq, D, dtype=torch.bfloat16, device="cuda")     # 8.8 GB
    b = Batch([(n, L)], Hq, 1, seed=25)
    for i, small in enumerate((b.q, b.gate)):
        rows[T - n:, i] = small
    slots = 9000000                                                          # 4.6 GB a pool
    kp, vp = (torch.zeros(slots, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp[-400:], vp[-400:] = 0.0, 0.0
    far = slots - b.k_pool.shape[0]
    kp[far:], vp[far:] = b.k_pool, b.v_pool
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    gda.prefill_paged(rows[:, 0], rows[:, 1], kp, vp, cu, b.indptr, b.indices + far, out=out, scale=1 / 16)
    want, _ = b.call(gda)
    assert torch.equal(out[T - n:], want) and bool((out[:T - n] == 7.0).all())


@pytest.mark.parametrize("kv", KV)
def test_wrong_lengths_stay_inside(gda, kv):
    """Lengths past the tensors are clamped to them."""
    b = Batch([(5, 300), (7, 200)], kv=kv, seed=26)
    cu, ip = b.cu.clone(), b.indptr.clone()
    cu[2], ip[2] = 2 ** 31 - 1, 2 ** 31 - 1
    want, _ = b.call(gda)
    b.cu, b.indptr = cu, ip
    got, _ = b.call(gda)
    assert torch.equal(got, want)
    b.cu, b.indptr = torch.tensor([-5, 12, 3], dtype=torch.int32).cuda(), torch.tensor([-9, 500, 100], dtype=torch.int32).cuda()
    got, _ = b.call(gda)
    assert bool(got.isfinite().all())


def test_a_prompt_in_chunks_through_the_cache(gda):
    """The calls as a server makes them: each chunk's rotary step, its rows into an 8-bit cache, attention over the
    cache; then single tokens over the same cache.  Against float64 on the rows that the cache holds."""
    Hq, Hkv, kd, vd = 8, 2, 0.0625, 0.03125
    g = torch.Generator(device="cuda").manual_seed(27)
    inv = (1e4 ** (-torch.arange(0, 64, 2, device="cuda") / 64)).float()
    axis = gda.mrope_pair_axis([16, 8, 8])
    kp = torch.zeros(500, Hkv, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vp = torch.zeros_like(kp)
    order = torch.randperm(500, generator=g, device="cuda").to(torch.int32)
    slots = [order[:250], order[250:]]                       # two users' slots
    done = [0, 0]
    for lens in ([70, 1], [130, 40], [1, 1], [4, 1]):        # prompts in chunks, then drafted and single tokens
        T = sum(lens)
        new = torch.cat([s[d:d + n] for s, d, n in zip(slots, done, lens)])
        pos = torch.cat([torch.arange(d, d + n, dtype=torch.int32) for d, n in zip(done, lens)]).cuda()
        qgkv = torch.randn(T, (2 * Hq + 2 * Hkv) * D, generator=g, device="cuda").bfloat16()
        q, k = gda.qk_norm_mrope_kv_write(qgkv, pos.expand(3, T).contiguous(), inv, axis, Hq, Hkv)
        x = qgkv.view(T, 2 * Hq + 2 * Hkv, D)
        gda.kv_write_e4m3(k, x[:, 2 * Hq + Hkv:], new, kp, vp, k_descale=kd, v_descale=vd)
        done = [d + n for d, n in zip(done, lens)]
        idx = torch.cat([s[:d] for s, d in zip(slots, done)])
        cu, ip = cum(lens).cuda(), cum(done).cuda()
        lse = torch.empty(Hq, T, device="cuda")
        out = gda.prefill_paged(q, x[:, Hq:2 * Hq], kp, vp, cu, ip, idx, lse=lse, window=90, keep_first=4, k_descale=kd,
                                v_descale=vd)
        a = paged64.paged(q, x[:, Hq:2 * Hq], paged64.values8(kp, kd).cuda(), paged64.values8(vp, vd).cuda(), cu, ip, idx,
                          1 / 16, 90, 4)
        plain64.check(out, lse.t(), a, 2.0 ** -11, max(done))


def test_refusals(gda):
    b = Batch([(3, 40)], seed=28)
    ok = lambda **kw: b.call(gda, lse=False, **kw)
    ok()
    with pytest.raises(ValueError, match="workspace"):
        ok(workspace=torch.empty(1 << 26, dtype=torch.uint8))
    with pytest.raises(gda.GdaError):
        ok(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    for bad in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="window"):
            ok(window=bad)
        with pytest.raises(ValueError, match="window"):
            ok(keep_first=bad)
    ok(window=(1 << 31) - 1, keep_first=(1 << 31) - 1)
    with pytest.raises(gda.GdaError):
        ok(scale=math.inf)
    with pytest.raises(ValueError, match="out must"):
        ok(out=torch.empty(3, 16, 2 * D, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="error_word"):
        ok(error_word=torch.zeros(1, dtype=torch.int32))
    for name, bad in (("q", b.q[:, :, :128]), ("cu", b.cu[:1]), ("indptr", b.indptr.long()), ("indices", b.indices.cpu()),
                      ("v_pool", b.v_pool[:, :1]), ("k_pool", b.k_pool.float()), ("gate", b.gate[:2])):
        good = getattr(b, name)
        setattr(b, name, bad)
        with pytest.raises((ValueError, TypeError, gda.GdaError)):
            ok()
        setattr(b, name, good)
    with pytest.raises(gda.GdaError):            # heads that are no multiple of the pools'
        gda.prefill_paged(b.q[:, :15], None, b.k_pool, b.v_pool, b.cu, b.indptr, b.indices)
    b.sinks = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="sinks"):
        ok()


@pytest.mark.parametrize("kv", KV)
def test_values_that_are_no_numbers(gda, kv):
    """A NaN in a query, or in a row that it sees, is in its results; tokens of other sequences keep their bits."""
    b = Batch([(3, 700), (40, 300), (1, 2000)], kv=kv, seed=29)
    o, lse = b.call(gda)
    first = b.indices[700 + 5].long()                # seen by every token of the second sequence
    v = b.v_pool.clone()
    if kv == "fp4":
        b.kw["kv_scales"] = b.kw["kv_scales"].clone()
        b.kw["kv_scales"][first, :, 1] = 0x7F
    else:
        v.view(torch.uint8)[first] = 0x7F if kv == "e4m3" else 0xFF
    b.v_pool = v
    b.q[1, 4, 7] = math.nan
    o2, lse2 = b.call(gda)
    assert bool(o2[3:43].isnan().all()) and bool(o2[1, 4].isnan().all()) and bool(lse2[4, 1].isnan())
    rest = torch.ones(44, 16, dtype=torch.bool, device="cuda")
    rest[3:43], rest[1, 4] = False, False
    assert torch.equal(o[rest], o2[rest])
