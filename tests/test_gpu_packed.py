"""Gated attention over packed prompts on the GPU against float64 (plain64): lengths around the
128-row tiles, empty sequences, prefixes, dead rows, row pitches, rows of no sequence,
non-finite values in other sequences, captures."""
import math
import random

import pytest
import torch

import plain64
from canary import Guarded, check_all

pytestmark = pytest.mark.gpu
D = 256
BF16 = 2.0 ** -8


def cu(lens, first=0):
    c = [first]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def make(nq, nk, Hq=4, Hkv=2, seed=0, head=0, tail=0):
    """q, gate and v as parts of wider rows; `head` and `tail` rows of no sequence around the batch."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tq, tk = sum(nq) + head + tail, sum(nk) + head + tail
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    rows = r(tq, 2 * Hq * D + 16)
    q, gate = rows[:, :Hq * D].unflatten(1, (Hq, D)), rows[:, Hq * D:2 * Hq * D].unflatten(1, (Hq, D))
    kv = r(tk, 3 * Hkv * D)
    k, v = kv[:, :Hkv * D].contiguous().unflatten(1, (Hkv, D)), kv[:, 2 * Hkv * D:].unflatten(1, (Hkv, D))
    gate.mul_(2.0)
    return dict(q=q, gate=gate, k=k, v=v, cq=cu(nq, head), ck=cu(nk, head))


def run(gda, b, causal=True, gated=True, **kw):
    Tq, Hq, _ = b["q"].shape
    go, gl = Guarded((Tq, Hq, D), torch.bfloat16, fill=7.0), Guarded((Hq, Tq), torch.float32, fill=7.0)
    gda.prefill_packed(b["q"], b["gate"] if gated else None, b["k"], b["v"], b["cq"], cu_seqlens_k=b["ck"], out=go.t, lse=gl.t,
                       scale=1 / 16, causal=causal, **kw)
    check_all(out=go, lse=gl)
    assert gda.prefill_read_error() == 0
    return go.t, gl.t.t()


def verify(gda, b, causal=True, gated=True):
    out, lse = run(gda, b, causal, gated)
    ref = plain64.packed(b["q"], b["gate"] if gated else None, b["k"], b["v"], b["cq"], b["ck"], 1 / 16, causal)
    own = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
    own[int(b["cq"][0]):int(b["cq"][-1])] = True
    assert (out[~own] == 7.0).all() and (lse[~own] == 7.0).all()      # rows of no sequence: left as they were
    for f in ("out", "pv", "lse", "sabs"):
        setattr(ref, f, getattr(ref, f)[own])
    plain64.check(out[own], lse[own], ref, BF16, 0, "causal" if causal else "dense")
    return out, lse


LENS = [
    ([1], [1]), ([128], [128]), ([127, 1, 129], None), ([300], None), ([0, 5, 0, 0, 200, 0], None), ([1] * 40, None),
    ([64, 64, 64], None), ([513, 255, 2, 384], None),
    ([1, 1, 100], [500, 1, 356]),                    # continued prompts, one a single token
    ([200, 300, 130], [50, 0, 129]),                 # fewer keys than queries: dead rows; no keys at all
    ([0, 0], [3, 200]),
]


@pytest.mark.parametrize("nq,nk", LENS)
@pytest.mark.parametrize("causal", [True, False])
def test_matches_float64(gda, nq, nk, causal):
    verify(gda, make(nq, nk or nq, seed=len(nq), head=3, tail=5), causal)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (16, 2), (32, 2), (12, 4), (5, 1)])
def test_head_layouts(gda, Hq, Hkv):
    verify(gda, make([140, 33], [140, 90], Hq, Hkv, seed=Hq))


def test_ungated(gda):
    verify(gda, make([140, 33], [140, 90], seed=3), gated=False)


@pytest.mark.parametrize("seed", range(6))
def test_every_block_is_taken_once(gda, seed):
    """Random batches (to more sequences than a warp keeps in registers): every row of every sequence is
    written, and nothing else -- the blocks are found from the lengths on the device."""
    r = random.Random(seed)
    n = [3, 40, 129, 200, 300, 700][seed]
    nq = [r.choice([0, 1, r.randrange(1, 40), r.randrange(1, 700 if n < 50 else 150)]) for _ in range(n)]
    nk = [x + r.choice([0, 0, r.randrange(200)]) if r.random() < 0.8 else r.randrange(0, x + 1) for x in nq]
    verify(gda, make(nq, nk, 2, 1, seed=seed), causal=seed != 2)


def test_long_prompt(gda):
    """A long sequence among short ones, at the order of blocks that starts the longest first."""
    b = make([2500, 5, 1300], [2500, 5, 2000], 2, 1, seed=21)
    verify(gda, b)


def test_packed_equals_each_sequence_alone(gda):
    nq, nk = [200, 77, 128], [200, 300, 128]
    b = make(nq, nk, seed=4)
    out, _ = run(gda, b)
    for i in range(3):
        rq, rk = slice(int(b["cq"][i]), int(b["cq"][i + 1])), slice(int(b["ck"][i]), int(b["ck"][i + 1]))
        one = gda.prefill_packed(b["q"][rq], b["gate"][rq], b["k"][rk], b["v"][rk], cu([nq[i]]), cu([nk[i]]), scale=1 / 16)
        assert torch.equal(one, out[rq])


def test_non_finite_values_of_other_sequences(gda):
    """NaN and infinities in the rows next to a sequence (another sequence's, or nobody's) reach nothing."""
    b = make([100, 60, 130], [100, 200, 130], seed=5, head=4, tail=9)
    out, lse = run(gda, b)
    ck, cq = b["ck"].tolist(), b["cq"].tolist()
    for name, lo, hi in (("k", ck[1], ck[2]), ("v", ck[1], ck[2]), ("q", cq[1], cq[2]), ("gate", cq[1], cq[2])):
        for rows in (slice(0, 4), slice(lo, hi), slice(b[name].shape[0] - 9, None)):
            b[name][rows] = math.nan
            b[name][rows, :, ::2] = math.inf
    out2, lse2 = run(gda, b)
    for i in (0, 2):
        rq = slice(cq[i], cq[i + 1])
        assert torch.equal(out2[rq], out[rq]) and torch.equal(lse2[rq], lse[rq])
    assert torch.isnan(out2[cq[1]:cq[2]].float()).all()


def test_bad_cu_seqlens_stay_inside_the_tensors(gda):
    """Contents are not checked: values outside [0, total] and decreasing ones are clamped, nothing outside is
    touched (the guard bands), and the sequences that are in order come out right."""
    b = make([100, 50], [100, 50], seed=6)
    want, _ = run(gda, b)
    b["cq"] = torch.tensor([0, 100, 10 ** 9], dtype=torch.int32, device="cuda")
    out, _ = run(gda, b)
    assert torch.equal(out[:100], want[:100])
    for bad in ([-5, 100, 50], [-(2 ** 31), 2 ** 31 - 1, 0], [150, 150, 151]):
        b["cq"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        b["ck"] = b["cq"].flip(0).contiguous()
        run(gda, b)


def test_captured_call_follows_the_lengths(gda):
    b = make([130, 70], [130, 70], seed=7)
    out, lse = torch.zeros(200, 4, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 200, device="cuda")
    call = lambda: gda.prefill_packed(b["q"], b["gate"], b["k"], b["v"], b["cq"], out=out, lse=lse, scale=1 / 16)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    b["cq"].copy_(cu([11, 189]))
    g.replay()
    torch.cuda.synchronize()
    ref = plain64.packed(b["q"], b["gate"], b["k"], b["v"], b["cq"], b["cq"], 1 / 16, True)
    plain64.check(out, lse.t(), ref, BF16, 0)


def test_two_streams_at_once(gda):
    bs = [make([400, 20], [400, 20], seed=8), make([33] * 20, [33] * 20, seed=9)]
    refs = [run(gda, b)[0] for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (s, b) in enumerate(zip(streams, bs)):
            with torch.cuda.stream(s):
                outs[i].append(gda.prefill_packed(b["q"], b["gate"], b["k"], b["v"], b["cq"], scale=1 / 16))
    torch.cuda.synchronize()
    assert all(torch.equal(o, refs[i]) for i in range(2) for o in outs[i])


def test_every_gate_code(gda):
    """All 65 536 gate values through the epilogue, in blocks written by TMA and row by row: bit for bit the
    standalone gate on the ungated output."""
    T, Hq = 128 + 128, 1                         # 65 536 gate values
    codes = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).view(T, Hq, D)
    for lens in ([128, 128], [100, 156]):
        b = make(lens, lens, Hq, 1, seed=10)
        b["gate"] = codes
        o = gda.prefill_packed(b["q"], None, b["k"], b["v"], b["cq"], scale=1 / 16)
        out = gda.prefill_packed(b["q"], codes, b["k"], b["v"], b["cq"], scale=1 / 16)
        w = gda.gate(o, codes)
        nan = torch.isnan(w.float())
        assert torch.equal(torch.isnan(out.float()), nan)
        assert torch.equal(out.view(torch.int16)[~nan], w.view(torch.int16)[~nan])


def test_a_prompt_continued_from_the_cache(gda):
    """A first chunk through the step before attention and the packed attention with its rows into the 4-bit
    cache; the second chunk attends to the gathered cache rows and its own.  Against float64 on the same rows."""
    Hq, Hkv, first, second = 8, 2, [70, 1], [50, 129]
    g = torch.Generator(device="cuda").manual_seed(22)
    inv = (1e4 ** (-torch.arange(0, 64, 2, device="cuda") / 64)).float()
    axis = gda.mrope_pair_axis([16, 8, 8])
    kp = torch.zeros(300, Hkv, D // 2, dtype=torch.uint8, device="cuda")
    vp, sc = torch.zeros_like(kp), torch.zeros(300, Hkv, 2, D // 16, dtype=torch.uint8, device="cuda")
    order = torch.randperm(300, generator=g, device="cuda").to(torch.int32)

    def step(lens, start, slots):
        T = sum(lens)
        qgkv = torch.randn(T, (2 * Hq + 2 * Hkv) * D, generator=g, device="cuda").bfloat16()
        pos = torch.cat([torch.arange(n, dtype=torch.int32) + s for n, s in zip(lens, start)]).cuda().expand(3, T).contiguous()
        q, k = gda.qk_norm_mrope_kv_write(qgkv, pos, inv, axis, Hq, Hkv, slots=slots, k_pool=kp, v_pool=vp, kv_scales=sc)
        x = qgkv.view(T, 2 * Hq + 2 * Hkv, D)
        return q, x[:, Hq:2 * Hq], k, x[:, 2 * Hq + Hkv:]

    q, gate, k, v = step(first, [0, 0], order[:71])
    out = gda.prefill_packed(q, gate, k, v, cu(first), scale=1 / 16)
    plain64.check(out, None, plain64.packed(q, gate, k, v, cu(first), cu(first), 1 / 16, True), BF16, 0)
    q, gate, k, v = step(second, first, order[71:71 + 179])
    ck, cv = gda.kv_gather_fp4(kp, vp, sc, order[:71])
    K = torch.cat([ck[:70], k[:50], ck[70:], k[50:]])
    V = torch.cat([cv[:70], v[:50], cv[70:], v[50:]])
    nk = cu([120, 130])
    out = gda.prefill_packed(q, gate, K, V, cu(second), cu_seqlens_k=nk, scale=1 / 16)
    plain64.check(out, None, plain64.packed(q, gate, K, V, cu(second), nk, 1 / 16, True), BF16, 0)


# ---------------------------------------------------------------- a wait that runs out

def test_wait_limit_gives_a_typed_timeout(gda):
    # 5 sequences, several items per CTA pair and more than one key tile: every role has waits
    lens = (300, 1, 129, 0, 513)
    T, hq, hkv = sum(lens), 16, 2
    g = torch.Generator().manual_seed(23)
    q, gate, k, v = (torch.randn(T, h, 256, generator=g).bfloat16().cuda() for h in (hq, hq, hkv, hkv))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: gda.prefill_packed(q, gate, k, v, cu, error_word=err)
    want = call()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    try:
        gda.debug_wait_limit(200)           # SM cycles: below the latency of a first load
        call()
        torch.cuda.synchronize()            # the call returns
    finally:
        gda.debug_wait_limit(0)
    assert int(err.item()) & gda.DEVERR_TIMEOUT
    err.zero_()
    got = call()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("lens", [(129, 195, 255, 131) * 8, (195,) * 24 + (1000,) * 4, (300, 449, 513) * 6])
def test_the_last_tile_waits_for_its_own_values(gda, lens):
    # ones as values: every output is the sum of the rounded probabilities over that of the unrounded
    # ones, within 2^-8 of 1, then rounded to BF16: 1 + 2^-7 at most (the step there), 1 - 2^-8 at
    # least.  Values cleared or replaced while a tile still reads them lower it
    T, hq, hkv = sum(lens), 32, 2
    g = torch.Generator().manual_seed(29)
    q, k = (torch.randn(T, h, 256, generator=g).bfloat16().cuda() for h in (hq, hkv))
    v = torch.ones(T, hkv, 256, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(24):
        cold.fill_(i)
        out = gda.prefill_packed(q, None, k, v, cu)
        assert float((out.float() - 1.0).abs().max()) <= 2.0 ** -7, i


def test_the_gate_alone_on_every_code(gda):
    """One key with ones as values: the attention result is exactly 1, and the output is the sigmoid of the gate
    to the nearest BF16, for all 65536 codes."""
    codes = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    want = 1.0 / (1.0 + torch.exp(-codes.double()))
    for lens in ([256], [1, 100, 155]):
        q = torch.randn(256, 1, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
        one = torch.ones(len(lens), 1, D, dtype=torch.bfloat16, device="cuda")
        cq = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        ck = torch.arange(len(lens) + 1, dtype=torch.int32, device="cuda")
        out = gda.prefill_packed(q, codes.cuda().view(256, 1, D), one, one, cq, ck, causal=False).cpu().view(-1)
        got = out.double()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        # a nearest value is within half a step of its own binade (2^-133 among the subnormal numbers), and no
        # sigmoid but 1/2 and those that round to 0 and 1 is a tie
        step = torch.maximum(torch.exp2(torch.floor(torch.log2(want[~nan].clamp(min=1e-45))) - 8), torch.tensor(2.0 ** -134))
        assert bool(((got - want)[~nan].abs() <= step).all())


def test_offsets_past_32_bits(gda):
    """Queries, gate and output whose last rows lie more than 2^32 bytes from the first."""
    T, Hq, n = 270000, 32, 130
    rows = torch.zeros(T, 2, Hq, D, dtype=torch.bfloat16, device="cuda")     # 8.8 GB
    k, v = (torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b = make([n], [n], Hq, 1, seed=31)
    for big, small in ((rows[:, 0], b["q"]), (rows[:, 1], b["gate"]), (k, b["k"]), (v, b["v"])):
        big[T - n:] = small[-n:]
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    c = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    gda.prefill_packed(rows[:, 0], rows[:, 1], k, v, c, out=out, scale=1 / 16)
    want = gda.prefill_packed(b["q"][-n:], b["gate"][-n:], b["k"][-n:], b["v"][-n:], cu([n]), scale=1 / 16)
    assert torch.equal(out[T - n:], want) and bool((out[:T - n] == 7.0).all())


def test_thousands_of_short_sequences(gda):
    r = random.Random(5)
    nq = [r.choice([0, 1, 1, 2, 3]) for _ in range(3000)]
    nk = [x + r.choice([0, 0, 1, 5]) for x in nq]
    verify(gda, make(nq, nk, 2, 1, seed=41))
