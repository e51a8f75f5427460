"""Attention over a paged cache at the ends of its arguments' ranges, against float64: scores of many
millions, queries and descales near the ends of FP32, slots at the end of int32."""
import math

import pytest
import torch

import paged64
import plain64
from test_gpu_paged import Batch, P_STEP

pytestmark = pytest.mark.gpu
D = 256
KV = ["bf16", "e4m3", "fp4"]
CODES = ["e4m3", "fp4"]
LN2 = float(torch.tensor(math.log(2.0)))      # float32(ln 2) log2(e) is 1 in float32: log2 scores are q . k


def set_keys(b, lens, digits):
    """K rows that are 0 but for three dimensions (0, 16, 32), whose values digits(j) gives for position j."""
    slots = b.k64.shape[0]
    k = torch.zeros(slots, b.hkv, D, dtype=torch.float64)
    at = 0
    for _, L in lens:
        slot = b.indices[at:at + L].long().cpu()
        for d, x in zip((0, 16, 32), digits(torch.arange(L))):
            k[slot, :, d] = x.double()[:, None]
        at += L
    b.k64 = k.cuda()
    if b.kv == "e4m3":
        b.k_pool = k.float().to(torch.float8_e4m3fn).cuda()
        assert torch.equal(b.k_pool.double(), b.k64)
    else:   # each value is its block's scale, times the code of 1
        codes = torch.zeros(slots, b.hkv, D // 2, dtype=torch.uint8)
        codes[..., [0, 8, 16]] = 2
        scales = b.kw["kv_scales"].cpu()
        scales[:, :, 0] = 0
        scales[:, :, 0, :3] = k[..., [0, 16, 32]].float().to(torch.float8_e4m3fn).view(torch.uint8)
        b.k_pool, b.kw["kv_scales"] = codes.cuda(), scales.cuda()
        assert torch.equal(plain64.values(codes, scales[:, :, 0]), k)
    b.kw["k_descale"] = 1.0


@pytest.mark.parametrize("kv", CODES)
@pytest.mark.parametrize("log2_base, step", [(24, 8), (25, 8), (26, 8), (27, 16)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("tokens, tile", [(1, 64), (17, 128)], ids=["lone", "pair"])
def test_large_scores_that_rise_slowly(gda, kv, log2_base, step, sign, tokens, tile):
    """Log2 scores of +-2^24 to +-2^27 (FP32 holds them 1 to 16 apart) that rise by 8 or 16 from tile to tile.  The
    scores are exact (sums of three products of powers of two and digits), so the bounds have no term for them."""
    n = 20 if tokens == 1 else 12
    lens = [(tokens, tile * n + 5)] * (60 if tokens == 1 else 24)
    b = Batch(lens, 8, 1, kv=kv, seed=40, gate=False)
    # (to 16 in 4 bits: 256 + 16 * 15 and more digits than 12 or 20 tiles need)
    set_keys(b, lens, lambda j: (torch.full_like(j, 256), (j // tile) % 16, (j // tile) // 16))
    b.q = torch.zeros_like(b.q)
    b.q[..., 0], b.q[..., 16], b.q[..., 32] = sign * 2.0 ** (log2_base - 8), step, 16 * step
    o, lse = b.call(gda, scale=LN2)
    a = b.want(scale=LN2)
    a.sabs = torch.zeros_like(a.sabs)
    plain64.check(o, lse.t(), a, P_STEP[kv], b.longest)


@pytest.mark.parametrize("kv", KV)
def test_a_large_row_leaves_its_neighbours_bits(gda, kv):
    """A row whose scores are of many millions changes no bit of the rows computed beside it."""
    b = Batch([(16, 900), (1, 400)], kv=kv, seed=41)
    o, lse = b.call(gda)
    for row, head in ((0, 0), (5, 11), (15, 7), (16, 3)):
        q = b.q.clone()
        b.q = q.clone()
        b.q[row, head] *= 2.0 ** 30
        o2, lse2 = b.call(gda)
        b.q = q
        rest = torch.ones(17, 16, dtype=torch.bool, device="cuda")
        rest[row, head] = False
        assert bool(o2.isfinite().all())
        assert torch.equal(o[rest], o2[rest]) and torch.equal(lse.t()[rest], lse2.t()[rest])


@pytest.mark.parametrize("kv, log2_q, log2_scale", [
    *[("bf16", e, -4 - e) for e in (-60, 60, 100)],
    *[(kv, e, s) for kv in CODES for e, s in ((60, -64), (100, -104), (124, -125), (-60, 56), (-90, 86), (-110, 106), (-131, 126))]])
def test_queries_near_the_ends_of_their_range(gda, kv, log2_q, log2_scale):
    """Query rows near 2^124, and down to subnormal ones, with a scale that brings the scores to ordinary size."""
    b = Batch([(40, 300), (1, 2000), (3, 3)], kv=kv, seed=42)
    b.q = torch.ldexp(b.q.float(), torch.tensor(log2_q, device="cuda")).bfloat16()
    assert bool(b.q.isfinite().all()) and bool((b.q != 0).any())
    b.check(gda, scale=2.0 ** log2_scale)


@pytest.mark.parametrize("kv", CODES)
def test_rows_of_many_sizes_in_one_call(gda, kv):
    """Query rows from 2^-100 to 2^100 side by side: the smaller ones' scores are 0, the larger ones' of order 1."""
    b = Batch([(40, 300)], kv=kv, seed=43)
    e = torch.randint(-100, 101, (40, 16, 1), generator=torch.Generator().manual_seed(1)).cuda()
    b.q = torch.ldexp(b.q.float(), e).bfloat16()
    b.check(gda, scale=2.0 ** -104)


@pytest.mark.parametrize("kv", CODES)
def test_scores_of_zero_under_a_factor_past_fp32(gda, kv):
    """A scale times a query past 2^128: keys of zeros still score 0, and weigh the same."""
    b = Batch([(3, 500), (1, 2000)], kv=kv, seed=44)
    b.k_pool = torch.zeros_like(b.k_pool.view(torch.uint8)).view(b.k_pool.dtype)
    b.k64 = torch.zeros_like(b.k64)
    b.q = torch.ldexp(b.q.float(), torch.tensor(124, device="cuda")).bfloat16()
    b.check(gda, scale=1024.0)


@pytest.mark.parametrize("kv", CODES)
@pytest.mark.parametrize("vd", [2.0 ** -133, 1e-37, 3e34])
@pytest.mark.parametrize("lens", [[(1, 30000)], [(1, 800)] * 300, [(20, 3000)] * 40], ids=["parts", "lone", "pair"])
def test_v_descales_near_the_ends_of_their_range(gda, kv, vd, lens):
    """A V descale below the normal numbers, near the smallest of them and far up, with outputs that BF16 holds as normal
    numbers; the sums that O is divided by are of hundreds of thousands and millions."""
    b = Batch(lens, 2 if len(lens) > 100 else 8, 1, kv=kv, seed=45, gate=False)
    b.q = torch.zeros_like(b.q)
    if kv == "e4m3":
        codes = 0x78 | (b.v_pool.view(torch.uint8) & 0x06)                # 256 to 448
        b.v_pool, b.v64 = codes.view(torch.float8_e4m3fn), paged64.values8(codes).cuda()
    else:
        b.v_pool = b.v_pool & 0x77
        b.kw["kv_scales"][:, :, 1] = 0x7E                                  # 448 times 0 to 6
        b.v64 = plain64.values(b.v_pool, b.kw["kv_scales"][:, :, 1]).cuda()
    b.kw["v_descale"] = vd = float(torch.tensor(vd))
    o, lse = b.call(gda)
    a = b.want()
    assert bool((a.out * vd > 2.0 ** -125).all()) and bool((a.out * vd < 1e38).all())
    # the bound's absolute terms are for values of ordinary size: without the descale on both sides
    plain64.check(o.double() / vd, lse.t(), a, P_STEP[kv], b.longest)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("slot", [-2 ** 31, -2 ** 31 + 1, -2])
def test_the_lowest_slots_are_reported(gda, kv, slot):
    b = Batch([(4, 300), (1, 200)], kv=kv, seed=46)
    b.indices[10] = slot
    o, lse = b.call(gda)
    torch.cuda.synchronize()
    assert gda.prefill_read_error() == gda.DEVERR_INDEX
    plain64.check(o, lse.t(), b.want(), P_STEP[kv], b.longest)
    b.check(gda, window=50)                        # no query sees it (asserts that the error word stays 0)
