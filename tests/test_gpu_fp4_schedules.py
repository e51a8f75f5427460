"""Decode over a 4-bit cache: the schedules.  One wave of splits that fills the CTAs, planned by the host and on
the device; pairs of query-head groups where a CTA takes many pieces of several tiles."""
import pytest
import torch

import plain64
import test_plan_model_fp4 as model
from test_gpu_fp4 import FP16, batch, run, want

pytestmark = pytest.mark.gpu


def plain_rule(b, Hq, Hkv):
    grid = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    heads = Hkv * -(-(-(-Hq // Hkv // 8)) // (2 if Hq // Hkv > 8 else 1))
    return heads, grid, model.uniform_splits(b["ip"].tolist(), heads, grid, 64)


@pytest.mark.parametrize("lens,Hq,Hkv", [([8192] * 8, 16, 2), ([5000] * 8, 32, 2), ([6500, 6400, 6550, 6300], 40, 2)])
def test_one_wave_that_fills_the_ctas(gda, lens, Hq, Hkv):
    """The rule on the host, the rule on the device and the model's count given explicitly cut alike: the same bits."""
    b = batch(lens, Hq, Hkv, seed=31)
    heads, grid, S = plain_rule(b, Hq, Hkv)
    assert S == grid // (len(lens) * heads) and S & (S - 1) != 0       # the branch that this is about
    o_host, l_host = run(gda, b, max_len=max(lens), total_len=sum(lens))
    o_dev, l_dev = run(gda, b)
    o_s, l_s = run(gda, b, num_splits=S)
    for o, l in ((o_dev, l_dev), (o_s, l_s)):
        assert torch.equal(o, o_host) and torch.equal(l, l_host)
    plain64.check(o_host, l_host, want(b), FP16, max(lens))


@pytest.mark.parametrize("Hq", [32, 40])
@pytest.mark.parametrize("kw", [{}, dict(bound=True), dict(num_splits=3), dict(num_splits=1), dict(window=333)])
def test_pairs_of_groups_with_many_pieces_a_cta(gda, Hq, kw):
    """Ragged batches of 200 sequences on pairs of groups (40 heads: a pair and a lone group per KV head)."""
    lens = torch.randint(0, 900, (200,), generator=torch.Generator().manual_seed(6)).tolist()
    b = batch(lens, Hq, 2, seed=32)
    kw = dict(max_len=max(lens), total_len=sum(lens)) if kw.pop("bound", False) else dict(kw)
    out, lse = run(gda, b, **kw)
    plain64.check(out, lse, want(b, window=kw.get("window", 0)), FP16, 900)
