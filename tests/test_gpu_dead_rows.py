"""Packed prompts: a query that sees no key gives zeros and lse -inf, whatever the keys and values that its block's
other queries see hold."""
import math

import pytest
import torch

from test_gpu_packed import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("gated", [True, False])
def test_dead_rows_beside_non_finite_values(gda, value, gated):
    # 150 of 200 queries see nothing, 22 of them in the block of those that see; 3 of 130; none of 5
    nq, nk = [200, 130, 5], [50, 127, 9]
    b = make(nq, nk, seed=11)
    want, lse = run(gda, b, gated=gated)
    b["v"][0], b["v"][50 + 64], b["k"][50 + 3] = value, value, value
    out, lse2 = run(gda, b, gated=gated)
    for rows in (slice(0, 150), slice(200, 203)):
        assert bool((out[rows] == 0).all()) and bool((lse2[rows] == -math.inf).all())
        assert torch.equal(want[rows].view(torch.int16), out[rows].view(torch.int16))
    assert torch.equal(out[330:], want[330:])          # (the third sequence has none of them)
    assert not bool(torch.isfinite(out[150:200].float()).any())
