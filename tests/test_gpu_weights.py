"""The weights that an attention call gives to the values of a row add up to 1: the rounded
probabilities that the matrix instructions multiply are the ones that the row's sum counts.  With
constant values every output is that constant, whatever the scores are."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 256


def spread(*shape, seed, std):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(*shape, generator=g)).bfloat16()


@pytest.mark.parametrize("std", [1.0, 3.0, 10.0])
@pytest.mark.parametrize("want_lse", [True, False])
def test_packed_prompts(gda, std, want_lse):
    """Ones as values.  The products and sums are FP32 sums of the same numbers in different orders, a relative
    2^-12 apart at most (1200 terms of one sign, 2^-24 each), and 1 - 2^-12 rounds to the BF16 1."""
    lens, hq, hkv = [1, 130, 300, 1200], 8, 2
    T = sum(lens)
    q, k = spread(T, hq, D, seed=1, std=std).cuda(), spread(T, hkv, D, seed=2, std=1.0).cuda()
    v = torch.ones(T, hkv, D, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    lse = torch.empty(hq, T, device="cuda") if want_lse else None
    out = gda.prefill_packed(q, None, k, v, cu, lse=lse)
    assert bool((out == 1.0).all()), (int((out != 1.0).sum()), out.numel())
