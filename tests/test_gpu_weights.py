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


# value 1 under scale 1, and a descale 2^-14 relative to one side of the border between the BF16 numbers 1 and
# 1 + 2^-7: weights that add up to less than 1 - 2^-14, or more than 1 + 2^-14, end on its other side
BORDER = 1.0 + 2.0 ** -8


@pytest.mark.parametrize("side,want", [(1 + 2.0 ** -14, 1.0 + 2.0 ** -7), (1 - 2.0 ** -14, 1.0)])
@pytest.mark.parametrize("lens,hq,kw", [
    ([700, 33, 1, 2000], 16, {}),                                  # the split path
    ([700, 33, 1, 2000], 16, dict(num_splits=3)),
    ([700, 33, 1, 2000], 32, {}),                                  # pairs of groups
    ([700, 33, 1, 600], 16, dict(max_len=700)),                    # one cluster kernel
])
@pytest.mark.parametrize("std", [0.3, 1.0, 3.0])
def test_decode_over_a_4bit_cache(gda, lens, hq, kw, side, want, std):
    hkv, n = 2, sum(lens)
    g = torch.Generator().manual_seed(3)
    kp = torch.randint(0, 256, (n, hkv, D // 2), generator=g, dtype=torch.uint8).cuda()
    vp = torch.full((n, hkv, D // 2), 0x22, dtype=torch.uint8, device="cuda")    # both codes 1
    sc = torch.full((n, hkv, 2, D // 16), 0x30, dtype=torch.uint8, device="cuda")  # e4m3 1/2
    sc[:, :, 1] = 0x38                                                           # e4m3 1
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    idx = torch.randperm(n, generator=g).to(torch.int32).cuda()
    q = spread(len(lens), hq, D, seed=4, std=std).cuda()
    out = gda.decode_ex(q, None, kp, vp, cu, idx, fuse_gate=False, kv_scales=sc, v_descale=BORDER * side, **kw)
    assert bool((out == want).all()), (int((out != want).sum()), out.numel())
