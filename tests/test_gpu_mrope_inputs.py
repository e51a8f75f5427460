"""The rotary step: large frequencies at far positions, the forms of pair_axis, keys that go only into the cache."""
import ctypes
from fractions import Fraction

import pytest
import torch

import gated_gqa_attention_gb300 as gda_module
import plain64
from test_gpu_mrope import make, near

D = 256
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679, 10 ** 100)


def angles(pos, inv, axis):
    """positions[axis[i], t] * inv_freq[i] less whole turns, exactly (float64 would lose it): [T, pairs]."""
    rows = []
    for t in range(pos.shape[1]):
        row = []
        for i, a in enumerate(axis):
            x = Fraction(int(pos[a, t])) * Fraction(float(inv[i])) / (2 * PI)
            row.append(float((x - round(x)) * 2 * PI))
        rows.append(row)
    return torch.tensor(rows, dtype=torch.float64)


def test_the_exact_angle_itself():
    pos, inv = torch.tensor([[3, -7, 100]], dtype=torch.int32), torch.tensor([0.5, 1.25])
    want = torch.remainder(pos[0].double()[:, None] * inv.double() + torch.pi, 2 * torch.pi) - torch.pi
    assert (angles(pos, inv, [0, 0]) - want).abs().max() < 1e-12


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1.0, 1e3, 1e6, 2.0 ** 24, 3e9, 2.0 ** 45, 1e19])
def test_large_frequencies_at_far_positions(gda, size):
    """The angle is a 64-bit fraction of a turn at every frequency, not at those below 1 alone."""
    T, Hq, Hkv = 10, 4, 1
    qgkv, _, _, _, wq, wk = make(T, Hq, Hkv, 128, 2, seed=3)
    g = torch.Generator().manual_seed(5)
    inv = (size * (0.5 + 0.5 * torch.rand(64, generator=g))).float() * torch.where(torch.arange(64) % 5 == 0, -1.0, 1.0)
    pos = torch.randint(-2 ** 31, 2 ** 31, (2, T), generator=g).to(torch.int32)
    pos[0, :4] = torch.tensor([2 ** 31 - 1, -(2 ** 31), 0, 1], dtype=torch.int32)
    axis = [i % 2 for i in range(64)]
    q, k = gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), axis, Hq, Hkv, w_q_norm=wq.cuda(), w_k_norm=wk.cuda())
    x = qgkv.reshape(T, 2 * Hq + 2 * Hkv, D)
    ang = angles(pos, inv, axis)
    near(q, plain64.norm_rope(x[:, :Hq], wq, 1e-6, ang), 128)
    near(k, plain64.norm_rope(x[:, 2 * Hq:2 * Hq + Hkv], wk, 1e-6, ang), 128)


def test_the_bytes_of_pair_axis():
    import numpy as np
    for form in (b"\x02\x00\x01", [2, 0, 1], (2, 0, 1), np.array([2, 0, 1]), torch.tensor([2, 0, 1]), range(2, -1, -1)):
        assert sorted(gda_module._axis_bytes(form)) == [0, 1, 2]
    for bad in (3, 0, None, "012", 1.5):
        with pytest.raises(TypeError, match="pair_axis must be a sequence"):
            gda_module._axis_bytes(bad)
    for bad in ([-1], [256]):
        with pytest.raises(ValueError):
            gda_module._axis_bytes(bad)


@pytest.mark.gpu
def test_pair_axis_is_a_sequence_of_axes(gda):
    """A number is not taken as that many zeros; sequences of any kind of integer are read by their values."""
    import numpy as np
    qgkv, pos, inv, axis, _, _ = make(5, 2, 1, 64, 3, seed=7)
    call = lambda a: gda.qk_norm_mrope_kv_write(qgkv.cuda(), pos.cuda(), inv.cuda(), a, 2, 1)
    ref = call(axis)
    for form in (bytes(axis), tuple(axis), np.array(axis), np.array(axis, dtype=np.uint8), torch.tensor(axis)):
        assert all(torch.equal(a, b) for a, b in zip(call(form), ref))
    with pytest.raises(TypeError):
        call(32)
    with pytest.raises((TypeError, ValueError)):
        call([-1] * 32)


@pytest.mark.gpu
@pytest.mark.parametrize("kv4", [False, True])
def test_keys_into_the_cache_alone(gda, kv4):
    """The C entry without k_out: the same cache rows and queries as with it."""
    T, Hq, Hkv, n = 21, 4, 2, 30
    qgkv, pos, inv, axis, wq, wk = (x.cuda() if isinstance(x, torch.Tensor) else x for x in make(T, Hq, Hkv, 64, 3, seed=9))
    qgkv = qgkv.contiguous()
    slots = torch.randperm(n)[:T].to(torch.int32).cuda()
    shape, dt = ((n, Hkv, D // 2), torch.uint8) if kv4 else ((n, Hkv, D), torch.bfloat16)
    pools = [[torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2)] + [torch.zeros(n, Hkv, 2, 16, dtype=torch.uint8, device="cuda")]
             for _ in range(2)]
    kw = dict(kv_scales=pools[0][2]) if kv4 else {}
    q, _ = gda.qk_norm_mrope_kv_write(qgkv, pos, inv, axis, Hq, Hkv, w_q_norm=wq, w_k_norm=wk, slots=slots, k_pool=pools[0][0],
                                      v_pool=pools[0][1], **kw)
    q2 = torch.empty_like(q)
    a = gda._MropeArgs(qgkv=qgkv.data_ptr(), row_stride=qgkv.shape[1], w_q_norm=wq.data_ptr(), w_k_norm=wk.data_ptr(), eps=1e-6,
                       n_axes=3, positions=pos.data_ptr(), pos_stride=T, inv_freq=inv.data_ptr(), pair_axis=bytes(axis), rope_dim=64,
                       kv_dtype=gda.KV_E2M1 if kv4 else gda.KV_BF16, q_out=q2.data_ptr(), slots=slots.data_ptr(), num_slots=n,
                       k_pool=pools[1][0].data_ptr(), v_pool=pools[1][1].data_ptr(),
                       kv_scales=pools[1][2].data_ptr() if kv4 else None, k_descale=1.0, v_descale=1.0, T=T, Hq=Hq, Hkv=Hkv, D=D)
    assert gda.load().gda_qk_norm_mrope_kv_write(a, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert torch.equal(q2, q) and all(torch.equal(x, y) for x, y in zip(*pools))
