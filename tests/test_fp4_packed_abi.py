"""The 4-bit cache, the multi-axis rotary step and packed prompts: the host-side checks of
their C entries and Python functions.  Every refusal here comes before any CUDA call."""
import ctypes

import pytest
import torch

import gated_gqa_attention_gb300 as gda
from gated_gqa_attention_gb300 import build

OK, NULL, ALIGN, SHAPE, UNSUPPORTED, SPLITS, WORKSPACE, ARG = 0, -1, -2, -3, -4, -5, -6, -10
NAN, INF = float("nan"), float("inf")
P = 4096                       # an aligned address that a refused call never reads
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gda.load()


# ---------------------------------------------------------------- decode

def decode_args(**kw):
    a = gda._Args(q=P, gate=P, k_pool=P, v_pool=P, kv_indptr=P, kv_indices=P, out=P, lse=None, num_slots=10, B=2,
                  Hq=16, Hkv=2, D=256, scale=0.0625, num_splits=0, fuse_gate=1, check_indices=0, variant=0,
                  min_chunk=0, window=0, sinks=None, kv_dtype=gda.KV_E2M1, k_descale=1.0, v_descale=1.0,
                  max_len=0, total_len=0, kv_scales=P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change, status", [
    (dict(kv_scales=None), NULL), (dict(kv_scales=P + 8), ALIGN), (dict(k_pool=P + 8), ALIGN),
    (dict(v_pool=P + 8), ALIGN), (dict(k_pool=None), NULL), (dict(gate=None), NULL), (dict(sinks=P + 2), ALIGN),
    (dict(lse=P + 2), ALIGN), (dict(variant=gda.VARIANT_SIMT), UNSUPPORTED),
    (dict(variant=gda.VARIANT_TMA), UNSUPPORTED), (dict(k_descale=NAN), ARG), (dict(v_descale=INF), ARG),
    (dict(v_descale=-INF), ARG), (dict(D=128), UNSUPPORTED), (dict(Hkv=3), SHAPE), (dict(num_splits=257), SPLITS),
    (dict(window=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(total_len=-1), SHAPE), (dict(min_chunk=-1), SHAPE),
    (dict(check_indices=1, num_slots=-1), SHAPE), (dict(kv_dtype=2), UNSUPPORTED), (dict(kv_dtype=4), UNSUPPORTED),
    (dict(kv_dtype=-1), UNSUPPORTED), (dict(B=0), OK), (dict(B=0, kv_scales=None), OK)])
def test_decode_ex_refusals(lib, change, status):
    assert lib.gda_decode_ex(decode_args(**change), P, BIG, None) == status


def test_decode_ex_workspace(lib):
    need = gda.workspace_bytes(2, 16, 2, 256)
    for ws, n in ((None, BIG), (P + 128, BIG), (P, need - 1), (P, 0)):
        assert lib.gda_decode_ex(decode_args(), ws, n, None) == WORKSPACE


def test_workspace_holds_pairs_of_groups(lib):
    # 16 query heads per KV head: two groups a pair, each with its partial [8][D] and lse [8]
    for B, S in ((1, 1), (3, 7), (8, 64)):
        assert gda.workspace_bytes(B, 32, 2, 256, S) >= 256 + B * 4 * S * 8 * (256 + 1) * 4


@pytest.mark.parametrize("change, status", [
    (dict(q=None), NULL), (dict(scales=None), NULL), (dict(scales=P + 4), ALIGN), (dict(v=P + 8), ALIGN),
    (dict(gate=None), NULL), (dict(indptr=P + 1), ALIGN), (dict(kd=NAN), ARG), (dict(vd=INF), ARG),
    (dict(D=64), UNSUPPORTED), (dict(Hkv=5), SHAPE), (dict(splits=300), SPLITS), (dict(B=-1), SHAPE),
    (dict(B=0, q=None, scales=None, out=None), OK)])
def test_decode_fp4_refusals(lib, change, status):
    a = dict(q=P, gate=P, k=P, v=P, scales=P, indptr=P, indices=P, out=P, B=2, Hq=16, Hkv=2, D=256, scale=0.0625,
             kd=1.0, vd=1.0, splits=0, stream=None)
    a.update(change)
    assert lib.gda_decode_fp4(*a.values()) == status


def test_step_host_takes_no_4bit_cache(lib):
    # it has no argument for a scale pool
    args = [t(P) if t is ctypes.c_void_p else t(1) for t in lib.gda_decode_step_host.argtypes]
    args[5] = ctypes.c_int(gda.KV_E2M1)
    assert lib.gda_decode_step_host(*args) == UNSUPPORTED


# ---------------------------------------------------------------- cache writes and reads

@pytest.mark.parametrize("change, status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(k_pool=None), NULL),
    (dict(v_pool=None), NULL), (dict(scales=None), NULL), (dict(k=P + 2), ALIGN), (dict(sk=513), ALIGN),
    (dict(sv=516), ALIGN), (dict(sk=504), SHAPE), (dict(sv=0), SHAPE), (dict(sk=-512), SHAPE), (dict(slots=P + 2), ALIGN),
    (dict(k_pool=P + 8), ALIGN), (dict(scales=P + 8), ALIGN), (dict(kd=0.0), ARG), (dict(kd=-1.0), ARG),
    (dict(vd=NAN), ARG), (dict(vd=INF), ARG), (dict(n=-1), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 40), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(D=128), UNSUPPORTED), (dict(T=0), OK), (dict(T=0, k=None, slots=None), OK)])
def test_kv_write_refusals(lib, change, status):
    a = dict(k=P, sk=512, v=P, sv=512, slots=P, n=10, k_pool=P, v_pool=P, scales=P, kd=1.0, vd=1.0, T=3, Hkv=2, D=256,
             stream=None)
    a.update(change)
    assert lib.gda_kv_write_fp4(*a.values()) == status


@pytest.mark.parametrize("change, status", [
    (dict(k_pool=None), NULL), (dict(scales=None), NULL), (dict(indices=None), NULL), (dict(k_out=None), NULL),
    (dict(v_out=None), NULL), (dict(k_pool=P + 4), ALIGN), (dict(v_out=P + 8), ALIGN), (dict(indices=P + 2), ALIGN),
    (dict(kd=NAN), ARG), (dict(vd=-INF), ARG), (dict(n=-1), SHAPE), (dict(N=-1), SHAPE), (dict(N=1 << 40), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(D=512), UNSUPPORTED), (dict(N=0), OK), (dict(N=0, k_out=None), OK)])
def test_kv_gather_refusals(lib, change, status):
    a = dict(k_pool=P, v_pool=P, scales=P, n=10, indices=P, N=3, kd=1.0, vd=1.0, k_out=P, v_out=P, Hkv=2, D=256,
             stream=None)
    a.update(change)
    assert lib.gda_kv_gather_fp4(*a.values()) == status


# ---------------------------------------------------------------- the rotary step

def mrope_args(axis=bytes(32), **kw):
    a = gda._MropeArgs(qgkv=P, row_stride=36 * 256, w_q_norm=P, w_k_norm=P, eps=1e-6, n_axes=3, positions=P,
                       pos_stride=7, inv_freq=P, pair_axis=axis, rope_dim=64, kv_dtype=gda.KV_E2M1, q_out=P,
                       gate_out=P, k_out=P, slots=P, num_slots=10, k_pool=P, v_pool=P, kv_scales=P, k_descale=1.0,
                       v_descale=1.0, T=7, Hq=16, Hkv=2, D=256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change, status", [
    (dict(qgkv=None), NULL), (dict(q_out=None), NULL), (dict(positions=None), NULL), (dict(inv_freq=None), NULL),
    (dict(pair_axis=None), NULL), (dict(slots=None), NULL), (dict(kv_scales=None), NULL), (dict(v_pool=None), NULL),
    (dict(k_pool=None), NULL), (dict(k_pool=None, v_pool=None, k_out=None), NULL), (dict(qgkv=P + 8), ALIGN),
    (dict(row_stride=36 * 256 + 4), ALIGN), (dict(row_stride=36 * 256 - 8), SHAPE), (dict(w_q_norm=P + 2), ALIGN),
    (dict(k_out=P + 8), ALIGN), (dict(gate_out=P + 8), ALIGN), (dict(positions=P + 2), ALIGN),
    (dict(slots=P + 2), ALIGN), (dict(kv_scales=P + 8), ALIGN), (dict(rope_dim=264), SHAPE), (dict(rope_dim=-16), SHAPE),
    (dict(rope_dim=40), UNSUPPORTED), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(n_axes=0), SHAPE),
    (dict(n_axes=256), SHAPE), (dict(pos_stride=6), SHAPE), (dict(kv_dtype=gda.KV_E4M3), UNSUPPORTED),
    (dict(kv_dtype=2), UNSUPPORTED), (dict(k_descale=0.0), ARG), (dict(v_descale=-2.0), ARG), (dict(v_descale=NAN), ARG),
    (dict(T=-1), SHAPE), (dict(T=1 << 40), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(num_slots=-1), SHAPE), (dict(D=128), UNSUPPORTED), (dict(T=0), OK), (dict(T=0, qgkv=None, q_out=None), OK)])
def test_mrope_refusals(lib, change, status):
    assert lib.gda_qk_norm_mrope_kv_write(mrope_args(**change), None) == status


def test_mrope_axis_of_every_pair_is_checked(lib):
    for i in (0, 31):
        assert lib.gda_qk_norm_mrope_kv_write(mrope_args(axis=bytes(3 if j == i else 2 for j in range(32))), None) == ARG
    assert lib.gda_qk_norm_mrope_kv_write(None, None) == NULL


def test_pair_axis_layouts():
    # contiguous sections of the rotated pairs, or the axes taken in turn while each lasts
    assert list(gda.mrope_pair_axis([2, 1, 1])) == [0, 0, 1, 2]
    got = list(gda.mrope_pair_axis([3, 2, 1], interleaved=True))
    assert sorted(got) == [0, 0, 0, 1, 1, 2] and got[:3] == [0, 1, 2]
    with pytest.raises((ValueError, TypeError)):
        gda.mrope_pair_axis([2, -1])


# ---------------------------------------------------------------- packed prompts

def packed_args(**kw):
    a = gda._PackedArgs(q=P, gate=P, k=P, v=P, q_stride=4096, gate_stride=4096, k_stride=512, v_stride=512,
                        cu_seqlens_q=P, cu_seqlens_k=P, out=P, lse=None, total_q=9, total_k=9, B=2, Hq=16, Hkv=2,
                        D=256, scale=0.0625, causal=1, error_word=P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change, status", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL),
    (dict(cu_seqlens_q=None), NULL), (dict(cu_seqlens_k=None), NULL), (dict(q=P + 8), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(gate=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(cu_seqlens_q=P + 2), ALIGN),
    (dict(cu_seqlens_k=P + 1), ALIGN), (dict(lse=P + 2), ALIGN), (dict(error_word=P + 2), ALIGN),
    (dict(q_stride=4100), ALIGN), (dict(gate_stride=4100), ALIGN), (dict(k_stride=516), ALIGN),
    (dict(v_stride=514), ALIGN), (dict(q_stride=4088), SHAPE), (dict(gate_stride=0), SHAPE), (dict(k_stride=504), SHAPE),
    (dict(v_stride=-512), SHAPE), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=NAN), ARG),
    (dict(scale=INF), ARG), (dict(Hq=15), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=128), UNSUPPORTED), (dict(B=-1), SHAPE),
    (dict(total_q=-1), SHAPE), (dict(total_k=-1), SHAPE), (dict(total_q=1 << 31), SHAPE), (dict(total_k=1 << 31), SHAPE),
    (dict(B=0), OK), (dict(total_q=0), OK), (dict(total_q=0, q=None, out=None), OK)])
def test_packed_refusals(lib, change, status):
    assert lib.gda_prefill_packed(packed_args(**change), None) == status


def test_packed_null_arguments(lib):
    assert lib.gda_prefill_packed(None, None) == NULL


# ---------------------------------------------------------------- the Python functions

def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_python_refuses_cpu_tensors_and_wrong_types():
    codes, scales = torch.zeros(8, 2, 128, dtype=torch.uint8), torch.zeros(8, 2, 2, 16, dtype=torch.uint8)
    i32 = torch.zeros(3, dtype=torch.int32)
    calls = [
        lambda t: gda.kv_write_fp4(t, bf(3, 2, 256), i32, codes, codes, scales),
        lambda t: gda.decode(t, bf(2, 16, 256), codes, codes, i32, i32, kv_scales=scales),
        lambda t: gda.decode_ex(t, bf(2, 16, 256), codes, codes, i32, i32, kv_scales=scales),
        lambda t: gda.prefill_packed(t, None, bf(3, 2, 256), bf(3, 2, 256), i32),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(bf(3, 2, 256))
        with pytest.raises(TypeError, match="must be torch.bfloat16"):
            call(torch.zeros(3, 2, 256))
        with pytest.raises(TypeError, match="torch.Tensor"):
            call([1.0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        gda.kv_gather_fp4(codes, codes, scales, i32)
    with pytest.raises(TypeError, match="uint8"):
        gda.kv_gather_fp4(bf(8, 2, 128), codes, scales, i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gda.qk_norm_mrope_kv_write(bf(3, 36 * 256), None, None, torch.zeros(1, 3, dtype=torch.int32), torch.zeros(32),
                                   bytes(32), 16, 2)
