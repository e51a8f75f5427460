"""Attention over a paged cache and the 8-bit cache's writes: the host-side checks of their C entries and
Python functions.  Every refusal here comes before any CUDA call."""
import pytest
import torch

import gated_gqa_attention_gb300 as gda
from gated_gqa_attention_gb300 import build

OK, NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE, ARG = 0, -1, -2, -3, -4, -6, -10
NAN, INF = float("nan"), float("inf")
P = 4096                       # an aligned address that a refused call never reads
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gda.load()


@pytest.mark.parametrize("change, status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(k_pool=None), NULL),
    (dict(v_pool=None), NULL), (dict(k=P + 2), ALIGN), (dict(sk=513), ALIGN), (dict(sv=516), ALIGN), (dict(sk=504), SHAPE),
    (dict(sv=0), SHAPE), (dict(sk=-512), SHAPE), (dict(slots=P + 2), ALIGN), (dict(k_pool=P + 8), ALIGN),
    (dict(v_pool=P + 8), ALIGN), (dict(kd=0.0), ARG), (dict(kd=-1.0), ARG), (dict(vd=NAN), ARG), (dict(vd=INF), ARG),
    (dict(n=-1), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 40), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=128), UNSUPPORTED),
    (dict(T=0), OK), (dict(T=0, k=None, slots=None), OK)])
def test_kv_write_refusals(lib, change, status):
    a = dict(k=P, sk=512, v=P, sv=512, slots=P, n=10, k_pool=P, v_pool=P, kd=1.0, vd=1.0, T=3, Hkv=2, D=256, stream=None)
    a.update(change)
    assert lib.gda_kv_write_e4m3(*a.values()) == status


@pytest.mark.parametrize("change, status", [
    (dict(k_pool=None), NULL), (dict(v_pool=None), NULL), (dict(indices=None), NULL), (dict(k_out=None), NULL),
    (dict(v_out=None), NULL), (dict(k_pool=P + 4), ALIGN), (dict(v_out=P + 8), ALIGN), (dict(indices=P + 2), ALIGN),
    (dict(kd=NAN), ARG), (dict(vd=-INF), ARG), (dict(n=-1), SHAPE), (dict(N=-1), SHAPE), (dict(N=1 << 40), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(D=512), UNSUPPORTED), (dict(N=0), OK), (dict(N=0, k_out=None), OK)])
def test_kv_gather_refusals(lib, change, status):
    a = dict(k_pool=P, v_pool=P, n=10, indices=P, N=3, kd=1.0, vd=1.0, k_out=P, v_out=P, Hkv=2, D=256, stream=None)
    a.update(change)
    assert lib.gda_kv_gather_e4m3(*a.values()) == status


def paged_args(**kw):
    a = gda._PagedArgs(q=P, gate=P, q_stride=4096, gate_stride=4096, k_pool=P, v_pool=P, kv_scales=P, num_slots=10,
                       cu_seqlens=P, kv_indptr=P, kv_indices=P, out=P, lse=None, sinks=None, total_q=9, nnz=30, B=2,
                       Hq=16, Hkv=2, D=256, scale=0.0625, window=0, keep_first=0, kv_dtype=gda.KV_E2M1, k_descale=1.0,
                       v_descale=1.0, error_word=P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change, status", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(k_pool=None), NULL), (dict(v_pool=None), NULL),
    (dict(kv_scales=None), NULL), (dict(cu_seqlens=None), NULL), (dict(kv_indptr=None), NULL), (dict(kv_indices=None), NULL),
    (dict(q=P + 8), ALIGN), (dict(gate=P + 8), ALIGN), (dict(out=P + 8), ALIGN), (dict(k_pool=P + 8), ALIGN),
    (dict(v_pool=P + 4), ALIGN), (dict(kv_scales=P + 8), ALIGN), (dict(cu_seqlens=P + 2), ALIGN), (dict(kv_indptr=P + 1), ALIGN),
    (dict(kv_indices=P + 2), ALIGN), (dict(lse=P + 2), ALIGN), (dict(sinks=P + 2), ALIGN), (dict(error_word=P + 2), ALIGN),
    (dict(q_stride=4100), ALIGN), (dict(gate_stride=4100), ALIGN), (dict(q_stride=4088), SHAPE), (dict(gate_stride=0), SHAPE),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=NAN), ARG), (dict(scale=INF), ARG),
    (dict(k_descale=0.0), ARG), (dict(k_descale=-1.0), ARG), (dict(v_descale=NAN), ARG), (dict(v_descale=INF), ARG),
    (dict(scale=1e-30, k_descale=1e-30), ARG), (dict(scale=1e30, k_descale=1e30), ARG), (dict(Hq=15), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(D=128), UNSUPPORTED), (dict(kv_dtype=2), UNSUPPORTED), (dict(kv_dtype=-1), UNSUPPORTED),
    (dict(B=-1), SHAPE), (dict(total_q=-1), SHAPE), (dict(nnz=-1), SHAPE), (dict(num_slots=-1), SHAPE),
    (dict(B=(1 << 31) - 1), SHAPE), (dict(total_q=1 << 28), SHAPE),   # (8 heads a group: 2^31 rows)
    (dict(total_q=1 << 31), SHAPE), (dict(nnz=1 << 31), SHAPE), (dict(window=-1), SHAPE), (dict(keep_first=-1), SHAPE),
    (dict(B=0), OK), (dict(total_q=0), OK), (dict(total_q=0, q=None, out=None), OK)])
def test_paged_refusals(lib, change, status):
    assert lib.gda_prefill_paged(paged_args(**change), P, BIG, None) == status


def test_paged_workspace(lib):
    need = gda.prefill_paged_workspace_bytes(9, 2, 16, 2, 256)
    assert need > 0
    for ws, n in ((None, BIG), (P + 128, BIG), (P, need - 1), (P, 0)):
        assert lib.gda_prefill_paged(paged_args(), ws, n, None) == WORKSPACE
    assert lib.gda_prefill_paged(None, P, BIG, None) == NULL
    for bad in ((-1, 2, 16, 2, 256), (9, -1, 16, 2, 256), (9, 2, 0, 2, 256), (9, 2, 16, 3, 256), (9, 2, 16, 2, 128)):
        assert gda.prefill_paged_workspace_bytes(*bad) == 0


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_python_refuses_cpu_tensors_and_wrong_types():
    codes, i32 = torch.zeros(8, 2, 256, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    calls = [
        lambda t: gda.kv_write_e4m3(t, bf(3, 2, 256), i32, codes, codes),
        lambda t: gda.prefill_paged(t, None, codes, codes, i32, i32, i32),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(bf(3, 2, 256))
        with pytest.raises(TypeError, match="must be torch.bfloat16"):
            call(torch.zeros(3, 2, 256))
        with pytest.raises(TypeError, match="torch.Tensor"):
            call([1.0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        gda.kv_gather_e4m3(codes, codes, i32)
    with pytest.raises(TypeError, match="uint8"):
        gda.kv_gather_e4m3(bf(8, 2, 256), codes, i32)
