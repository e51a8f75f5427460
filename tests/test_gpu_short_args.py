"""gda_args grew by kv_scales at its end.  A program built with a header from before that passes a struct that ends
there, and nothing behind it may be read for the caches that such a program knows."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import ctypes, sys, torch
import gated_gqa_attention_gb300 as gda
gda.load()
lib = ctypes.CDLL(gda.LIB_PATH)                             # with argument types of its own
libc = ctypes.CDLL(None, use_errno=True)
libc.mmap.restype = ctypes.c_void_p
libc.mmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long]
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
page = 1 << 16
at = libc.mmap(None, 2 * page, 3, 0x22, -1, 0)              # private, anonymous, read and write
assert at not in (None, ctypes.c_void_p(-1).value)
assert libc.mprotect(at + page, page, 0) == 0               # the second page: no access
n = gda._Args.kv_scales.offset                              # the old struct's size
old = ctypes.c_void_p(at + page - n)
B, Hq, Hkv, D, L = 2, 16, 2, 256, 40
g = torch.Generator().manual_seed(1)
q, gate = (torch.randn(B, Hq, D, generator=g).bfloat16().cuda() for _ in range(2))
k, v = (torch.randn(B * L, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
ip = torch.tensor([0, L, 2 * L], dtype=torch.int32, device="cuda")
idx = torch.arange(2 * L, dtype=torch.int32, device="cuda")
ws = torch.zeros(gda.workspace_bytes(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
lib.gda_decode_ex.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
for kv, max_len in ((gda.KV_BF16, 0), (gda.KV_BF16, L), (gda.KV_E4M3, 0), (gda.KV_E4M3, L)):
    kc, vc = (k, v) if kv == gda.KV_BF16 else (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn))
    want = gda.decode_ex(q, gate, kc, vc, ip, idx, max_len=max_len)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    a = gda._Args(q=q.data_ptr(), gate=gate.data_ptr(), k_pool=kc.data_ptr(), v_pool=vc.data_ptr(), kv_indptr=ip.data_ptr(),
                  kv_indices=idx.data_ptr(), out=out.data_ptr(), num_slots=B * L, B=B, Hq=Hq, Hkv=Hkv, D=D, scale=1 / 16,
                  fuse_gate=1, kv_dtype=kv, k_descale=1.0, v_descale=1.0, max_len=max_len)
    ctypes.memmove(old, ctypes.addressof(a), n)
    assert lib.gda_decode_ex(old, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want), (kv, max_len)
print("all read in place")
"""


def test_nothing_is_read_behind_the_older_struct(gda):
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all read in place" in r.stdout, (r.returncode, r.stderr[-2000:])
