"""Calls that name a stream other than the current one: what a call allocates for itself belongs to the
stream that it runs on."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 256
BUSY = 200_000_000            # GPU cycles of a busy stream: about 0.1 s


def prompt(T=200, hq=4, hkv=2, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, gate, k, v = (torch.randn(T, h, D, generator=g).bfloat16().cuda() for h in (hq, hq, hkv, hkv))
    return q, gate, k, v, torch.tensor([0, 60, T], dtype=torch.int32, device="cuda")


def cache(slots=256, hkv=2, seed=1):
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (slots, hkv, D // 2), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    return (*codes, torch.randint(0x30, 0x40, (slots, hkv, 2, D // 16), generator=g, dtype=torch.uint8).cuda())


def step(hq=4, hkv=2, T=200):
    qgkv = torch.randn(T, (2 * hq + 2 * hkv) * D, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(3, T).contiguous()
    return qgkv, pos, torch.full((32,), 0.01, device="cuda"), [0, 1, 2, 0] * 8, hq, hkv


def calls(gda):
    """name -> (a call that allocates its outputs, as a function of the stream)"""
    p, c, s = prompt(), cache(), step()
    idx = torch.arange(200, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 120, 200], dtype=torch.int32, device="cuda")
    q, g = p[0][:2].contiguous(), p[1][:2].contiguous()
    return {
        "prefill_packed": lambda st: (gda.prefill_packed(*p, stream=st),),
        "qk_norm_mrope_kv_write": lambda st: gda.qk_norm_mrope_kv_write(*s, stream=st),
        "kv_gather_fp4": lambda st: gda.kv_gather_fp4(*c, idx, stream=st),
        "decode": lambda st: (gda.decode(q, g, c[0], c[1], cu, idx, kv_scales=c[2], stream=st),),
        "decode_ex": lambda st: (gda.decode_ex(q, g, c[0], c[1], cu, idx, kv_scales=c[2], stream=st),),
    }


NAMES = ["prefill_packed", "qk_norm_mrope_kv_write", "kv_gather_fp4", "decode", "decode_ex"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_allocated_for_another_stream(gda, name):
    """The current stream is busy: nothing that the call needs may wait in it, and memory that it still has to read
    may not be handed to the call."""
    call = calls(gda)[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes that the current stream reads after it has been busy, freed before the call
    held = [torch.full_like(t, 1.0) for t in want for _ in range(2)]
    copies = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for a, b in zip(copies, held):
        a.copy_(b)
    del held, a, b
    got = call(side)
    side.synchronize()
    early = [t.clone() for t in copies]          # (behind the copies, in the current stream)
    torch.cuda.synchronize()
    assert all(bool((t == 1.0).all()) for t in early)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_workspace_allocated_for_another_stream(gda, monkeypatch):
    """A workspace that decode_ex allocates is still in use when the call returns: the current stream's next
    allocations may not get its memory."""
    call = calls(gda)["decode_ex"]
    want = call(None)[0].clone()
    seen = []
    init = gda.workspace_init
    monkeypatch.setattr(gda, "workspace_init", lambda ws, st=None: (seen.append((ws.data_ptr(), ws.numel())), init(ws, st))[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = call(side)[0]
    ptr, n = seen[0]
    nexts = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() + n <= ptr or ptr + n <= t.data_ptr() for t in nexts)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
