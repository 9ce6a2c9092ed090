"""Workspaces of wq_attn_kv4 on the GPU."""
import pytest
import torch

import weight_only_quantized_tma_gb300 as wq
from weight_only_quantized_tma_gb300 import _attn

pytestmark = pytest.mark.gpu

D, G, P, H, Hq = 64, 32, 16, 2, 8


def _problem(n, L=3000):
    gen = torch.Generator(device="cuda").manual_seed(n)
    each = -(-L // P)
    pages = wq.wq_kv4_pages(each, H, D, G, P, "cuda")
    kv = torch.randn(2, L, H, D, device="cuda", generator=gen).bfloat16()
    wq.wq_kv4_write(kv[0], kv[1], torch.arange(L, device="cuda"), pages, G, P)
    q = torch.randn(n, Hq, D, device="cuda", generator=gen).bfloat16()
    return dict(q=q, pages=pages, block_table=torch.arange(each, device="cuda", dtype=torch.int32)[None],
                kv_lens=torch.tensor([L], dtype=torch.int32, device="cuda"), group=G, page_size=P,
                cu_q=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n)


@pytest.mark.parametrize("clear_only", [False, True])
@pytest.mark.parametrize("n", [1, 50])
def test_counters_left_by_a_timeout_reach_no_later_call(n, clear_only):
    call = _problem(n)
    want = wq.wq_attn_kv4(**call)
    buf = _attn._ws_cache[(0, _attn._stream(torch.device("cuda", 0)))]
    assert (buf[:16384] == 0).all()
    buf[:16384].view(torch.int32).fill_(1)      # as blocks leave them that arrive when another one has given up
    wq.wq_debug_wait_probe(1_000_000)           # a wait that nothing satisfies runs out after 1 ms
    torch.cuda.synchronize()
    if not clear_only:
        assert wq.wq_device_status() == 1 << 5
    wq.wq_clear_device_status()
    assert wq.wq_device_status() == 0
    got = wq.wq_attn_kv4(**call, out=torch.full_like(want, 7.0))
    assert torch.equal(got, want) and (buf[:16384] == 0).all()


@pytest.mark.parametrize("n", [1, 5, 50])
def test_a_workspace_of_the_callers_own(n):
    call = _problem(n)
    want = wq.wq_attn_kv4(**call)
    need = wq.wq_attn_kv4_workspace_bytes(call["pages"], Hq, D, G, P, torch.bfloat16, max_q=n)
    room = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    room[need:] = 5
    for _ in range(3):
        assert torch.equal(wq.wq_attn_kv4(**call, ws=room[:need]), want)
    assert (room[:16384] == 0).all() and (room[need:] == 5).all()
    with pytest.raises(wq.WQError):
        wq.wq_attn_kv4(**call, ws=room[: need - 16])
