"""Calls of the operators that use nothing of their workspace but its status word, without a
workspace of the caller's: one word of each GPU's for all of them, whatever streams and graphs they run
on.  Bounds as in the operators' own tests."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests.test_gpu_lin_attn import D

pytestmark = pytest.mark.gpu


def lin_call(lengths, seed, H=3):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)
    q, k, v = (torch.randn(1, T, H, D, generator=gen).bfloat16().cuda() for _ in "qkv")
    g = -torch.rand(1, T, H, generator=gen).cuda()
    cu = torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32)
    pool = torch.randn(N, H, D, D, generator=gen).cuda()
    idx, has = torch.arange(N, dtype=torch.int32).cuda(), torch.ones(N, dtype=torch.bool).cuda()
    out = torch.empty(1, T, H, D, dtype=torch.bfloat16, device="cuda")
    cud = cu.cuda()

    def call(**kw):
        return kda.lin_attn_fwd(q, k, v, g, cud, state_cache=pool, state_indices=idx, has_initial_state=has, out=out,
                                cu_seqlens_cpu=cu, **kw)

    ws = torch.empty(kda.lin_attn_workspace_size(T, N, H), dtype=torch.uint8, device="cuda")
    before = pool.clone()
    call(workspace=ws)
    want = out.clone(), pool.clone()
    pool.copy_(before)
    out.fill_(float("nan"))

    def right():
        ok = torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(pool, want[1])
        pool.copy_(before)
        out.fill_(float("nan"))
        return ok

    return call, right


@pytest.mark.parametrize("lengths", [[1], [8], [3, 0, 5], [9], [1] * 9, [200, 40]])
def test_linear_attention_without_a_workspace(lengths):
    call, right = lin_call(lengths, 80)
    call()
    assert right()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream=s)
    s.synchronize()
    assert right()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert right()


def test_calls_of_four_streams_at_once():
    calls = [lin_call([1] * 8, 81 + i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(3):
        for (call, _), s in zip(calls, streams):
            call(stream=s)
        torch.cuda.synchronize()
        assert all([right() for _, right in calls])
        torch.cuda.synchronize()


def test_single_tokens_allocate_nothing():
    call, right = lin_call([1], 90)
    call()
    torch.cuda.synchronize()
    n = torch.cuda.memory_stats()["allocation.all.allocated"]
    call()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == n
