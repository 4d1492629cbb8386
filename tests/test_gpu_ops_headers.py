"""Calls of the operators that use nothing of their workspace but its status word, without a
workspace of the caller's: one word of each GPU's for all of them, whatever streams and graphs they run
on.  Bounds as in the operators' own tests."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests.test_gpu_gated_delta import D, check, expected, make, run

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


@pytest.mark.parametrize("op", ["lin", "delta"])
def test_a_header_is_not_memory_that_another_stream_still_reads(op):
    """The word that a call on one stream makes may lie where that stream's earlier work still reads;
    a call on another stream does not write it."""
    if op == "lin":
        calls = [lin_call([1], 92 + i)[0] for i in range(2)]
    else:
        calls = []
        for i in range(2):
            c = make([1], 2, seed=92 + i, init=[True])
            cu, idx, has = c["cu"].cuda(), c["idx"].cuda(), c["has"].cuda()
            out = torch.empty(c["v"].shape, dtype=torch.bfloat16, device="cuda")
            calls.append(lambda c=c, cu=cu, idx=idx, has=has, out=out, **kw: kda.gated_delta_fwd(
                c["q"], c["k"], c["v"], c["g"], c["beta"], cu, state_cache=c["cache"], state_indices=idx,
                has_initial_state=has, out=out, cu_seqlens_cpu=c["cu"], **kw))
    for call in calls:  # the bounds' tables
        call(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    kda.ops._headers.clear()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        x = torch.full((256,), 7, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(2 * 10 ** 8)  # a tenth of a second
        y = x.clone()
        del x
        calls[0]()
    with torch.cuda.stream(b):
        calls[1]()
    torch.cuda.synchronize()
    assert bool((y == 7).all())


def allocations(f):
    torch.cuda.synchronize()
    n = torch.cuda.memory_stats()["allocation.all.allocated"]
    f()
    return torch.cuda.memory_stats()["allocation.all.allocated"] - n


@pytest.mark.parametrize("lengths,few", [([1] * 300, True), ([4] * 90 + [16] * 2 + [0] * 5, True), ([9, 16, 12], True),
                                         ([1] * 200 + [40], False), ([17], False), ([0] * 20 + [17, 100], False)])
def test_the_delta_rule_without_a_workspace(lengths, few):
    """Sequences of at most 16 tokens: nothing is allocated; with a longer one among them the call
    takes its workspace as any other."""
    c = make(lengths, 2, seed=91, init=[i % 3 != 0 for i in range(len(lengths))])
    want, before = expected(c), c["storage"].clone()
    out = torch.empty(c["v"].shape, dtype=torch.bfloat16, device="cuda")
    args = c["q"], c["k"], c["v"], c["g"], c["beta"], c["cu"].cuda()
    kw = dict(state_cache=c["cache"], state_indices=c["idx"].cuda(), has_initial_state=c["has"].cuda(), out=out)

    def call(**more):
        c["storage"].copy_(before)
        return allocations(lambda: kda.gated_delta_fwd(*args, **kw, **more))

    call(cu_seqlens_cpu=c["cu"])
    check(c, out, want, before)
    assert (call(cu_seqlens_cpu=c["cu"]) == 0) == few
    check(c, out, want, before)
    call()
    check(c, out, want, before)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    if few:
        call(cu_seqlens_cpu=c["cu"], workspace=ws)
        check(c, out, want, before)
        assert kda.check_status(ws) == 0
        with pytest.raises(ValueError, match="too small"):
            kda.gated_delta_fwd(*args, **kw, cu_seqlens_cpu=c["cu"], workspace=ws[:128])
    else:
        with pytest.raises((ValueError, kda.KDAError), match="workspace"):
            kda.gated_delta_fwd(*args, **kw, cu_seqlens_cpu=c["cu"], workspace=ws)


@pytest.mark.parametrize("lengths,shared", [([90, 3, 0, 17], True), ([1] * 9, True), ([90, 9], False), ([16, 1], False)])
def test_operators_share_the_tables_of_a_batch(lengths, shared):
    """A batch without sequences of 9 to 16 tokens, which linear attention takes in a chunk and the
    delta rule token by token, has one set of tables for both: either may be captured once the other ran."""
    kda.release_cache()
    call, right = lin_call(lengths, 95, H=2)
    assert right is not None  # (it ran once)
    c = make(lengths, 2, seed=96, init=[True] * len(lengths))
    want, before = expected(c), c["storage"].clone()
    n = kda.cache_entries()
    check(c, run(c), want, before)
    assert kda.cache_entries() - n == (0 if shared else 1)
    if shared:
        kda.release_cache()
        call()
        c["storage"].copy_(before)
        out = torch.empty(c["v"].shape, dtype=torch.bfloat16, device="cuda")
        args = c["q"], c["k"], c["v"], c["g"], c["beta"], c["cu"].cuda()
        kw = dict(state_cache=c["cache"], state_indices=c["idx"].cuda(), has_initial_state=c["has"].cuda(), out=out,
                  cu_seqlens_cpu=c["cu"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.gated_delta_fwd(*args, **kw)
        graph.replay()
        torch.cuda.synchronize()
        check(c, out, want, before)
