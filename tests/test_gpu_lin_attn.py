"""Linear attention with a decay for each head on the GPU, against the recurrence
in 64 bits.

Bounds, element by element.  With A the sum of the absolute terms of a value
(decayed products of |q|, |k|, |v| and the initial state):
  out    the kernels carry decayed scores and states as pairs of bf16 (16 bits)
         or better, so each term is off by at most 2^-16, twice; sums in fp32
         and the decays' exponents stay below that.  With the rounding of out
         to bf16 (8 significant bits, so half a step is at most 2^-8): 2^-8 |o| + 2^-14 A.
  state  terms to 2^-23, decays to a few units of fp32 and at most a few dozen
         roundings of partial sums within a decay's reach: 2^-17 A in fp32, and
         the rounding to a 2-byte pool, 2^-8 or 2^-11 |S| (2^-25 where fp16 is
         subnormal).
"""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
D = 128


def make(lengths, H, Hk=None, *, decay="head", pool=torch.float32, seed=0, fused=False, pad=0,
         init=None, g=None, std=1.0):
    Hk = Hk or H
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)

    def normal(*shape):
        return std * torch.randn(*shape, generator=gen)

    if fused:
        qkv = normal(1, T, 2 * Hk + H, D).bfloat16().cuda()
        q, k, v = qkv[:, :, :Hk], qkv[:, :, Hk:2 * Hk], qkv[:, :, 2 * Hk:]
    else:
        q, k, v = (normal(1, T, h, D).bfloat16().cuda() for h in (Hk, Hk, H))
    if g is None:
        slope = torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
        g = -slope if decay == "head" else -slope * torch.exp(torch.randn(1, T, H, generator=gen))
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lengths, dtype=torch.int64), 0)
    slots = N + 2
    storage = torch.full((slots, H * D * D + pad), float("nan"), dtype=pool)
    storage[:, :H * D * D] = (0.1 * torch.randn(slots, H * D * D, generator=gen)).to(pool)
    storage = storage.cuda()
    cache = storage.as_strided((slots, H, D, D), (H * D * D + pad, D * D, D, 1))
    idx = torch.randperm(slots, generator=gen)[:N].to(torch.int32)
    has = torch.rand(N, generator=gen) < 0.5 if init is None else torch.tensor(init, dtype=torch.bool)
    return dict(q=q, k=k, v=v, g=g.float().cuda(), cu=cu, cache=cache, storage=storage, idx=idx,
                has=has, lengths=lengths)


def run(c, scale=None, out=None, host=True, **kw):
    v = c["v"]
    out = torch.full(v.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    kda.lin_attn_fwd(c["q"], c["k"], v, c["g"], c["cu"].cuda(), state_cache=c["cache"],
                     state_indices=c["idx"].cuda(), has_initial_state=c["has"].cuda(), out=out,
                     scale=scale, cu_seqlens_cpu=c["cu"] if host else None, **kw)
    return out


def expected(c, scale=None):
    g = c["g"] if c["g"].dim() == 1 else c["g"][0]
    return ref.lin_attn(c["q"][0], c["k"][0], c["v"][0], g, c["lengths"],
                        c["cache"][c["idx"].long().cuda()].clone(), c["has"],
                        D ** -0.5 if scale is None else scale)


def check(c, out, want, before):
    o, S, mag, smag = want
    err = (out[0].double() - o).abs()
    lim = 2.0 ** -8 * o.abs() + 2.0 ** -14 * mag + 1e-30
    assert bool((err <= lim).all()), float((err / lim).max())
    sel = c["idx"].long().cuda()
    pool = c["cache"]
    got = pool[sel].double()
    step = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[pool.dtype]
    lim = step * S.abs() + 2.0 ** -17 * smag + (2.0 ** -25 if pool.dtype == torch.float16 else 0) + 1e-30
    err = (got - S).abs()
    assert bool((err <= lim).all()), float((err / lim).max())
    # nothing else is written: other slots and the padding keep their bytes
    keep = torch.ones(pool.shape[0], dtype=torch.bool, device="cuda")
    keep[sel] = False
    plane = pool.shape[1] * D * D
    now = c["storage"]
    bits = torch.int32 if now.dtype == torch.float32 else torch.int16
    assert torch.equal(now[keep].view(bits), before[keep].view(bits))
    assert torch.equal(now[:, plane:].contiguous().view(bits), before[:, plane:].contiguous().view(bits))


def run_and_check(c, **kw):
    want, before = expected(c, kw.get("scale")), c["storage"].clone()
    out = run(c, **kw)
    check(c, out, want, before)
    return out


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257,
                               383, 640, 1025])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_lengths(n, decay):
    run_and_check(make([n], 2, decay=decay, seed=n, init=[n % 2 == 0]))


@pytest.mark.parametrize("pool", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fused", [False, True])
def test_ragged_batch(pool, fused):
    run_and_check(make([37, 0, 59, 1, 300, 8, 128, 0, 131, 9], 6, 2, decay="token", pool=pool,
                       fused=fused, pad=64, seed=3))


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (12, 4), (5, 5)])
def test_heads(H, Hk):
    run_and_check(make([200, 3, 150], H, Hk, seed=H, fused=True))


def test_many_sequences():
    lens = [(7 * i * i) % 311 for i in range(90)]
    run_and_check(make(lens, 3, decay="token", seed=5))


def test_several_segments_of_one_prompt():
    run_and_check(make([2500], 1, decay="token", seed=6, init=[1]))


@pytest.mark.parametrize("lengths,H", [([1025], 2), ([3000], 1), ([4096, 40], 3), ([2500, 1400, 1300, 20, 0, 900], 4),
                                       ([6000] + [130] * 30, 6), ([2048] * 40, 4)])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_cut_sequences(lengths, H, decay):
    """Long sequences that are walked in segments, alone and beside others."""
    run_and_check(make(lengths, H, 1, decay=decay, seed=len(lengths), fused=True,
                       init=[i % 2 == 0 for i in range(len(lengths))]))


@pytest.mark.parametrize("lengths", [[257], [384], [385, 20], [512], [513], [641], [767], [769], [897], [640, 640], [897, 800], [700, 1100, 513]])
@pytest.mark.parametrize("H", [1, 12])
def test_shortest_cut_sequences(lengths, H):
    """Around the lengths from which sequences are cut, for few and more heads."""
    run_and_check(make(lengths, H, 1, decay="token", seed=sum(lengths),
                       init=[i % 2 == 0 for i in range(len(lengths))]))


def test_cut_sequences_extreme_decays():
    gen = torch.Generator().manual_seed(3)
    g = -0.01 * torch.rand(1, 3333, 2, generator=gen)
    g[0, 700, 0] = -float("inf")
    g[0, 1500:1800, 1] = -50.0
    g[0, 3000, 1] = -float("inf")
    run_and_check(make([3333], 2, g=g, seed=4, init=[1]))


def test_decode_batch():
    run_and_check(make([1] * 200, 4, 2, seed=7, pool=torch.bfloat16, init=[1] * 200))


def test_scale():
    run_and_check(make([140, 2], 2, seed=8), scale=-0.3)


@pytest.mark.parametrize("n", [5, 200])
def test_extreme_decays(n):
    """Decays of one (nothing forgotten), of zero (the state cleared) and far below
    exp's range, mixed within a chunk."""
    gen = torch.Generator().manual_seed(n)
    g = torch.randn(1, n, 3, generator=gen).abs().neg() * 0.1
    pick = torch.rand(1, n, 3, generator=gen)
    g[pick < 0.05] = -float("inf")
    g[(pick > 0.1) & (pick < 0.15)] = -1e30
    g[(pick > 0.2) & (pick < 0.5)] = 0.0
    g[(pick > 0.9)] = -30.0
    run_and_check(make([n], 3, g=g, seed=n, init=[1]))


@pytest.mark.parametrize("std", [1e-4, 300.0])
def test_magnitudes(std):
    run_and_check(make([150, 4], 2, seed=9, std=std, init=[0, 0]))


def test_no_decay_over_a_long_prompt():
    """Sums of a thousand terms of one sign: partial sums round, in one direction or both."""
    c = make([1100], 1, g=torch.zeros(1), seed=10, init=[0])
    c["k"].abs_()
    c["v"].abs_()
    run_and_check(c)


@pytest.mark.parametrize("n", [3, 150])
def test_nonfinite_values_stay_in_their_place(n):
    """An infinity or NaN in v reaches its value column from its token on, and no
    other sequence; one in q reaches its own token."""
    c = make([n, 20, n], 2, seed=11, init=[1, 1, 0])
    clean = make([n, 20, n], 2, seed=11, init=[1, 1, 0])
    at = n + 20 + n // 2  # in the last sequence
    c["v"][0, at, 1, 5] = float("nan")
    c["v"][0, n + 20, 0, 77] = float("inf")   # first token of the last sequence
    c["v"][0, n - 1, 0, 3] = -float("inf")    # last token of the first
    c["q"][0, n + 2, 1] = float("nan")
    out, good = run(c), run(clean)
    bad = torch.zeros(good.shape, dtype=torch.bool, device="cuda")
    bad[0, at:, 1, 5] = True
    bad[0, n + 20:, 0, 77] = True
    bad[0, n - 1, 0, 3] = True
    bad[0, n + 2, 1] = True
    assert bool((~torch.isfinite(out[bad])).all())
    assert torch.equal(out[~bad], good[~bad])
    S, T = c["cache"][c["idx"].long().cuda()], clean["cache"][clean["idx"].long().cuda()]
    hit = torch.zeros(S.shape, dtype=torch.bool, device="cuda")
    hit[2, 1, 5] = hit[2, 0, 77] = hit[0, 0, 3] = True
    assert bool((~torch.isfinite(S[hit])).all())
    assert torch.equal(S[~hit], T[~hit])


def test_nan_in_slots_that_are_not_read():
    c = make([150, 1, 0], 2, seed=12, init=[0, 0, 0])
    c["cache"][c["idx"].long().cuda()] = float("nan")
    run_and_check(c)


def test_empty_and_zero():
    c = make([0, 0], 2, seed=13, init=[1, 0])
    run_and_check(c)
    q = torch.empty(1, 0, 2, D, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    kda.lin_attn_fwd(q, q, q, torch.zeros(2, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                     state_cache=c["cache"], state_indices=none, has_initial_state=none.bool(),
                     out=torch.empty_like(q))


def test_same_bits_again_and_without_host_bounds():
    outs = []
    for host in (True, True, False):
        c = make([700, 3, 90], 3, seed=14, decay="token")
        outs.append((run(c, host=host), c["cache"]))
    for o, s in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(s, outs[0][1])


def test_split_call_continues_the_state():
    """A prompt in two calls, the second from the first one's state."""
    c = make([300], 2, seed=15, init=[1])
    want, before = expected(c), c["storage"].clone()
    outs = []
    for a, b, init in ((0, 170, 1), (170, 300, 1)):
        part = dict(c, q=c["q"][:, a:b], k=c["k"][:, a:b], v=c["v"][:, a:b].contiguous(),
                    cu=torch.tensor([0, b - a], dtype=torch.int32), has=torch.tensor([init > 0]))
        outs.append(run(part))
    check(c, torch.cat(outs, 1), want, before)


def test_bad_slots_are_reported():
    c = make([150, 4, 20], 2, seed=16, init=[1, 1, 1])
    c["idx"] = torch.tensor([-1, 77, 2], dtype=torch.int32)
    before = c["storage"].clone()
    ws = torch.empty(kda.lin_attn_workspace_size(174, 3, 2), dtype=torch.uint8, device="cuda")
    run(c, workspace=ws)
    assert kda.check_status(ws) == kda.STATUS_BAD_SLOT
    keep = [i for i in range(before.shape[0]) if i != 2]
    assert torch.equal(c["storage"][keep].view(torch.int32), before[keep].view(torch.int32))
    c["idx"] = torch.tensor([0, 1, 2], dtype=torch.int32)
    run(c, workspace=ws)
    assert kda.check_status(ws) == 0


def test_bad_slots_of_short_sequences_are_reported():
    """Batches of short sequences alone write the status themselves, whatever it held."""
    lengths = [1, 8, 0, 3] + [1] * 300
    c = make(lengths, 2, seed=21, init=[1] * len(lengths))
    ws = torch.full((kda.lin_attn_workspace_size(312, len(lengths), 2),), 255, dtype=torch.uint8, device="cuda")
    good = c["idx"].clone()
    for n, slot in ((0, -1), (2, 999), (303, len(lengths) + 2)):
        c["idx"] = good.clone()
        c["idx"][n] = slot
        before = c["storage"].clone()
        run(c, workspace=ws)
        assert kda.check_status(ws) == kda.STATUS_BAD_SLOT
        c["storage"].copy_(before)
        c["idx"] = good
        run(c, workspace=ws)
        assert kda.check_status(ws) == 0


@pytest.mark.parametrize("lengths", [[1500, 3], [40, 50], [20] * 200 + [1]])
def test_bad_slots_of_long_sequences_are_reported(lengths):
    """Cut, in one wave of CTAs and in several, whatever the status word held."""
    c = make(lengths, 2, seed=22, init=[1] * len(lengths))
    ws = torch.full((kda.lin_attn_workspace_size(sum(lengths), len(lengths), 2),), 255, dtype=torch.uint8,
                    device="cuda")
    good = c["idx"].clone()
    for n in (0, len(lengths) - 1):
        c["idx"] = good.clone()
        c["idx"][n] = -1
        before = c["storage"].clone()
        run(c, workspace=ws)
        assert kda.check_status(ws) == kda.STATUS_BAD_SLOT
        c["storage"].copy_(before)
        c["idx"] = good
        want = expected(c)
        check(c, run(c, workspace=ws), want, before)
        assert kda.check_status(ws) == 0


def test_on_another_stream_and_captured():
    c, d = (make([260, 1, 12], 2, seed=17, decay="token") for _ in range(2))
    want = run(c)
    s = torch.cuda.Stream()
    out = torch.empty_like(want)
    cu, idx, has = d["cu"].cuda(), d["idx"].cuda(), d["has"].cuda()
    start = d["storage"].clone()
    ws = torch.empty(kda.lin_attn_workspace_size(273, 3, 2), dtype=torch.uint8, device="cuda")

    def call():
        kda.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], cu, state_cache=d["cache"],
                         state_indices=idx, has_initial_state=has, out=out,
                         cu_seqlens_cpu=d["cu"], workspace=ws, stream=s)

    s.wait_stream(torch.cuda.current_stream())
    call()
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(d["cache"], c["cache"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    d["storage"].copy_(start)
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(d["cache"], c["cache"])


def test_slots_past_32_bits_of_elements():
    """A pool whose last slot starts beyond 2^32 elements (2-byte states)."""
    H = 16
    per = H * D * D
    slots = 2 ** 32 // per + 3
    free, _ = torch.cuda.mem_get_info()
    if free < 2 * slots * per + (8 << 30):
        pytest.skip("needs 17 GB of free device memory")
    c = make([20, 1], H, seed=18, pool=torch.bfloat16, init=[1, 1])
    big = torch.empty(slots, H, D, D, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([slots - 1, slots - 2])
    big[at] = c["cache"][c["idx"].long().cuda()]
    d = dict(c, cache=big, idx=at.to(torch.int32))
    assert torch.equal(run(c), run(d))
    assert torch.equal(big[at], c["cache"][c["idx"].long().cuda()])


def test_cut_sequences_captured():
    """Sequences walked in segments, in a captured call that is replayed twice."""
    c, d = (make([2600, 1, 1300, 200], 2, seed=19, decay="token", init=[1, 1, 0, 1]) for _ in range(2))
    want = run(c)
    cu, idx, has = d["cu"].cuda(), d["idx"].cuda(), d["has"].cuda()
    ws = torch.empty(kda.lin_attn_workspace_size(4101, 4, 2), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    start = d["storage"].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        kda.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], cu, state_cache=d["cache"], state_indices=idx,
                         has_initial_state=has, out=out, cu_seqlens_cpu=d["cu"], workspace=ws)
    for _ in range(2):
        d["storage"].copy_(start)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(d["cache"], c["cache"])
    assert kda.check_status(ws) == 0


def test_nonfinite_values_in_cut_sequences():
    """As within a chunk: the value's column from its token on, in every later segment."""
    c, clean = (make([3100, 20], 2, seed=20, init=[1, 0]) for _ in range(2))
    c["v"][0, 1700, 1, 9] = float("inf")
    c["v"][0, 100, 0, 64] = float("nan")
    out, good = run(c), run(clean)
    bad = torch.zeros(good.shape, dtype=torch.bool, device="cuda")
    bad[0, 1700:3100, 1, 9] = True
    bad[0, 100:3100, 0, 64] = True
    assert bool((~torch.isfinite(out[bad])).all())
    assert torch.equal(out[~bad], good[~bad])
    S, T = c["cache"][c["idx"].long().cuda()], clean["cache"][clean["idx"].long().cuda()]
    hit = torch.zeros(S.shape, dtype=torch.bool, device="cuda")
    hit[0, 1, 9] = hit[0, 0, 64] = True
    assert bool((~torch.isfinite(S[hit])).all())
    assert torch.equal(S[~hit], T[~hit])
