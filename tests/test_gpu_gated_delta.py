"""The gated delta rule with a decay for each head on the GPU, against the recurrence in
64 bits.

Bounds.  A token's factor I - beta k k^T has norm at most one for beta in [0, 2], so an error
once made does not grow; E, for each value row, is the sum of what its tokens wrote,
|beta (v - S k)|, undecayed for 64 tokens (a chunk carries its tokens on one scale).
  state  products' operands carry 22 bits or better, the triangular inverse at most
         quadruples and the keys double a chunk's errors, sums and splits take two bits
         more: a row is off by at most 2^-17 E in length, plus the rounding to a 2-byte
         pool, 2^-8 or 2^-11 |S| (2^-25 where fp16 is subnormal) each.
  out    four operands of 11 bits: 2^-9 scale E, and the rounding to bf16 (8 significant
         bits, half a step is at most 2^-8): 2^-8 |o|.
Rounding errors are of either sign, so over a whole tensor they stay near their mean square:
out within 2.5e-3 relative (its rounding alone gives up to 1.7e-3), fp32 states within 2^-19.
"""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests import delta_reference as ref

pytestmark = pytest.mark.gpu
D = 128


def make(lengths, H, Hk=None, *, decay="token", pool=torch.float32, seed=0, fused=False, pad=0,
         init=None, g=None, beta=None, std=1.0, state=0.1):
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
    if beta is None:
        beta = torch.sigmoid(2 * torch.randn(1, T, H, generator=gen))
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lengths, dtype=torch.int64), 0)
    slots = N + 2
    storage = torch.full((slots, H * D * D + pad), float("nan"), dtype=pool)
    storage[:, :H * D * D] = (state * torch.randn(slots, H * D * D, generator=gen)).to(pool)
    storage = storage.cuda()
    cache = storage.as_strided((slots, H, D, D), (H * D * D + pad, D * D, D, 1))
    idx = torch.randperm(slots, generator=gen)[:N].to(torch.int32)
    has = torch.rand(N, generator=gen) < 0.5 if init is None else torch.tensor(init, dtype=torch.bool)
    return dict(q=q, k=k, v=v, g=g.float().cuda(), beta=beta.float().cuda(), cu=cu, cache=cache,
                storage=storage, idx=idx, has=has, lengths=lengths)


def run(c, scale=None, out=None, host=True, **kw):
    v = c["v"]
    out = torch.full(v.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    kda.gated_delta_fwd(c["q"], c["k"], v, c["g"], c["beta"], c["cu"].cuda(), state_cache=c["cache"],
                        state_indices=c["idx"].cuda(), has_initial_state=c["has"].cuda(), out=out,
                        scale=scale, cu_seqlens_cpu=c["cu"] if host else None, **kw)
    return out


def expected(c, scale=None):
    g = c["g"] if c["g"].dim() == 1 else c["g"][0]
    return ref.gated_delta(c["q"][0], c["k"][0], c["v"][0], g, c["beta"][0], c["lengths"],
                           c["cache"][c["idx"].long().cuda()].clone(), c["has"],
                           D ** -0.5 if scale is None else scale)


def check(c, out, want, before, whole=True):
    o, S, emag, smag = want
    err = (out[0].double() - o).abs()
    lim = 2.0 ** -8 * o.abs() + 2.0 ** -9 * emag + 1e-30
    assert bool((err <= lim).all()), float((err / lim).max())
    sel = c["idx"].long().cuda()
    pool = c["cache"]
    got = pool[sel].double()
    step = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[pool.dtype]
    tiny = D ** 0.5 * (2.0 ** -25 if pool.dtype == torch.float16 else 1e-30)
    serr = (got - S).norm(dim=-1)
    slim = step * S.norm(dim=-1) + 2.0 ** -17 * smag + tiny
    assert bool((serr <= slim).all()), float((serr / slim).max())
    if whole and o.numel():
        assert float(err.norm() / o.norm()) <= 2.5e-3, float(err.norm() / o.norm())
        if pool.dtype == torch.float32:
            assert float(serr.norm() / S.norm()) <= 2.0 ** -19, float(serr.norm() / S.norm())
    # nothing else of the pool's memory has changed
    after = c["storage"].clone()
    H = pool.shape[1]
    keep = torch.ones_like(after, dtype=torch.bool)
    keep[sel, :H * D * D] = False
    bits = {4: torch.int32, 2: torch.int16}[after.element_size()]
    assert torch.equal(after.view(bits)[keep], before.view(bits)[keep])


def go(c, scale=None, whole=True, **kw):
    want, before = expected(c, scale), c["storage"].clone()
    out = run(c, scale, **kw)
    torch.cuda.synchronize()
    check(c, out, want, before, whole)
    return out


LENGTHS = [1, 8, 9, 0, 63, 64, 65, 2, 128, 200, 129, 700]


@pytest.mark.parametrize("pool", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,Hk,fused,decay", [(1, 1, False, "head"), (3, 3, True, "token"), (6, 2, True, "token"),
                                              (4, 1, False, "token")])
def test_ragged(pool, H, Hk, fused, decay):
    go(make(LENGTHS, H, Hk, pool=pool, fused=fused, decay=decay, pad=64, seed=H))


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 128, 129, 191, 192, 193, 1000])
@pytest.mark.parametrize("init", [False, True])
def test_lengths(n, init):
    go(make([n], 2, 1, init=[init], seed=n))


@pytest.mark.parametrize("lengths", [[0], [0, 0, 0], [0, 1, 0], []])
def test_empty(lengths):
    c = make(lengths, 2, seed=3, init=[i % 2 == 0 for i in range(len(lengths))])
    go(c, whole=False)


@pytest.mark.parametrize("H,n", [(1, 5000), (2, 4097), (5, 3333), (12, 2100)])
@pytest.mark.parametrize("pool", [torch.float32, torch.bfloat16])
def test_few_long(H, n, pool):
    go(make([n], H, pool=pool, init=[True], seed=n))


def test_long_beside_short():
    go(make([3000, 1, 2900, 5, 0, 900, 64, 9], 2, seed=5, fused=True))


@pytest.mark.parametrize("H,N,hi", [(2, 400, 40), (3, 200, 130), (12, 40, 300)])
def test_many(H, N, hi):
    gen = torch.Generator().manual_seed(N)
    go(make([int(x) for x in torch.randint(0, hi, (N,), generator=gen)], H, seed=N))


@pytest.mark.parametrize("n", [5, 200])
@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0, 1e-6])
def test_strengths(n, beta):
    go(make([n, n], 2, seed=n, beta=torch.full((1, 2 * n, 2), beta), init=[True, False]))


@pytest.mark.parametrize("n", [8, 300])
@pytest.mark.parametrize("beta", [1.0, 2.0])
def test_repeated_keys(n, beta):
    """One key in all tokens: the inverse's entries do not fall off."""
    c = make([n], 2, seed=1, init=[True], beta=torch.full((1, n, 2), beta))
    c["k"] = c["k"][:, :1].expand(1, n, 2, D).contiguous()
    c["g"] = torch.zeros(2, device="cuda")
    go(c, whole=False)


@pytest.mark.parametrize("n", [6, 400])
@pytest.mark.parametrize("rate", [0.0, 1e-4, 0.3, 5.0, 20.0, 80.0, 1000.0])
def test_decays(n, rate):
    c = make([n, n // 2 + 9], 2, seed=2, init=[True, True])
    c["g"] = -rate * torch.rand(1, c["v"].shape[1], 2, generator=torch.Generator().manual_seed(4)).cuda()
    go(c, whole=False)


def test_weak_decays_behind_strong_ones():
    n = 256
    g = torch.full((1, n, 2), -0.01)
    g[:, 5:60] = -300.0
    g[:, 130:180] = -60.0
    go(make([n], 2, seed=9, g=g, init=[True]))


@pytest.mark.parametrize("std,state", [(1e-4, 1e-5), (1e4, 1e3), (1.0, 1e4), (30.0, 1e-6)])
@pytest.mark.parametrize("n", [4, 500])
def test_magnitudes(n, std, state):
    go(make([n, n], 2, seed=7, std=std, state=state, init=[True, True]))


def test_rows_of_other_magnitudes():
    c = make([300], 2, seed=8, init=[True])
    c["v"] *= torch.exp2(torch.arange(D) % 24 - 12.0).bfloat16().cuda()
    go(c)


def test_zero_keys_and_queries():
    c = make([200], 2, seed=11, init=[True])
    c["k"][:, 20:90] = 0
    c["q"][:, 50:120] = 0
    out = go(c)
    assert torch.isfinite(out).all()


def test_scale():
    go(make([3, 100], 2, seed=12), scale=-2.5)


def test_device_bounds_and_repeatable():
    c = make(LENGTHS, 3, 1, seed=13)
    before = c["storage"].clone()
    a = run(c, host=True).clone()
    sa = c["storage"].clone()
    for host in (False, True):
        c["storage"].copy_(before)
        b = run(c, host=host)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert torch.equal(sa.view(torch.int32), c["storage"].view(torch.int32))


def test_strided_views():
    """q, k and v with gaps between heads and tokens, head-major."""
    c = make([70, 9], 4, 2, seed=14)
    for name in ("q", "k", "v"):
        x = c[name]
        big = torch.full((x.shape[2], x.shape[1] + 3, 2 * D), float("nan"), dtype=x.dtype, device="cuda")
        view = big[:, 1:1 + x.shape[1], 8:8 + D].transpose(0, 1)[None]
        view.copy_(x)
        c[name] = view
    go(c)


def test_unread_states_may_hold_anything():
    c = make([100, 3, 0], 2, seed=15, init=[False, False, False])
    want = expected(c)
    c["cache"][c["idx"].long().cuda()] = float("nan")
    before = c["storage"].clone()
    check(c, run(c), want, before)


def test_slots_outside_the_pool():
    c = make([100, 3, 70, 5], 2, seed=16, init=[True] * 4)
    want = expected(c)
    good, before = c["idx"].clone(), c["storage"].clone()
    c["idx"][0], c["idx"][1] = c["cache"].shape[0], -1
    ws = torch.empty(kda.gated_delta_workspace_size(178, 4, 2), dtype=torch.uint8, device="cuda")
    out = run(c, workspace=ws)
    torch.cuda.synchronize()
    assert kda.check_status(ws) == kda.STATUS_BAD_SLOT
    o = want[0]
    for a, b in ((103, 173), (173, 178)):
        err = (out[0, a:b].double() - o[a:b]).norm() / o[a:b].norm()
        assert float(err) <= 2.5e-3
    sel = torch.tensor([int(good[2]), int(good[3])]).cuda()
    keep = torch.ones(len(before), dtype=torch.bool, device="cuda")
    keep[sel] = False
    assert torch.equal(c["storage"][keep].view(torch.int32), before[keep].view(torch.int32))
    run(dict(c, idx=good), workspace=ws)
    assert kda.check_status(ws) == 0


def test_rows_behind_the_last_sequence():
    c = make([70, 3], 2, seed=17)
    room = torch.full((1, 90, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    go(c, out=room[:, :73])
    assert bool((room[:, 73:] == 7.0).all())


@pytest.mark.parametrize("lengths", [[1], [5000], [300, 1, 40, 0, 9]])
def test_captured_and_replayed(lengths):
    c = make(lengths, 2, seed=18)
    before = c["storage"].clone()
    out = torch.empty(c["v"].shape, dtype=torch.bfloat16, device="cuda")
    args = dict(state_cache=c["cache"], state_indices=c["idx"].cuda(), has_initial_state=c["has"].cuda(),
                out=out, cu_seqlens_cpu=c["cu"])
    ws = torch.empty(kda.gated_delta_workspace_size(sum(lengths), len(lengths), 2), dtype=torch.uint8, device="cuda")
    cu = c["cu"].cuda()

    def call():
        kda.gated_delta_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], cu, workspace=ws, **args)

    call()
    first, state = out.clone(), c["storage"].clone()
    call()
    second, state2 = out.clone(), c["storage"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    c["storage"].copy_(before)
    for o, st in ((first, state), (second, state2)):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.int16), out.view(torch.int16))
        assert torch.equal(st.view(torch.int32), c["storage"].view(torch.int32))


def test_two_streams_at_once():
    cs = [make([600, 5, 70], 2, seed=20 + i) for i in range(2)]
    wants, befores = [expected(c) for c in cs], [c["storage"].clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for c, b in zip(cs, befores):
            c["storage"].copy_(b)
        room = [torch.full(c["v"].shape, float("nan"), dtype=torch.bfloat16, device="cuda") for c in cs]
        rest = [(c["cu"].cuda(), c["idx"].cuda(), c["has"].cuda()) for c in cs]
        torch.cuda.synchronize()
        outs = [kda.gated_delta_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], r[0], state_cache=c["cache"],
                                    state_indices=r[1], has_initial_state=r[2], out=o, cu_seqlens_cpu=c["cu"],
                                    stream=s) for c, s, o, r in zip(cs, streams, room, rest)]
        torch.cuda.synchronize()
    for c, o, w, b in zip(cs, outs, wants, befores):
        check(c, o, w, b)


def test_served_token_by_token():
    """A prompt and then single tokens end where the same tokens at once do."""
    n, steps = 150, 20
    c = make([n + steps], 2, seed=22, init=[True])
    want, before = expected(c), c["storage"].clone()
    at_once = go(c)
    c["storage"].copy_(before)
    outs = []
    for a, b in [(0, n)] + [(n + i, n + i + 1) for i in range(steps)]:
        cu = torch.tensor([0, b - a], dtype=torch.int32)
        part = dict(c, q=c["q"][:, a:b], k=c["k"][:, a:b], v=c["v"][:, a:b], g=c["g"][:, a:b].contiguous(),
                    beta=c["beta"][:, a:b].contiguous(), cu=cu, lengths=[b - a])
        outs.append(run(part))
    check(c, torch.cat(outs, 1), want, before)
    assert at_once.shape == torch.cat(outs, 1).shape


@pytest.mark.parametrize("n", [8, 200])
@pytest.mark.parametrize("where", ["q", "k", "v", "state"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite(n, where, bad):
    """They reach their own sequence and head (in v and the state: their value row, in q: its
    token) from their token on, and a clearing token stops them."""
    t, col, clear = n // 2, 5, n - 2
    g = torch.full((1, 2 * n, 2), -0.1)
    g[:, clear] = -torch.inf
    g[:, n + clear] = -torch.inf
    c = make([n, n], 2, seed=23, g=g, init=[True, True])
    want, before = expected(c), c["storage"].clone()
    o, S = want[0], want[1]
    if where == "state":
        c["cache"][int(c["idx"][0]), 0, col, 3] = bad
        t = 0
    else:
        c[where][0, t, 0, col] = bad
    out = run(c)[0].double()
    torch.cuda.synchronize()
    hit = torch.zeros_like(out, dtype=torch.bool)
    if where == "q":
        hit[t, 0] = True
    elif where == "k":
        hit[t:clear, 0] = True
    else:
        hit[t:clear, 0, col] = True
    assert not torch.isfinite(out[hit]).any()
    err, lim = (out - o).abs(), 2.0 ** -8 * o.abs() + 2.0 ** -9 * want[2] + 1e-30
    assert bool((err <= lim)[~hit].all())
    got = c["cache"][c["idx"].long().cuda()].double()
    assert bool(((got - S).norm(dim=-1) <= 2.0 ** -17 * want[3]).all())
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("n", [8, 200])
def test_not_finite_states_stay(n):
    c = make([n, n], 2, seed=24, init=[True, True])
    want = expected(c)
    c["v"][0, n // 2, 1, 7] = float("nan")
    run(c)
    got = c["cache"][c["idx"].long().cuda()].double()
    hit = torch.zeros(got.shape[:3], dtype=torch.bool, device="cuda")
    hit[0, 1, 7] = True
    assert torch.isnan(got[hit]).all()
    assert bool(((got - want[1]).norm(dim=-1) <= 2.0 ** -17 * want[3])[~hit].all())
