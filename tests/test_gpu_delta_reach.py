"""The gated delta rule on the GPU where calls meet or offsets are large: one workspace for
several calls and graphs, cut sequences whose tokens clear the state or are not finite, pools and
tensors that reach past 32 bits.  Bounds as in test_gpu_gated_delta.py."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests.test_gpu_gated_delta import D, check, expected, go, make, run

pytestmark = pytest.mark.gpu


def workspace(c, fill=None):
    n = kda.gated_delta_workspace_size(sum(c["lengths"]), len(c["lengths"]), c["v"].shape[2])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    return ws if fill is None else ws.fill_(fill)


@pytest.mark.parametrize("lengths", [[3], [500, 2, 64], [4200]])
def test_workspace_may_hold_anything(lengths):
    c = make(lengths, 2, seed=40)
    before = c["storage"].clone()
    a = run(c, workspace=workspace(c, 0)).clone()
    sa = c["storage"].clone()
    for fill in (0xFF, 0x7F):
        c["storage"].copy_(before)
        b = run(c, workspace=workspace(c, fill))
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert torch.equal(sa.view(torch.int32), c["storage"].view(torch.int32))


def test_graphs_of_one_workspace():
    """Two captured calls of other shapes and an eager one take turns on one workspace."""
    cs = [make([4200], 2, seed=41), make([90, 1, 300], 2, seed=42), make([1, 1], 2, seed=43)]
    wants, befores = [expected(c) for c in cs], [c["storage"].clone() for c in cs]
    ws = max((workspace(c, 0) for c in cs), key=len)
    outs = [torch.empty(c["v"].shape, dtype=torch.bfloat16, device="cuda") for c in cs]
    rest = [(c["cu"].cuda(), c["idx"].cuda(), c["has"].cuda()) for c in cs]

    def call(i):
        c, r = cs[i], rest[i]
        kda.gated_delta_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], r[0], state_cache=c["cache"], state_indices=r[1],
                            has_initial_state=r[2], out=outs[i], cu_seqlens_cpu=c["cu"], workspace=ws)

    for i in range(3):
        call(i)
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=s):
            call(i)
    for _ in range(2):
        for c, b, o in zip(cs, befores, outs):
            c["storage"].copy_(b)
            o.fill_(float("nan"))
        for i in (1, 2, 0):
            graphs[i].replay() if i < 2 else call(i)
        torch.cuda.synchronize()
        for c, o, w, b in zip(cs, outs, wants, befores):
            check(c, o, w, b)


@pytest.mark.parametrize("H,n", [(1, 4500), (6, 3000)])
def test_clears_in_cut_sequences(H, n):
    gen = torch.Generator().manual_seed(44)
    g = -torch.rand(1, n, H, generator=gen) * 0.2
    g[:, torch.randint(n, (n // 500,), generator=gen)] = float("-inf")
    g[:, 700:1400] = 0.0
    go(make([n], H, seed=44, g=g, init=[True]))


@pytest.mark.parametrize("where", ["v", "k", "state"])
def test_not_finite_in_cut_sequences(where):
    """From the token on until one clears the state; in v, its value row alone."""
    n, H, at, clear = 4500, 1, 1000, 3333
    gen = torch.Generator().manual_seed(45)
    g = -torch.rand(1, n, H, generator=gen) * 0.1
    g[:, clear] = float("-inf")
    c = make([n], H, seed=45, g=g, init=[True])
    before = c["storage"].clone()
    clean = run(c).clone()
    final = c["storage"].clone()
    c["storage"].copy_(before)
    slot = int(c["idx"][0])
    if where == "state":
        c["cache"][slot, 0, 5, 7] = float("nan")
        at, rows = 0, [5]
    elif where == "v":
        c["v"][0, at, 0, 5] = float("inf")
        rows = [5]
    else:
        c["k"][0, at, 0, 5] = float("nan")
        rows = list(range(D))
    out = run(c)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[0, at:clear, 0, rows] = True
    assert bool(torch.isnan(out[hit]).all())
    # (the other rows' operands keep their scales; at the clearing token the row's own scale
    # may differ from the clean run's, by what 22 bits allow)
    same = ~hit.any(3, keepdim=True).expand_as(hit) | ~hit
    assert float((out[same].double() - clean[same].double()).norm() / clean[same].double().norm()) <= 2.5e-3
    a, b = c["cache"][slot].double(), final.view_as(c["cache"])[slot].double()
    assert float((a - b).norm() / b.norm()) <= 2.0 ** -17


def test_slots_past_32_bits():
    H, big = 2, 2 ** 32 + 2 ** 31
    c = make([150, 3], H, pool=torch.bfloat16, seed=46, init=[True, True])
    want = expected(c)
    storage = torch.empty(big + H * D * D, dtype=torch.bfloat16, device="cuda")
    cache = storage.as_strided((2, H, D, D), (big, D * D, D, 1))
    order = [1, 0]  # the longer one far away
    for i, slot in enumerate(order):
        cache[slot] = c["cache"][int(c["idx"][i])]
    small = torch.stack([cache[i] for i in range(2)])
    far = dict(c, cache=cache, idx=torch.tensor(order, dtype=torch.int32))
    out = run(far)
    near = dict(c, cache=small, idx=torch.tensor(order, dtype=torch.int32))
    ref = run(near)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    assert torch.equal(cache[0], small[0]) and torch.equal(cache[1], small[1])
    assert float((out[0].double() - want[0]).norm() / want[0].norm()) <= 2.5e-3


@pytest.mark.parametrize("lengths", [[2100], [1030, 4, 1066]])
def test_tokens_past_32_bits(lengths):
    """A token's row 2^21 elements after the last one's: the last rows lie past 2^32."""
    step, H = 2 ** 21 + 8, 2
    c = make(lengths, H, seed=47, init=[True] * len(lengths))
    T = sum(lengths)
    want, before = expected(c), c["storage"].clone()
    room = torch.empty(step * (T - 1) + 3 * H * D, dtype=torch.bfloat16, device="cuda")
    for i, name in enumerate(("q", "k", "v")):
        view = room[i * H * D:].as_strided((1, T, H, D), (T * step, step, D, 1))
        view.copy_(c[name])
        c[name] = view
    check(c, run(c), want, before)


def test_norms_and_turns_past_32_bits():
    T, step = 2100, 2 ** 21 + 8
    gen = torch.Generator().manual_seed(48)
    x = torch.randn(1, T, 3, D, generator=gen).bfloat16().cuda()
    pos = torch.arange(T).cuda()
    freq, _ = kda.rope_frequencies(D)
    want, _ = kda.qk_norm_rope(x.clone(), None, None, None, pos, freq)
    room = torch.empty(step * (T - 1) + 3 * D, dtype=torch.bfloat16, device="cuda")
    view = room.as_strided((1, T, 3, D), (T * step, step, D, 1))
    view.copy_(x)
    kda.qk_norm_rope(view, None, None, None, pos, freq)
    assert torch.equal(view, want)


def test_single_tokens_first_seen_in_a_capture():
    """A call that needs no workspace but its header, made for the first time while a graph is
    captured, on a stream of its own and eagerly afterwards."""
    kda.ops._headers.clear()
    c = make([1, 4], 2, seed=49, init=[True, True])
    want, before = expected(c), c["storage"].clone()
    go(dict(c, cache=c["cache"].clone()))  # the bounds' tables have to be there
    kda.ops._headers.clear()
    out = torch.empty(c["v"].shape, dtype=torch.bfloat16, device="cuda")
    cu, idx, has = c["cu"].cuda(), c["idx"].cuda(), c["has"].cuda()

    def call(**kw):
        kda.gated_delta_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], cu, state_cache=c["cache"], state_indices=idx,
                            has_initial_state=has, out=out, cu_seqlens_cpu=c["cu"], **kw)

    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        call()
    assert not kda.ops._headers
    c["storage"].copy_(before)
    graph.replay()
    torch.cuda.synchronize()
    check(c, out, want, before)
    c["storage"].copy_(before)
    torch.cuda.synchronize()
    call(stream=s)
    s.synchronize()
    assert not kda.ops._headers
    check(c, out, want, before)
    for _ in range(2):
        c["storage"].copy_(before)
        call()
        assert list(kda.ops._headers) == [torch.cuda.current_device()]
        check(c, out, want, before)


def test_the_quick_look_hands_over_what_the_checks_do():
    """The binding's look at the usual forms gives the fields that the checks of each argument
    give, and leaves every other form to them."""
    ops = kda.ops
    x = torch.randn(1, 6, 9, D, device="cuda").bfloat16()
    q, k = x[:, :, :4], x[:, :, 4:6]
    qo, ko = torch.empty(1, 6, 4, D, device="cuda").bfloat16(), torch.empty(1, 6, 2, D, device="cuda").bfloat16()
    w, wq, wk = torch.ones(D, device="cuda"), torch.ones(4, D, device="cuda"), torch.ones(2, D, device="cuda")
    pos, freq = torch.arange(6, device="cuda"), kda.rope_frequencies(D)[0]
    taken = [(q, k, q, k, w, w, pos, freq), (q, k, qo, ko, None, wk, pos.int(), freq), (q, k, q, ko, wq, None, pos, freq[:8]),
             (qo, ko, qo, ko, None, None, pos, freq)]
    for a in taken:
        assert ops._usual_turn(*a) == ops._checked_turn(*a, "half")
    left = [(q[0], k[0], q[0], k[0], w, w, pos, freq), (q[:, :1], k[:, :1], q[:, :1], k[:, :1], w, w, pos[:1], freq),
            (q[:, :, :1], k, q[:, :, :1], k, w, w, pos, freq), (q, k, qo, ko[0], w, w, pos, freq)]
    for a in left:
        assert ops._usual_turn(*a) is None
        ops._checked_turn(*a, "half")
    wrong = [(q, k.half(), q, k.half(), w, w, pos, freq), (q, k, qo.float(), ko, w, w, pos, freq),
             (q, k, q, k, w.half(), w, pos, freq), (q, k, q, k, wk, w, pos, freq), (q, k, q, k, w, w[::2], pos, freq),
             (q, k, q, k, w, w, pos[:5], freq), (q, k, q, k, w, w, pos.float(), freq), (q, k, q, k, w, w, pos, freq.float()),
             (q, k, q, k, w, w, pos, torch.cat([freq, freq])), (q, k[:, :5], q, k[:, :5], w, w, pos, freq),
             (q, k, qo[..., :64], ko, w, w, pos, freq), (q[..., ::2], k[..., ::2], q[..., ::2], k[..., ::2], None, None, pos, freq[:8]),
             (q, k, q, k, w, w, pos.cpu(), freq), (q, k, q, k, w.cpu(), w, pos, freq)]
    for i, a in enumerate(wrong):
        assert ops._usual_turn(*a) is None, i
        with pytest.raises((TypeError, ValueError)):
            ops._checked_turn(*a, "half")


@pytest.mark.parametrize("pool", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lengths", [[16, 9, 17, 3, 12, 0, 100, 15, 1], [9] * 5, [16, 8, 16], [17, 16], [10] * 150 + [1] * 150])
def test_lengths_about_where_chunks_begin(lengths, pool):
    go(make(lengths, 3, 1, seed=50, pool=pool))


def test_bad_slots_of_token_by_token_sequences():
    c = make([12, 9, 2], 2, seed=51, init=[True] * 3)
    c["idx"][0] = -1
    before = c["storage"].clone()
    ws = workspace(c, 0xFF)
    run(c, workspace=ws)
    torch.cuda.synchronize()
    assert kda.check_status(ws) == kda.STATUS_BAD_SLOT
    keep = torch.ones(len(before), dtype=torch.bool, device="cuda")
    keep[c["idx"][1:].long().cuda()] = False
    assert torch.equal(c["storage"][keep].view(torch.int32), before[keep].view(torch.int32))
