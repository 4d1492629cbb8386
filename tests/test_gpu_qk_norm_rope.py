"""Norms of queries and keys for each head with the rotary positions on the GPU, against the
formula in 64 bits.

Bounds.  A value is a sum of two terms, each of a normed, weighted value (three roundings of
2^-24 each and the mean's few) and cos or sin (angles within 1e-6, their tables in fp32): off
by at most 2^-19 (|x1| + |x2|) of the weighted norms, then rounded to the type."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests import delta_reference as ref

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(T, H, Hk, D, rot, dtype, seed=0, far=0, weights="dim"):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(1, T, H, D, generator=gen).to(dtype).cuda()
    k = torch.randn(1, T, Hk, D, generator=gen).to(dtype).cuda()
    pos = torch.randint(0, far, (T,), generator=gen) if far else torch.arange(T)
    shapes = {"none": (None, None), "dim": ((D,), (D,)), "head": ((H, D), (Hk, D))}[weights]
    w = [None if s is None else (1 + 0.3 * torch.randn(*s, generator=gen)).cuda() for s in shapes]
    freq = kda.rope_frequencies(rot)[0] if rot else torch.empty(0, dtype=torch.float64, device="cuda")
    return q, k, w[0], w[1], pos.cuda(), freq


def check(x, y, weight, pos, freq, layout, factor, eps):
    want = ref.qk_norm_rope(x, weight, pos, freq, layout, factor, eps)
    n = ref.qk_norm_rope(x, weight, pos * 0, freq, layout, 1.0, eps).abs()
    r = 2 * freq.numel()
    mag = n.clone()
    i = torch.arange(r // 2, device=x.device)
    one, two = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
    mag[..., one] = mag[..., two] = abs(factor) * (n[..., one] + n[..., two])
    err = (y.double() - want).abs()
    lim = HALF[y.dtype] * want.abs() + 2.0 ** -19 * mag + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    assert bool((err <= lim).all()), float((err / lim).max())


def go(q, k, qw, kw, pos, freq, layout="half", factor=1.0, eps=1e-6, **kwargs):
    q0, k0 = q.clone(), None if k is None else k.clone()
    a, b = kda.qk_norm_rope(q, k, qw, kw, pos, freq, layout=layout, factor=factor, eps=eps, **kwargs)
    torch.cuda.synchronize()
    check(q0[0], a[0], qw, pos, freq, layout, factor, eps)
    if k is not None:
        check(k0[0], b[0], kw, pos, freq, layout, factor, eps)
    return a, b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 64), (64, 32), (192, 192), (192, 96), (256, 256),
                                   (256, 64), (80, 80), (96, 24), (40, 8), (6, 4), (7, 2), (128, 0), (512, 512),
                                   (1024, 512), (1, 0), (130, 130), (33, 32)])
def test_dimensions(dtype, layout, D, rot):
    go(*make(37, 3, 2, D, rot, dtype, seed=D + rot), layout=layout)


@pytest.mark.parametrize("weights", ["none", "dim", "head"])
@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (1, 12, 2), (5, 7, 3), (513, 12, 12), (3001, 5, 1), (9, 64, 8), (20, 40, 40)])
def test_sizes(weights, T, H, Hk):
    go(*make(T, H, Hk, 128, 128, torch.bfloat16, seed=T, weights=weights, far=100000))


def test_many_tokens():
    go(*make(16384, 4, 1, 128, 64, torch.bfloat16, seed=2, weights="head"), layout="interleaved", factor=1.2)


def test_queries_alone():
    q, k, qw, kw, pos, freq = make(50, 4, 1, 128, 128, torch.bfloat16)
    assert go(q, None, qw, None, pos, freq)[1] is None


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (66, torch.bfloat16), (512, torch.float32)])
def test_out_of_place_into_views(D, dtype):
    q, k, qw, kw, pos, freq = make(70, 4, 2, D, D // 4 * 2, dtype, seed=4, weights="head")
    big = torch.full((1, 70, 8, D + 8), 7.0, dtype=dtype, device="cuda")
    q0, k0 = q.clone(), k.clone()
    go(q, k, qw, kw, pos, freq, q_out=big[:, :, 1:5, :D], k_out=big[:, :, 5:7, :D])
    assert torch.equal(q, q0) and torch.equal(k, k0)
    assert bool((big[..., D:] == 7).all()) and bool((big[:, :, [0, 7]] == 7).all())


def test_in_place_on_parts_of_one_projection():
    q, k, qw, kw, pos, freq = make(100, 4, 2, 128, 128, torch.bfloat16, seed=5)
    buf = torch.cat([q, k, q], 2)
    qv, kv = buf[:, :, :4], buf[:, :, 4:6]
    rest = buf[:, :, 6:].clone()
    go(qv, kv, qw, kw, pos, freq)
    assert torch.equal(buf[:, :, 6:], rest)


@pytest.mark.parametrize("std", [1e-4, 1.0, 1e4])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
def test_magnitudes(std, eps):
    q, k, qw, kw, pos, freq = make(40, 3, 2, 128, 128, torch.bfloat16, seed=6)
    go(q * std, k * std, qw, kw, pos, freq, eps=eps)


def test_zero_rows():
    q, k, qw, kw, pos, freq = make(40, 3, 2, 128, 128, torch.bfloat16, seed=7)
    q[:, 3] = 0
    a, _ = go(q, k, qw, kw, pos, freq)
    assert bool((a[:, 3] == 0).all())


def test_rows_that_are_not_finite_stay_alone():
    q, k, qw, kw, pos, freq = make(40, 3, 2, 128, 128, torch.bfloat16, seed=8)
    clean, _ = kda.qk_norm_rope(q.clone(), k.clone(), qw, kw, pos, freq)
    q[0, 11, 1, 5], q[0, 20, 2, 9] = float("nan"), float("inf")
    out, _ = kda.qk_norm_rope(q, k, qw, kw, pos, freq)
    rows = torch.ones(40, 3, dtype=torch.bool, device="cuda")
    rows[11, 1] = rows[20, 2] = False
    assert torch.equal(out[0][rows], clean[0][rows]) and torch.isnan(out[0, 11, 1]).all()


def test_positions_of_both_types_and_far():
    for dtype in (torch.int32, torch.int64):
        q, k, qw, kw, pos, freq = make(64, 2, 2, 128, 128, torch.bfloat16, seed=9, far=2 ** 24)
        go(q, k, qw, kw, pos.to(dtype), freq)
    q, k, qw, kw, pos, freq = make(64, 2, 2, 128, 128, torch.bfloat16, seed=9)
    go(q, k, qw, kw, -pos, freq)


def test_the_same_as_norm_and_rope():
    """fp32 rows: the pass gives what gated_norm and rope give one after the other."""
    q, k, qw, kw, pos, freq = make(300, 4, 2, 128, 128, torch.float32, seed=10)
    a = kda.gated_norm(q, qw, eps=1e-6)
    kda.rope(a, None, pos, freq)
    b, _ = kda.qk_norm_rope(q, k, qw, kw, pos, freq)
    assert float((a - b).abs().max()) <= 2.0 ** -20 * float(a.abs().max())


def test_captured_on_another_stream():
    q, k, qw, kw, pos, freq = make(100, 4, 2, 128, 128, torch.bfloat16, seed=11)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    want = [x.clone() for x in kda.qk_norm_rope(q, k, qw, kw, pos, freq, q_out=qo, k_out=ko)]
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        kda.qk_norm_rope(q, k, qw, kw, pos, freq, q_out=qo, k_out=ko)
    qo.zero_(), ko.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    qo.zero_()
    torch.cuda.synchronize()
    kda.qk_norm_rope(q, k, qw, kw, pos, freq, q_out=qo, k_out=ko, stream=s)
    s.synchronize()
    assert torch.equal(qo, want[0])


@pytest.mark.parametrize("T", [0])
def test_no_tokens(T):
    q, k, qw, kw, pos, freq = make(1, 3, 2, 128, 128, torch.bfloat16)
    kda.qk_norm_rope(q[:, :0], k[:, :0], qw, kw, pos[:0], freq)
