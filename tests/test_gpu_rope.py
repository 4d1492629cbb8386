"""Rotary positions on the GPU against the definition in 64 bits.

Bounds, element by element: the angle is off by at most 1e-6 radians, cos and sin
by 2^-23 and the two products and their sum by 2^-23 of |x1| + |x2|; the result is
rounded to the type: 2^-8 (bf16), 2^-11 (fp16) or 2^-24 (fp32) of it."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def check(y, x, pos, freq, layout, factor, inverse=False):
    want = ref.rope(x, pos, freq, layout, factor, inverse)
    r = 2 * freq.numel()
    size = torch.zeros_like(want)
    size[..., :r] = x.double()[..., :r].abs().amax(-1, keepdim=True) if r else 0
    lim = STEP[x.dtype] * want.abs() + 2 * abs(factor) * (1e-6 + 2.0 ** -21) * size
    if x.dtype == torch.float16:
        lim += 2.0 ** -25
    err = (y.double() - want).abs()
    assert bool((err <= lim).all()), float((err / lim.clamp(min=1e-30)).max())
    assert torch.equal(y[..., r:], x[..., r:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 32), (192, 64), (80, 40), (7, 6),
                                   (128, 2), (96, 96), (128, 0), (1024, 1024)])
def test_shapes(layout, dtype, D, rot):
    T = 37
    q, k = (torch.randn(1, T, h, D, device="cuda").to(dtype) for h in (5, 2))
    pos = torch.randint(0, 10000, (T,), device="cuda", dtype=torch.int32)
    freq = kda.rope_frequencies(rot)[0] if rot else torch.empty(0, dtype=torch.float64, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kda.rope(q, k, pos, freq, layout=layout, factor=1.2, q_out=qo, k_out=ko)
    check(qo[0], q[0], pos, freq, layout, 1.2)
    check(ko[0], k[0], pos, freq, layout, 1.2)
    a, b = q.clone(), k.clone()
    assert kda.rope(a, b, pos, freq, layout=layout, factor=1.2)[0] is a
    assert torch.equal(a, qo) and torch.equal(b, ko)


@pytest.mark.parametrize("T", [1, 2, 3, 255, 700, 5000])
def test_lengths(T):
    q = torch.randn(1, T, 12, 128, device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda")
    freq, _ = kda.rope_frequencies(128)
    out, none = kda.rope(q, None, pos, freq, q_out=torch.empty_like(q))
    assert none is None
    check(out[0], q[0], pos, freq, "half", 1.0)


@pytest.mark.parametrize("scaling", [None, "linear", "base", "ramp"])
def test_far_and_negative_positions(scaling):
    pos = torch.tensor([0, 1, -1, 4097, 131071, 1 << 20, (1 << 28) - 1, -(1 << 28)], device="cuda")
    freq, factor = kda.rope_frequencies(128, scaling=scaling, factor=8.0 if scaling else 1.0,
                                        original_positions=4096)
    x = torch.randn(1, 8, 3, 128, device="cuda")
    y, _ = kda.rope(x, None, pos, freq, factor=factor, q_out=torch.empty_like(x))
    # the definition's own product is exact to 2^-53 of the angle only: 2^28 * 2^-53 = 3e-8
    check(y[0], x[0], pos, freq, "half", factor)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_views_in_place(layout):
    """q and k as views of one projection's output, rotated where they are."""
    qkv = torch.randn(1, 50, 9, 128, device="cuda").bfloat16()
    was = qkv.clone()
    freq, _ = kda.rope_frequencies(64)
    pos = torch.arange(50, device="cuda")
    kda.rope(qkv[:, :, :4], qkv[:, :, 4:6], pos, freq, layout=layout)
    check(qkv[0, :, :6], was[0, :, :6], pos, freq, layout, 1.0)
    assert torch.equal(qkv[:, :, 6:], was[:, :, 6:])


def test_odd_strides_and_offsets():
    """Rows that start off 16-byte boundaries take the narrow path."""
    buf = torch.randn(30 * 517 + 3, device="cuda").bfloat16()
    x = buf[3:].as_strided((30, 4, 128), (517, 129, 1))
    y = torch.empty(30, 4, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(30, device="cuda", dtype=torch.int32)
    freq, _ = kda.rope_frequencies(128)
    kda.rope(x, None, pos, freq, q_out=y)
    check(y, x, pos, freq, "half", 1.0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_the_gradient(layout):
    """<rope(x), dy> has the gradient rope(dy, inverse): checked against the formula's
    gradient, and against differences of the fp32 forward, whose error over a step
    of 0.5 is a few 2^-23 of the values for a linear map."""
    T, H, D = 9, 2, 32
    x, dy = torch.randn(1, T, H, D, device="cuda"), torch.randn(1, T, H, D, device="cuda")
    pos = torch.randint(0, 5000, (T,), device="cuda")
    freq, _ = kda.rope_frequencies(24)
    dx, _ = kda.rope(dy, None, pos, freq, layout=layout, factor=1.3, inverse=True, q_out=torch.empty_like(dy))
    xr = x[0].double().requires_grad_()
    (ref_y,) = [ref.rope(xr, pos, freq, layout, 1.3)]
    want = torch.autograd.grad(ref_y, xr, dy[0].double())[0]
    # the copied dimensions' gradient is dy itself
    assert float((dx[0, ..., :24].double() - want[..., :24]).abs().max()) < 3e-5
    assert torch.equal(dx[..., 24:], dy[..., 24:])
    def fwd(z):
        return kda.rope(z, None, pos, freq, layout=layout, factor=1.3, q_out=torch.empty_like(z))[0].double()
    for e in [(0, 0, 0), (3, 1, 5), (8, 0, 23), (4, 1, 30)]:
        step = torch.zeros_like(x)
        step[(0,) + e] = 0.5
        diff = ((fwd(x + step) - fwd(x - step)) * dy.double()).sum()
        assert abs(float(diff) - float(dx[(0,) + e])) < 1e-4


def test_no_tokens_and_no_heads():
    freq, _ = kda.rope_frequencies(128)
    q = torch.empty(1, 0, 4, 128, device="cuda")
    kda.rope(q, q.clone(), torch.empty(0, dtype=torch.int32, device="cuda"), freq)
    x, none = torch.randn(1, 3, 2, 128, device="cuda"), torch.empty(1, 3, 0, 128, device="cuda")
    was = x.clone()
    kda.rope(x, none, torch.zeros(3, dtype=torch.int32, device="cuda"), freq)
    assert torch.equal(x, was)  # position 0 turns by nothing
