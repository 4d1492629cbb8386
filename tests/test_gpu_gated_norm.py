"""The gated norm on the GPU against its definition in 64 bits.

Bounds, element by element: the sum of squares of D values in fp32, by lanes and
then a tree, is off by at most D 2^-24 relative (a lane adds at most D / 8 of
them, but rows off 16-byte boundaries may take one value a step); square root,
quotient, exp and the products add about 2^-20; the result is rounded to the
type."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def check(y, x, weight, gate, activation, eps):
    want = ref.gated_norm(x, weight, gate, activation, eps)
    rel = STEP[x.dtype] + 2.0 ** -20 + x.shape[-1] * 2.0 ** -25
    lim = rel * want.abs() + (2.0 ** -25 if x.dtype == torch.float16 else 1e-37)
    err = (y.double() - want).abs()
    assert bool((err <= lim).all()), float((err / lim).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [1, 7, 8, 64, 100, 128, 136, 256, 512, 1000, 8192])
def test_row_lengths(dtype, D):
    x, z = (torch.randn(1, 33, 3, D, device="cuda").to(dtype) for _ in range(2))
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    y = kda.gated_norm(x, w, gate=z, eps=1e-5)
    check(y[0], x[0], w, z[0], "sigmoid", 1e-5)


@pytest.mark.parametrize("activation", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_forms(activation, weight, gated):
    x, z = (3 * torch.randn(1, 70, 5, 128, device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(128, device="cuda") if weight else None
    y = kda.gated_norm(x, w, gate=z if gated else None, activation=activation)
    check(y[0], x[0], w, z[0] if gated else None, activation, 1e-6)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 12), (5, 3), (513, 12), (4097, 2)])
def test_sizes(T, H):
    x, z = (torch.randn(1, T, H, 128, device="cuda").bfloat16() for _ in range(2))
    y = kda.gated_norm(x, None, gate=z, activation="silu")
    check(y[0], x[0], None, z[0], "silu", 1e-6)


def test_views_and_in_place():
    xz = torch.randn(1, 40, 8, 128, device="cuda").bfloat16()
    x, z = xz[:, :, :4], xz[:, :, 4:]
    out = torch.empty(1, 40, 4, 128, device="cuda", dtype=torch.bfloat16)
    kda.gated_norm(x, None, gate=z, out=out)
    check(out[0], x[0], None, z[0], "sigmoid", 1e-6)
    y = x.contiguous()
    assert kda.gated_norm(y, None, gate=z, out=y) is y
    assert torch.equal(y, out)
    buf = torch.randn(40 * 260 + 1, device="cuda").bfloat16()
    odd = buf[1:].as_strided((40, 2, 128), (260, 129, 1))
    y = kda.gated_norm(odd, None)
    check(y, odd, None, None, "none", 1e-6)


def test_extremes():
    """Rows of zeros, of one large value, gates at both ends and non-finite rows that
    leave the others alone."""
    x = torch.randn(1, 6, 1, 128, device="cuda")
    z = torch.randn(1, 6, 1, 128, device="cuda")
    x[0, 0] = 0
    x[0, 1] = 0
    x[0, 1, 0, 5] = 1e15
    z[0, 2, 0, :64] = -float("inf")
    z[0, 2, 0, 64:] = float("inf")
    z[0, 3] = -1e4
    y = kda.gated_norm(x, None, gate=z, eps=1e-6)
    check(y[0], x[0], None, z[0], "sigmoid", 1e-6)
    s = kda.gated_norm(x, None, gate=z, activation="silu")
    assert bool((s[0, 2, 0, :64] == 0).all()) and bool((s[0, 3] == 0).all())
    x[0, 4, 0, 7] = float("nan")
    x[0, 5, 0, 7] = float("inf")
    t = kda.gated_norm(x, None, gate=z)
    assert torch.equal(t[0, :4], y[0, :4]) and bool(t[0, 4].isnan().all())
    assert bool(t[0, 5, 0, 7].isnan()) and float(t[0, 5].nansum()) == 0.0


def test_nothing():
    x = torch.empty(1, 0, 4, 128, device="cuda")
    assert kda.gated_norm(x, None).shape == x.shape
