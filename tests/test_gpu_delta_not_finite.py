"""The gated delta rule on the GPU where one entry of a state, or a row's length, is not finite
and a token clears the state soon after.  Bounds as in test_gpu_gated_delta.py; what a token
behind the clearing one gives does not depend on what the state held, so it keeps the relative
bound as well."""
import pytest
import torch

from tests.test_gpu_gated_delta import D, check, expected, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool", [torch.float32, torch.float16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("silent", [False, True])
@pytest.mark.parametrize("n,clear", [(200, 10), (17, 12), (100, 40), (4500, 25)])
def test_one_entry_beside_large_ones_and_an_early_clear(n, clear, silent, bad, pool):
    """A state's rows with finite entries of 1e4 around the bad one; v is zero up to the clearing
    token, or not."""
    H, row, key = 1, 37, 70
    g = torch.full((1, n, H), -0.01)
    g[:, clear] = -torch.inf
    c = make([n], H, seed=60, g=g, init=[True], state=1e4, pool=pool)
    if silent:
        c["v"][:, :clear] = 0
    want = expected(c)
    slot = int(c["idx"][0])
    c["cache"][slot, 0, row, key] = bad
    before = c["storage"].clone()
    out = run(c)[0].double()
    torch.cuda.synchronize()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:clear, 0, row] = True
    assert not torch.isfinite(out[hit]).any()
    err, lim = (out - want[0]).abs(), 2.0 ** -8 * want[0].abs() + 2.0 ** -9 * want[2] + 1e-30
    assert bool((err <= lim)[~hit].all())
    assert float(err[clear:].norm() / want[0][clear:].norm()) <= 2.5e-3
    got, S = c["cache"][slot].double(), want[1][0]
    step = 2.0 ** -11 if pool == torch.float16 else 0.0
    assert bool(((got - S).norm(dim=-1) <= step * S.norm(dim=-1) + 2.0 ** -17 * want[3][0] + D ** 0.5 * 2.0 ** -25).all())
    keep = torch.ones(len(before), dtype=torch.bool, device="cuda")
    keep[slot] = False
    bits = torch.int16 if pool == torch.float16 else torch.int32
    assert torch.equal(c["storage"][keep].view(bits), before[keep].view(bits))


@pytest.mark.parametrize("n", [1, 8, 16, 17, 200])
@pytest.mark.parametrize("where", ["q", "k"])
def test_finite_rows_whose_squares_are_not(n, where):
    """Entries of 1e20: |q|^2 and |k|^2 are infinite in fp32, so such a row counts as one that is
    not finite, however long its sequence."""
    t, clear = n // 2, n - 1
    g = torch.full((1, 2 * n, 2), -0.1)
    if n > 4:
        g[:, clear] = g[:, n + clear] = -torch.inf
    c = make([n, n], 2, seed=61, g=g, init=[True, True])
    want, before = expected(c), c["storage"].clone()
    c[where][0, t, 0] = 1e20 * torch.sign(c[where][0, t, 0])
    assert bool(torch.isfinite(c[where]).all())
    out = run(c)[0].double()
    torch.cuda.synchronize()
    hit = torch.zeros_like(out, dtype=torch.bool)
    if where == "q":
        hit[t, 0] = True
    else:
        hit[t:clear if n > 4 else n, 0] = True
    assert torch.isnan(out[hit]).all()
    err, lim = (out - want[0]).abs(), 2.0 ** -8 * want[0].abs() + 2.0 ** -9 * want[2] + 1e-30
    assert bool((err <= lim)[~hit].all())
    if where == "q" or n > 4:
        check(c, torch.where(hit, want[0], out)[None], want, before)
    else:
        got = c["cache"][c["idx"].long().cuda()]
        assert torch.isnan(got[0, 0]).all() and torch.isfinite(got[1]).all() and torch.isfinite(got[0, 1]).all()
