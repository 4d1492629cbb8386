"""Linear attention on the GPU: a decay of -inf clears the state whatever it held, in
every kernel (token by token, chunk by chunk, in segments).

From a clearing token on a sequence is as one that starts there without a state, so the
64-bit form of that tail is what is expected, with the bounds of test_gpu_lin_attn.
Rows before the poison keep the bits they have without it.
"""
import pytest
import torch

from tests import ops_reference as ref
from tests.test_gpu_lin_attn import D, make, run

pytestmark = pytest.mark.gpu

# (tokens, heads): token by token, one chunk, several, and cut in more and in few segments
SIZES = [(6, 2), (100, 2), (128, 1), (300, 2), (700, 2), (3000, 1), (512, 12)]


def decays(n, H, clears, seed):
    g = -0.02 * torch.rand(1, n, H, generator=torch.Generator().manual_seed(seed))
    for t in clears:
        g[0, t, 0] = -float("inf")
    return g


def check_tail(c, out, seq, start, end, clear, H):
    """Rows from `clear` on and the final state of head 0 of sequence `seq`, against the tail
    alone."""
    sl = slice(start + clear, end)
    o, S, mag, smag = ref.lin_attn(c["q"][0, sl, :1], c["k"][0, sl, :1], c["v"][0, sl, :1], c["g"][0, sl, :1],
                                   [end - start - clear], torch.zeros(1, 1, D, D, device="cuda"), [0], D ** -0.5)
    got = out[0, sl, :1].double()
    assert bool(torch.isfinite(got).all())
    err, lim = (got - o).abs(), 2.0 ** -8 * o.abs() + 2.0 ** -14 * mag + 1e-30
    assert bool((err <= lim).all()), float((err / lim).max())
    state = c["cache"][int(c["idx"][seq]), 0].double()
    err, lim = (state - S[0, 0]).abs(), 2.0 ** -17 * smag[0, 0] + 1e-30
    assert bool(torch.isfinite(state).all())
    assert bool((err <= lim).all()), float((err / lim).max())


def places(n):
    """Clearing tokens: the first, in the first chunk, at a chunk's start and end, the last."""
    return sorted({0, min(3, n - 1), n // 2, min(127, n - 1), min(128, n - 1), min(255, n - 1), n - 1})


@pytest.mark.parametrize("n,H", SIZES)
@pytest.mark.parametrize("held", ["nan", "inf"])
def test_a_state_that_is_not_finite_is_cleared(n, H, held):
    for clear in places(n):
        c, clean = (make([n, 5], H, seed=n, g=decays(n + 5, H, [clear], n), init=[1, 1]) for _ in range(2))
        c["cache"][int(c["idx"][0]), 0, 3:90] = float(held)
        out, good = run(c), run(clean)
        if clear:
            rows = out[0, :clear, 0, 3:90]
            assert not bool(torch.isfinite(rows).any())
        check_tail(c, out, 0, 0, n, clear, H)
        # value rows of the state that held numbers, the other heads and the other sequence
        assert torch.equal(out[0, :, 0, 90:], good[0, :, 0, 90:])
        assert torch.equal(out[0, :, 1:], good[0, :, 1:]) and torch.equal(out[0, n:], good[0, n:])
        assert torch.equal(c["cache"][int(c["idx"][1])], clean["cache"][int(clean["idx"][1])])


@pytest.mark.parametrize("n,H", SIZES)
@pytest.mark.parametrize("poison", ["v", "k", "q"])
def test_tokens_that_are_not_finite_are_cleared(n, H, poison):
    """Infinities and NaN in tokens before the clearing one."""
    for at, clear in {(0, 1), (0, n - 1), (n // 3, n // 2), (n // 2, n // 2 + 1), (n - 2, n - 1),
                      (min(100, n - 2), min(126, n - 1)), (min(100, n - 2), min(140, n - 1))}:
        if not at < clear < n:
            continue
        c, clean = (make([n, 5], H, seed=n + 1, g=decays(n + 5, H, [clear], n), init=[1, 1]) for _ in range(2))
        c[poison][0, at, 0, 17] = float("nan")
        c[poison][0, at, 0, 81] = float("inf")
        out, good = run(c), run(clean)
        rows = out[0, at:clear if poison != "q" else at + 1, 0]
        assert not bool(torch.isfinite(rows if poison != "v" else rows[:, [17, 81]]).any())
        if poison == "q":
            assert torch.equal(out[0, at + 1:clear, 0], good[0, at + 1:clear, 0])
        check_tail(c, out, 0, 0, n, clear, H)
        assert torch.equal(out[0, :at], good[0, :at]) and torch.equal(out[0, :, 1:], good[0, :, 1:])
        assert torch.equal(out[0, n:], good[0, n:])


@pytest.mark.parametrize("n,H", SIZES)
def test_what_follows_a_clear_stays(n, H):
    """A value that is not finite after a clearing token, or at it, reaches its column from
    its token to the next clearing one, and the state where there is none."""
    for clear, at in {(0, 0), (0, n // 2), (n // 3, n // 3), (n // 3, n - 1), (n - 1, n - 1)}:
        c, clean = (make([n], H, seed=n + 2, g=decays(n, H, [clear], n), init=[1]) for _ in range(2))
        c["v"][0, at, 0, 33] = -float("inf")
        out, good = run(c), run(clean)
        assert not bool(torch.isfinite(out[0, at:, 0, 33]).any())
        keep = torch.ones(out.shape, dtype=torch.bool, device="cuda")
        keep[0, at:, 0, 33] = False
        o, S = out[keep].double(), good[keep].double()
        # (one of the two may have taken the state in another order)
        assert bool(((o - S).abs() <= 2.0 ** -7 * S.abs() + 1e-3).all())
        state = c["cache"][int(c["idx"][0])]
        assert not bool(torch.isfinite(state[0, 33]).any())
        state[0, 33] = 0
        assert bool(torch.isfinite(state).all())


def test_clears_at_every_other_token():
    """As many clearing tokens as can be, over a state and tokens that are not finite."""
    n = 400
    c = make([n], 1, seed=9, g=decays(n, 1, range(1, n, 2), 9), init=[1])
    c["cache"][int(c["idx"][0])] = float("nan")
    for t in range(0, n - 2, 4):
        c["v"][0, t, 0, t % 128] = float("nan")
        c["k"][0, t, 0, t % 128] = float("inf")
    out = run(c)
    for t in range(1, n, 2):
        last = t + 1 == n
        rows = slice(t, t + 1 if (t + 1) % 4 == 0 or last else t + 2)
        o, _, mag, _ = ref.lin_attn(c["q"][0, rows], c["k"][0, rows], c["v"][0, rows], c["g"][0, rows],
                                    [rows.stop - t], torch.zeros(1, 1, D, D, device="cuda"), [0], D ** -0.5)
        err = (out[0, rows].double() - o).abs()
        assert bool((err <= 2.0 ** -8 * o.abs() + 2.0 ** -14 * mag + 1e-30).all()), t
    assert bool(torch.isfinite(c["cache"][int(c["idx"][0])]).all())
