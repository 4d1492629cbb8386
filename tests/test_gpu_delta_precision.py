"""How well the gated delta rule's chunked outputs keep what is left of a large state.

Bounds.  The states' bound of test_gpu_gated_delta.py, 2^-17 E with E what a value row's tokens
wrote (undecayed for 64 tokens), says what operands of 22 bits leave; an output is S q with
|q| <= 1, so the same products once more: 2^-16 E scale, and its rounding to bf16, 2^-8 |o|.  Over a
tensor the rounding gives up to 1.7e-3, and the states' mean 2^-19 for each unit of E / |o|:
with values `ratio` times those that are read, and E of at most twice the largest, below
1.7e-3 + ratio 2^-18: 2.1e-3 at 100."""
import pytest
import torch

from tests.test_gpu_gated_delta import D, expected, make, run

pytestmark = pytest.mark.gpu


def compare(c, rows=slice(None), most=None):
    o, _, emag, _ = expected(c)
    out = run(c)[0].double()
    err = (out - o).abs()
    lim = 2.0 ** -8 * o.abs() + 2.0 ** -16 * emag + 1e-30
    assert bool((err <= lim).all()), float((err / lim).max())
    rel = float(err[rows].norm() / o[rows].norm())
    if most is not None:
        assert rel <= most, rel


@pytest.mark.parametrize("ratio", [1.0, 10.0, 100.0, 1000.0])
@pytest.mark.parametrize("n,old,new", [(17, 2, 9), (64, 3, 30), (200, 60, 70), (200, 5, 150), (4500, 40, 2000)])
def test_old_values_overwritten_by_smaller_ones(n, old, new, ratio):
    """One key holds a large value, then a small one, and is read: the two terms of an output,
    the state's and the chunk's, cancel."""
    c = make([n], 1, seed=70, init=[False], g=torch.zeros(1, n, 1), beta=torch.zeros(1, n, 1))
    c["beta"][:, [old, new]] = 1.0
    c["k"][0, new] = c["k"][0, old]
    c["q"][0, new:] = c["k"][0, old]
    c["v"][0, old] *= ratio
    compare(c, slice(new, None), 2.5e-3 if ratio <= 100 else None)


@pytest.mark.parametrize("ratio", [10.0, 100.0])
@pytest.mark.parametrize("n", [150, 4500])
def test_states_overwritten_by_smaller_values(n, ratio):
    """The same of 64 keys at right angles, overwritten one after the other: at its token each output is
    the value just written, the difference of terms `ratio` times as large.  Its row of the state has
    one entry for each key, so the 22 bits of that entry alone count: 2^-22 ratio of the output."""
    c = make([n], 1, seed=71, init=[False], g=torch.zeros(1, n, 1), beta=torch.ones(1, n, 1))
    keys = torch.zeros(n, D)
    keys[torch.arange(n), torch.arange(n) * 5 % 64] = 1.0
    c["k"][0, :, 0] = keys.bfloat16().cuda()
    c["q"][0, :, 0] = keys.bfloat16().cuda()
    c["v"][0, :64] *= ratio
    compare(c, slice(64, None), 2.5e-3)


@pytest.mark.parametrize("rate,upto", [(0.3, 64), (0.4, 48)])
@pytest.mark.parametrize("n", [64, 100])
def test_one_write_and_a_decaying_state(n, rate, upto):
    """Reads of a value written once, at each token that it fades over: P's entries and their row's
    power of two, at most 2^15, are then down to 2^-12 (2^-27 2^15), which two fp16 keep to 2^-25: 2^-13
    of an output, beside its own rounding."""
    c = make([n], 2, seed=72, init=[False], g=torch.full((1, n, 2), -rate), beta=torch.zeros(1, n, 2))
    c["beta"][:, 0] = 1.0
    c["q"][0, :] = c["k"][0, :1]
    o = expected(c)[0]
    out = run(c)[0].double()
    for t in range(upto):
        assert float((out[t] - o[t]).norm() / o[t].norm()) <= 2.5e-3, t
    compare(c)


def test_keys_of_entries_of_many_magnitudes():
    """Entries far below their row's length lose bits where rows are scaled to fp16 (at most 2^-24 of
    the length)."""
    n = 300
    c = make([n], 2, seed=73, init=[True], g=torch.full((1, n, 2), -0.05))
    spread = torch.exp2(-(torch.arange(D) % 31).float())
    c["k"] = (c["k"].float() * spread.cuda()).bfloat16()
    c["q"] = (c["q"].float() * spread.flip(0).cuda()).bfloat16()
    compare(c, most=2.5e-3)
    c["k"][:, :, :, 1:] *= 1e-6
    compare(c, most=2.5e-3)


@pytest.mark.parametrize("n", [17, 64, 300])
@pytest.mark.parametrize("big", [1e2, 1e4, 1e6])
def test_small_states_in_the_chunk_of_large_values(n, big):
    """A value row has one scale in a chunk, made from a bound that is at most 2^10 too large, and
    terms are kept to 2^-39 of it: 2^-29 of the most that the chunk writes for each of an output's 128
    terms, whose factors, of a vector no longer than one, add up to less than 2^4."""
    c = make([n], 2, seed=74, init=[True], g=torch.full((1, n, 2), -0.01), state=1e-4)
    late = n // 2
    c["v"][:, :late] *= 1e-4
    c["v"][:, late:] *= big
    o, S, emag, smag = expected(c)
    out = run(c)[0].double()
    most = torch.zeros_like(emag)
    for a in range(0, n, 64):
        most[a:a + 64] = emag[a:a + 64].amax(0, keepdim=True)
    lim = 2.0 ** -8 * o.abs() + 2.0 ** -16 * emag + 2.0 ** -25 * most
    assert bool(((out - o).abs() <= lim).all()), float(((out - o).abs() / lim).max())
