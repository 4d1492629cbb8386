"""Linear attention on the GPU: decays of scores behind strong ones in the same chunk.

Each value column holds two tokens of opposite sign, a few tokens apart with slow
decays between them, so that the output is the small difference of two terms and the
bounds of test_gpu_lin_attn, 2^-8 |o| + 2^-14 A, show the terms' own errors: strong
decays earlier in the chunk may not take bits from the weak ones behind them.
"""
import pytest
import torch

from tests.test_gpu_lin_attn import D, make, run_and_check

pytestmark = pytest.mark.gpu

INF = float("inf")
# decays in the order of the tokens: (tokens, log decay), repeated to the length
PATTERNS = {
    "96 cleared": [(96, -INF), (32, -0.01)],
    "64 cleared": [(64, -INF), (64, -0.003)],
    "8 cleared in a block": [(8, -INF), (24, -0.02)],
    "every third cleared": [(1, -INF), (2, -0.05)],
    "64 of -20": [(64, -20.0), (64, -0.01)],
    "16 of -20 in a block": [(16, -20.0), (16, -0.01)],
    "40 of -50": [(40, -50.0), (88, -0.004)],
    "ramp": [(8, -60.0), (8, -6.0), (8, -0.6), (104, -0.006)],
}


@pytest.mark.parametrize("name", sorted(PATTERNS))
@pytest.mark.parametrize("n", [128, 300, 1400])
def test_weak_decays_behind_strong_ones(n, name):
    g, t = torch.empty(n), 0
    while t < n:
        for m, value in PATTERNS[name]:
            g[t:t + m] = value
            t += m
    c = make([n], 2, seed=n, g=g[None, :, None].expand(1, n, 2).contiguous(), init=[1])
    gen = torch.Generator().manual_seed(n + 1)
    v = torch.zeros(1, n, 2, D)
    for col in range(D):
        # every 16 tokens: tokens a and b, 1 to 9 apart
        for base in range(0, n, 16):
            a = base + int(torch.randint(0, 16, (1,), generator=gen))
            b = a + int(torch.randint(1, 10, (1,), generator=gen))
            if b < n:
                v[0, a, :, col] += 1.0
                v[0, b, :, col] -= 1.0
    c["v"] = v.bfloat16().cuda()
    # alike in every token, so that a pair's scores cancel but for their decays
    c["k"][:] = c["k"][:, :1]
    run_and_check(c)
