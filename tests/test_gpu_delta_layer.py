"""The norms with rotary positions, the gated delta rule and the gated norm one after the other
on the GPU, as the example runs them: prompts and then single tokens over one state pool,
against 64 bits.

Bounds, in relative L2.  The 64-bit form rounds q and k to bf16 where the layer does; 32-bit
sums are off by 2^-20 or so, so about one value in 2^10 rounds the other way, by 2^-7 at most:
2^-12 in L2, which the rule, whose tokens' factors have norm at most one, carries to its
states and outputs as any error of a key: at most a few times 2^-12 / (1 - decay)^1/2, well
below 2^-8.  The attention's output is rounded to bf16, at most 2^-8 of each value, and the norm,
which divides by what it was given, passes that on at most twice; its own output is rounded once
more.  Together below 4 * 2^-8.  Fed token by token or at once, q, k, decay and strength are
the same bits: outputs differ by their roundings, at most 3 * 2^-8, and fp32 states by twice the
operators' own bound, 2^-17 of what the tokens wrote, which is below 8 |S| here: 2^-13.
"""
import os
import sys

import pytest
import torch

from tests import delta_reference as ref
from tests import ops_reference

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_delta_layer as example  # noqa: E402

pytestmark = pytest.mark.gpu
D = 128


def test_example():
    out, state = example.main()
    # the projections are library products of other shapes, which round a few of their values
    # the other way: q, k, v, gate, strength, decay and the layer's output by at most 2^-8 each
    assert out < 8 * 2.0 ** -8 and state < 4 * 2.0 ** -8


@pytest.mark.parametrize("state_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads, qk_heads", [(3, 3), (6, 2)])
def test_between_the_projections(heads, qk_heads, state_dtype):
    lengths, steps = [530, 1, 9, 128], 5
    layer = example.GatedDeltaLayer(64, heads, qk_heads, len(lengths), state_dtype=state_dtype)
    gen = torch.Generator().manual_seed(3)
    width = 2 * (qk_heads + heads) * D
    proj = [torch.randn(m + steps, width, generator=gen).bfloat16().cuda() for m in lengths]
    small = [torch.randn(m + steps, 2 * heads, generator=gen).bfloat16().cuda() for m in lengths]
    n = len(lengths)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    fresh, kept = (torch.full((n,), s, dtype=torch.bool, device="cuda") for s in (False, True))

    def prompts(ms):
        bounds = torch.tensor([0] + ms).cumsum(0).to(torch.int32)
        y = layer.mix(*(torch.cat([x[i][:m] for i, m in enumerate(ms)]) for x in (proj, small)),
                      torch.cat([torch.arange(m) for m in ms]).cuda(), bounds, slots, fresh)
        return list(y[0].split(ms))

    by_token = prompts(lengths)
    for s in range(steps):
        y = layer.mix(*(torch.stack([x[i][m + s] for i, m in enumerate(lengths)]) for x in (proj, small)),
                      torch.tensor([m + s for m in lengths]).cuda(),
                      torch.arange(n + 1, dtype=torch.int32), slots, kept)[0]
        by_token = [torch.cat([o, y[i:i + 1]]) for i, o in enumerate(by_token)]
    states = layer.pool.clone()
    at_once = prompts([m + steps for m in lengths])
    exact = state_dtype == torch.float32
    round_pool = 0.0 if exact else (steps + 1) * 2.0 ** -8
    for i, m in enumerate(lengths):
        m += steps
        q, k, v, z = proj[i].view(m, -1, D).split([qk_heads, qk_heads, heads, heads], 1)
        pos = torch.arange(m).cuda()
        q, k = (ref.qk_norm_rope(x, w, pos, layer.inv_freq, "half", layer.factor, 1e-6).bfloat16()
                for x, w in ((q, layer.q_weight), (k, layer.k_weight)))
        g, beta = layer.gates(small[i])
        zero = torch.zeros(1, heads, D, D, device="cuda")
        o, S = ref.gated_delta(q, k, v, g[0], beta[0], [m], zero, torch.tensor([False]), D ** -0.5)[:2]
        y = ops_reference.gated_norm(o, layer.norm_weight, z, "silu", 1e-6)
        assert example.difference(by_token[i], y) < 4 * 2.0 ** -8 + 2 * round_pool
        assert example.difference(at_once[i], y) < 4 * 2.0 ** -8
        assert example.difference(by_token[i], at_once[i]) < 3 * 2.0 ** -8 + 2 * round_pool
        assert example.difference(states[i], S[0]) < 2.0 ** -8 + round_pool
        assert example.difference(states[i], layer.pool[i]) < (2.0 ** -13 if exact else 2 * round_pool)
