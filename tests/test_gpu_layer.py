"""The linear-attention layer's operators one after the other on the GPU, as the example
runs them: prompts and then single tokens over one state pool, against 64 bits.

Bounds, in relative L2.  Between the projections q, k, the attention's output and the
normed output are rounded to bf16, each by at most 2^-8 of a value; the norm divides by
what it was given, so an error of its input is passed on at most twice.  Together below
6 * 2^-8; the states take the roundings of k alone, 2^-8.  Fed token by token or at
once, q and k are the same bits: only the two outputs' roundings and the operators' own
bounds (2^-14 of the sums of absolute terms, far below) are left, 3 * 2^-8.
"""
import os
import sys

import pytest
import torch

from tests import ops_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import linear_attention_layer as example  # noqa: E402

pytestmark = pytest.mark.gpu
D = 128


def test_example():
    out, state = example.main()
    # the projections are library products of other shapes: one more rounding of each
    # of q, k, v, gate and the layer's output
    assert out < 8 * 2.0 ** -8 and state < 3 * 2.0 ** -8


@pytest.mark.parametrize("state_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads, qk_heads", [(3, 3), (6, 2)])
def test_between_the_projections(heads, qk_heads, state_dtype):
    lengths, steps = [530, 1, 9, 128], 5
    layer = example.LinearAttentionLayer(64, heads, qk_heads, len(lengths), state_dtype=state_dtype)
    gen = torch.Generator().manual_seed(3)
    width = 2 * (qk_heads + heads) * D
    proj = [torch.randn(m + steps, width, generator=gen).bfloat16().cuda() for m in lengths]
    n = len(lengths)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    fresh, kept = (torch.full((n,), s, dtype=torch.bool, device="cuda") for s in (False, True))

    def prompts(ms):
        bounds = torch.tensor([0] + ms).cumsum(0).to(torch.int32)
        y = layer.mix(torch.cat([proj[i][:m] for i, m in enumerate(ms)]),
                      torch.cat([torch.arange(m) for m in ms]).cuda(), bounds, slots, fresh)
        return list(y[0].split(ms))

    by_token = prompts(lengths)
    for s in range(steps):
        y = layer.mix(torch.stack([proj[i][m + s] for i, m in enumerate(lengths)]),
                      torch.tensor([m + s for m in lengths]).cuda(),
                      torch.arange(n + 1, dtype=torch.int32), slots, kept)[0]
        by_token = [torch.cat([o, y[i:i + 1]]) for i, o in enumerate(by_token)]
    states = layer.pool.clone()
    at_once = prompts([m + steps for m in lengths])
    round_pool = 0.0 if state_dtype == torch.float32 else (steps + 1) * 2.0 ** -8
    for i, m in enumerate(lengths):
        m += steps
        q, k, v, z = proj[i].view(m, -1, D).split([qk_heads, qk_heads, heads, heads], 1)
        pos = torch.arange(m).cuda()
        q, k = (ref.rope(x, pos, layer.inv_freq, "half", layer.factor) for x in (q, k))
        zero = torch.zeros(1, heads, D, D, device="cuda")
        o, S = ref.lin_attn(q, k, v, layer.log_decay, [m], zero, torch.tensor([False]), D ** -0.5)[:2]
        y = ref.gated_norm(o, layer.norm_weight, z, "sigmoid", 1e-6)
        assert example.difference(by_token[i], y) < 6 * 2.0 ** -8 + 2 * round_pool
        assert example.difference(at_once[i], y) < 6 * 2.0 ** -8
        assert example.difference(by_token[i], at_once[i]) < 3 * 2.0 ** -8 + 2 * round_pool
        assert example.difference(states[i], S[0]) < 2.0 ** -8 + round_pool
        assert example.difference(layer.pool[i], S[0]) < 2.0 ** -8 + round_pool


def test_memory_made_by_a_call_belongs_to_its_stream(monkeypatch):
    """Workspace and output that a call makes for itself come from the pool of the stream
    it runs on, so that they are not given out again while it runs."""
    s = torch.cuda.Stream()
    made, empty = [], torch.empty

    def spy(*args, **kw):
        made.append(torch.cuda.current_stream())
        return empty(*args, **kw)

    q = torch.randn(1, 5, 2, D, device="cuda").bfloat16()
    pool = torch.zeros(1, 2, D, D, device="cuda")
    cu, idx = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 5], [0]))
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", spy)
    example.kda.lin_attn_fwd(q, q, q, -torch.ones(2, device="cuda"), cu, state_cache=pool, state_indices=idx,
                             has_initial_state=idx.bool(), out=out,
                             cu_seqlens_cpu=torch.tensor([0, 5], dtype=torch.int32), stream=s)
    example.kda.gated_norm(q, stream=s)
    assert made == [s, s]
    example.kda.gated_norm(q)
    assert made[2:] == [torch.cuda.current_stream()]
    monkeypatch.undo()
    torch.cuda.synchronize()
