"""A layer of the gated delta rule served with a paged state pool: prompts first, then one
token of every sequence a step.

    python examples/gated_delta_layer.py

Each call projects its tokens to q, k, v, a gate, the decay and the strength of the writes,
norms and turns q and k (``kda.qk_norm_rope``), runs the rule over the sequences' states
(``kda.gated_delta_fwd``), norms and gates its output (``kda.gated_norm``) and projects
back.  The example checks that a sequence fed token by token ends where the same sequence
fed at once does.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_prefill_gb300 as kda  # noqa: E402
from linear_attention_layer import difference, serve  # noqa: E402

D = 128


class GatedDeltaLayer:
    """Random weights; ``heads`` value heads, q and k shared by groups of them."""

    def __init__(self, hidden, heads, qk_heads, slots, *, state_dtype=torch.float32, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen) / cols ** 0.5).bfloat16().cuda()

        self.heads, self.qk_heads = heads, qk_heads
        self.w_in = weight(2 * (qk_heads + heads) * D, hidden)
        self.w_small = weight(2 * heads, hidden)
        self.w_out = weight(hidden, heads * D)
        self.q_weight, self.k_weight = ((1 + 0.1 * torch.randn(D, generator=gen)).cuda() for _ in "qk")
        self.norm_weight = torch.ones(D, device="cuda")
        # head h forgets at the rate of 2^{-8 (h + 1) / H} a token where its input says nothing
        self.rate = torch.exp2(-8.0 * torch.arange(1, heads + 1) / heads).cuda()
        self.inv_freq, self.factor = kda.rope_frequencies(D)
        self.pool = torch.zeros(slots, heads, D, D, dtype=state_dtype, device="cuda")

    def gates(self, small):
        """small [T, 2 H] to the log decay, at most zero, and the strength, 0 to 1."""
        a, b = small.float().chunk(2, 1)
        return (-self.rate * torch.exp(a))[None], torch.sigmoid(b)[None].contiguous()

    def mix(self, proj, small, positions, bounds, slots, has_state, workspace=None):
        """The part between the projections: proj [T, 2 (Hqk + H) 128] (q and k are normed and
        turned in place) to [1, T, H, 128].  ``bounds`` is a host tensor [N + 1]."""
        q, k, v, z = proj.view(1, len(proj), -1, D).split(
            [self.qk_heads, self.qk_heads, self.heads, self.heads], 2)
        kda.qk_norm_rope(q, k, self.q_weight, self.k_weight, positions, self.inv_freq, factor=self.factor)
        decay, strength = self.gates(small)
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        kda.gated_delta_fwd(q, k, v, decay, strength, bounds.cuda(), state_cache=self.pool,
                            state_indices=slots, has_initial_state=has_state, out=out,
                            cu_seqlens_cpu=bounds, workspace=workspace)
        return kda.gated_norm(out, self.norm_weight, gate=z, activation="silu", out=out)

    def __call__(self, x, positions, bounds, slots, has_state):
        y = self.mix(x @ self.w_in.t(), x @ self.w_small.t(), positions, bounds, slots, has_state)
        return y.view(len(x), -1) @ self.w_out.t()


def main(hidden=1536, heads=12, qk_heads=4, lengths=(1500, 1, 40, 700), steps=12):
    gen = torch.Generator().manual_seed(1)
    x = [torch.randn(m + steps, hidden, generator=gen).bfloat16().cuda() for m in lengths]
    layer = GatedDeltaLayer(hidden, heads, qk_heads, len(lengths))
    by_token = serve(layer, x, list(lengths), steps)
    states = layer.pool.clone()
    at_once = serve(layer, x, [m + steps for m in lengths], 0)
    worst = max(difference(a, b) for a, b in zip(by_token, at_once))
    state = difference(states, layer.pool)
    print(f"{len(lengths)} prompts of {sum(lengths)} tokens and {steps} steps: outputs within "
          f"{worst:.1e}, states within {state:.1e} of the same tokens at once")
    return worst, state


if __name__ == "__main__":
    main()
