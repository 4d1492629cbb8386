"""Plain 64-bit forms of the gated delta rule and of the norms of queries and keys with the
rotary positions, from their definitions, and the magnitudes their error bounds are made of."""
from __future__ import annotations

import torch

WINDOW = 64  # tokens within which the bounds count no decay


def gated_delta(q, k, v, g, beta, lengths, state, has_init, scale):
    """Token by token, all sequences at once: (out [T, H, V], final [N, H, V, K]) in fp64,
    and (emag [T, H, V], fmag [N, H, V]): for each value row the sum over the tokens so far
    of |beta (v - e^g S k)|, each with the decays that lie more than WINDOW tokens behind
    it, and of the initial state's length.

    q, k [T, Hqk, K], v [T, H, V], g [H] or [T, H], beta [T, H], state [N, H, V, K]."""
    T, H = v.shape[0], v.shape[1]
    rep = H // q.shape[1]

    def unit(x):
        x = x.double()
        return (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(rep, 1)

    q, k, v, b = unit(q), unit(k), v.double(), beta.double()
    d = torch.exp(g.double()).expand(T, H)
    lens = [int(x) for x in lengths]
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    start = torch.zeros(len(lens) + 1, dtype=torch.long)
    start[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.long), 0)
    start = start[:-1][order].to(v.device)
    S = torch.stack([state[n].double() if bool(has_init[n]) else torch.zeros_like(state[n], dtype=torch.float64)
                     for n in order]) if lens else state.double()[:0]
    out, emag = torch.zeros_like(v), torch.zeros_like(v)
    E = S.norm(dim=-1)          # [N, H, V], of all but the last WINDOW tokens
    recent = torch.zeros_like(E)  # the sum of those
    window = []                 # and their decays and terms
    for t in range(max(lens, default=0)):
        n = sum(1 for a in lens if a > t)
        at = start[:n] + t
        w = d[at][..., None, None]
        old = torch.where(w == 0, 0.0, w * S[:n])
        new = b[at][..., None] * (v[at] - (old @ k[at][..., None])[..., 0])
        S[:n] = old + new[..., :, None] * k[at][..., None, :]
        out[at] = scale * (S[:n] @ q[at][..., None])[..., 0]
        window.append((d[at][..., None], new.abs()))
        recent[:n] += new.abs()
        if len(window) > WINDOW:
            decay, term = window.pop(0)
            E[:n] = E[:n] * decay[:n] + term[:n]
            recent[:n] = (recent[:n] - term[:n]).clamp(min=0)
        emag[at] = abs(scale) * (E[:n] + recent[:n])
    back = torch.tensor([order.index(n) for n in range(len(lens))], dtype=torch.long, device=v.device)
    return out, S[back], emag, (E + recent)[back]


def qk_norm_rope(x, weight, positions, inv_freq, layout, factor, eps):
    """x [T, H, D] normed, weighted and turned, fp64."""
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    r = 2 * inv_freq.numel()
    a = positions.double()[:, None] * inv_freq.double()
    c, s = factor * torch.cos(a)[:, None], factor * torch.sin(a)[:, None]
    i = torch.arange(r // 2, device=x.device)
    one, two = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
    z = y.clone()
    z[..., one] = y[..., one] * c - y[..., two] * s
    z[..., two] = y[..., two] * c + y[..., one] * s
    return z
