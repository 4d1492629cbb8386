"""Plain 64-bit forms of the operators beside the KDA forward, from their
definitions, and the magnitudes their error bounds are made of."""
from __future__ import annotations

import torch


def lin_attn(q, k, v, g, lengths, state, has_init, scale):
    """Token by token: (out [T, H, V], final [N, H, V, K]) in fp64 on the inputs'
    device, and the same sums over absolute values (what rounding errors of the
    terms are bounded by).  q, k [T, Hqk, K], v [T, H, V], g [H] or [T, H], state
    [N, H, V, K]."""
    T, H = v.shape[0], v.shape[1]
    rep = H // q.shape[1]
    q = q.double().repeat_interleave(rep, 1)
    k = k.double().repeat_interleave(rep, 1)
    v = v.double()
    d = torch.exp(g.double()).expand(T, H)
    out, mag = torch.zeros_like(v), torch.zeros_like(v)
    fin = torch.zeros_like(state, dtype=torch.float64)
    fmag = torch.zeros_like(fin)
    t = 0
    for n, ln in enumerate(lengths):
        S = state[n].double() if bool(has_init[n]) else torch.zeros_like(fin[n])
        A = S.abs()
        for _ in range(int(ln)):
            w = d[t][:, None, None]
            S = torch.where(w == 0, 0.0, w * S) + v[t][:, :, None] * k[t][:, None, :]
            A = w * A + (v[t][:, :, None] * k[t][:, None, :]).abs()
            out[t] = scale * (S * q[t][:, None, :]).sum(-1)
            mag[t] = abs(scale) * (A * q[t][:, None, :].abs()).sum(-1)
            t += 1
        fin[n], fmag[n] = S, A
    return out, fin, mag, fmag


def rope(x, positions, inv_freq, layout, factor, inverse=False):
    """x [T, H, D] turned, fp64."""
    y = x.double().clone()
    r = 2 * inv_freq.numel()
    a = positions.double()[:, None] * inv_freq.double() * (-1.0 if inverse else 1.0)
    c, s = factor * torch.cos(a)[:, None], factor * torch.sin(a)[:, None]
    i = torch.arange(r // 2, device=x.device)
    one, two = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
    x1, x2 = x.double()[..., one], x.double()[..., two]
    y[..., one] = x1 * c - x2 * s
    y[..., two] = x2 * c + x1 * s
    return y


def gated_norm(x, weight, gate, activation, eps):
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    if gate is not None:
        z = gate.double()
        if activation == "sigmoid":
            y = y * torch.sigmoid(z)
        elif activation == "silu":
            y = y * torch.where(z == -torch.inf, 0.0, z * torch.sigmoid(z))
        else:
            y = y * z
    return y
