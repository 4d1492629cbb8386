"""The operators of a linear-attention layer with a decay for each head, as cases to be
measured: rotary positions on q and k, the attention itself (packed prompts and single
tokens over a paged pool of states), and the gated norm of its output.

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is set,
by the calls a user makes of this package.
"""
import math
import random

import torch

own = False

D = 128     # head size of q, k and v
CHUNK = 64  # tokens per chunk of the plain form of the attention
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _lin(name, *, ones=0, seqs=0, lo=1, hi=1, empty=0.0, heads=12, qk_heads=12, decay="head",
         pool="fp32", fused=False, init=0.5, lens_seed=0):
    c = dict(op="lin_attn", ones=ones, seqs=seqs, lo=lo, hi=hi, empty=empty, heads=heads,
             qk_heads=qk_heads, decay=decay, pool=pool, fused=fused, init=init,
             lens_seed=lens_seed)
    return dict(c, name=name) if name else c


def _rope(name, *, tokens, heads=12, k_heads=12, dim=D, rot=D, layout="half", scaled=False,
          far=0, dtype="bf16"):
    c = dict(op="rope", tokens=tokens, heads=heads, k_heads=k_heads, dim=dim, rot=rot,
             layout=layout, scaled=scaled, far=far, dtype=dtype)
    return dict(c, name=name) if name else c


def _norm(name, *, tokens, heads=12, dim=D, gate="sigmoid", dtype="bf16"):
    c = dict(op="gated_norm", tokens=tokens, heads=heads, dim=dim, gate=gate, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request answering: the latency of a single token
        _lin("lin_step_1", ones=1, init=1.0),
        # a full decode batch, one token for each of 512 requests
        _lin("lin_step_512", ones=512, init=1.0),
        # one prompt, one token over a round length
        _lin("lin_prompt_4097", seqs=1, lo=4097, hi=4097, init=1.0),
        # one long prompt
        _lin("lin_prompt_16384", seqs=1, lo=16384, hi=16384, init=0.0),
        # the same on a shard with few heads, decays of each token
        _lin("lin_prompt_16384_h2", seqs=1, lo=16384, hi=16384, heads=2, qk_heads=2,
             decay="token", init=0.0),
        # a prompt batch of ragged requests, q and k heads shared by groups of three v heads,
        # all three views of one projection's output
        _lin("lin_varlen_128", seqs=128, lo=1, hi=2048, empty=0.05, qk_heads=4, decay="token",
             fused=True, lens_seed=3),
        # decode and prompts in one batch, 2-byte states
        _lin("lin_mixed", ones=512, seqs=4, lo=2048, hi=2048, pool="bf16", lens_seed=4),
        # a decode batch deep in long contexts
        _rope("rope_step_512", tokens=512, scaled=True, far=131072),
        # a long prompt, half of each head rotated
        _rope("rope_prompt_16384", tokens=16384, rot=64, layout="interleaved"),
        # the decode batch's outputs
        _norm("norm_step_512", tokens=512),
        # the long prompt's outputs
        _norm("norm_prompt_16384", tokens=16384),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "prompt", "batch", "mixed", "rope", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "rope":
        dim = rng.choice([64, 128, 192])
        rot = rng.choice([dim, dim // 2])
        return _rope(None, tokens=_log_int(rng, 1, 16384), heads=rng.randint(1, 12),
                     k_heads=rng.randint(1, 12), dim=dim, rot=rot,
                     layout=rng.choice(["half", "interleaved"]), scaled=rng.random() < 0.5,
                     far=rng.choice([0, _log_int(rng, 4096, 131072)]), dtype=dtype)
    if kind == "norm":
        return _norm(None, tokens=_log_int(rng, 1, 16384), heads=rng.randint(1, 12),
                     dim=rng.choice([64, 128, 256]), gate=rng.choice(["sigmoid", "silu"]),
                     dtype=dtype)
    groups, per = rng.choice([1, 2, 4]), rng.choice([1, 2, 3])
    kw = dict(heads=groups * per, qk_heads=groups, decay=rng.choice(["head", "token"]),
              pool=rng.choice(["fp32", "fp32", "bf16", "fp16"]), fused=rng.random() < 0.5,
              init=rng.choice([0.0, 0.5, 1.0]), lens_seed=rng.randrange(1 << 20))
    if kind == "step":
        return _lin(None, ones=_log_int(rng, 1, 512), **kw)
    if kind == "prompt":
        n = _log_int(rng, 2, 16384)
        return _lin(None, seqs=1, lo=n, hi=n, **kw)
    if kind == "batch":
        return _lin(None, seqs=_log_int(rng, 2, 96), lo=1, hi=_log_int(rng, 9, 2048), empty=0.05,
                    **kw)
    hi = _log_int(rng, 64, 2048)
    return _lin(None, ones=_log_int(rng, 1, 512), seqs=rng.randint(1, 8), lo=max(1, hi // 2),
                hi=hi, **kw)


def _lengths(case):
    r = random.Random(case["lens_seed"])
    lens = [1] * case["ones"]
    for _ in range(case["seqs"]):
        n = r.randint(case["lo"], case["hi"])
        lens.append(0 if r.random() < case["empty"] else n)
    return lens


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _inv_freq(case):
    """Frequencies of the rotated pairs and the factor on cos and sin: base 10000, or the same
    stretched 8 times from 16384 positions, fast pairs kept and slow ones divided, with a linear
    ramp between those that turn 32 times and once in 16384 positions."""
    r, base = case["rot"], 10000.0
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if not case["scaled"]:
        return f, 1.0
    span, factor = 16384.0, 8.0

    def dim_of(turns):
        return r * math.log(span / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), r - 1)
    keep = [1.0 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(r // 2)]
    return [x * (w + (1 - w) / factor) for x, w in zip(f, keep)], 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev).to(dtype)

    if case["op"] == "rope":
        T, H, Hk, dim = case["tokens"], case["heads"], case["k_heads"], case["dim"]
        dt = DTYPES[case["dtype"]]
        q, k = normal(1, T, H, dim, dtype=dt), normal(1, T, Hk, dim, dtype=dt)
        if case["far"]:  # requests at their own places
            pos = torch.randint(0, case["far"], (T,), generator=gen, device=dev)
        else:            # one prompt from its start
            pos = torch.arange(T, device=dev)
        freq, factor = _inv_freq(case)
        return dict(case=case, q=q, k=k, pos=pos.to(torch.int32), factor=factor,
                    inv_freq=torch.tensor(freq, dtype=torch.float64, device=dev),
                    q_out=torch.empty_like(q), k_out=torch.empty_like(k))

    if case["op"] == "gated_norm":
        T, H, dim = case["tokens"], case["heads"], case["dim"]
        dt = DTYPES[case["dtype"]]
        x = normal(1, T, H, dim, dtype=dt)
        return dict(case=case, x=x, gate=normal(1, T, H, dim, dtype=dt),
                    weight=1.0 + 0.1 * normal(dim, dtype=torch.float32),
                    out=torch.empty_like(x), eps=1e-5)

    lens = _lengths(case)
    N, T, H, Hk = len(lens), sum(lens), case["heads"], case["qk_heads"]
    if case["fused"]:
        qkv = normal(1, T, 2 * Hk + H, D)
        q, k, v = qkv[:, :, :Hk], qkv[:, :, Hk:2 * Hk], qkv[:, :, 2 * Hk:]
    else:
        q, k, v = normal(1, T, Hk, D), normal(1, T, Hk, D), normal(1, T, H, D)
    # rates from one token to 256, over the heads, as fixed slopes or as the middle of what
    # the tokens ask for
    slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)
    if case["decay"] == "head":
        g = -slope
    else:
        g = -slope * torch.exp(torch.randn(1, T, H, generator=gen, device=dev))
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0).to(torch.int32)
    slots = N + 3
    pool = (0.1 * torch.randn(slots, H, D, D, generator=gen, device=dev)).to(DTYPES[case["pool"]])
    idx = torch.randperm(slots, generator=gen, device=dev)[:N].to(torch.int32)
    has = torch.rand(N, generator=gen, device=dev) < case["init"]
    return dict(case=case, q=q, k=k, v=v, g=g, cu=cu.to(dev), cu_cpu=cu, pool=pool, idx=idx,
                has=has, out=torch.empty(1, T, H, D, dtype=torch.bfloat16, device=dev))


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import kda_prefill_gb300 as kda
        if op == "rope":
            kda.rope(state["q"], state["k"], state["pos"], state["inv_freq"],
                     layout=state["case"]["layout"], factor=state["factor"],
                     q_out=state["q_out"], k_out=state["k_out"])
            return {"q": state["q_out"], "k": state["k_out"]}
        if op == "gated_norm":
            return kda.gated_norm(state["x"], state["weight"], gate=state["gate"],
                                  activation=state["case"]["gate"], eps=state["eps"],
                                  out=state["out"])
        kda.lin_attn_fwd(state["q"], state["k"], state["v"], state["g"], state["cu"],
                         state_cache=state["pool"], state_indices=state["idx"],
                         has_initial_state=state["has"], out=state["out"],
                         cu_seqlens_cpu=state["cu_cpu"])
        return {"out": state["out"], "pool": state["pool"]}
    if op == "rope":
        return _plain_rope(state)
    if op == "gated_norm":
        return _plain_norm(state)
    return _plain_lin(state)


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"].float()[:, None] * s["inv_freq"].float()
    cos, sin = torch.cos(angle) * s["factor"], torch.sin(angle) * s["factor"]
    return {"q": _rotate(s["q"], cos, sin, c), "k": _rotate(s["k"], cos, sin, c)}


def _rotate(x, cos, sin, c):
    r = c["rot"]
    y = x.float()
    cos, sin = cos[None, :, None], sin[None, :, None]
    if c["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def _plain_norm(s):
    x, z = s["x"].float(), s["gate"].float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    a = 1 / (1 + torch.exp(-z))
    return (y * (a if s["case"]["gate"] == "sigmoid" else z * a)).to(s["x"].dtype)


def _plain_lin(s):
    """The sequences cut into chunks: pairs inside a chunk by a masked matrix, chunks among each
    other by a masked matrix of decays over their states. Sums of log decays start at the place
    they are counted from."""
    q, k, v, pool, dev = s["q"][0], s["k"][0], s["v"][0], s["pool"], s["q"].device
    T, H = v.shape[0], v.shape[1]
    has, idx = s["has"], s["idx"].long()
    S0 = torch.where(has[:, None, None, None], pool[idx].float(), 0.0)     # [N, H, V, K]
    rep = H // q.shape[1]
    lens = (s["cu_cpu"][1:] - s["cu_cpu"][:-1]).long()
    n_chunks = (lens + CHUNK - 1) // CHUNK
    M = int(n_chunks.sum())
    seq = torch.repeat_interleave(torch.arange(len(lens)), n_chunks)       # of each chunk
    first = torch.cumsum(n_chunks, 0) - n_chunks                           # of each sequence
    at = torch.arange(M) - first[seq]                                      # place in its sequence
    tok = (s["cu_cpu"].long()[seq] + at * CHUNK)[:, None] + torch.arange(CHUNK)
    live = (tok < s["cu_cpu"].long()[seq + 1][:, None]).to(dev)            # [M, C]
    tok = tok.clamp(max=T - 1).to(dev)
    seq, last, some = seq.to(dev), (first + n_chunks - 1).to(dev), (n_chunks > 0).to(dev)
    at = at.to(dev)
    grid = live[:, None, :, None]

    def chunks(x, heads):  # [M, H, C, d]
        y = x[tok].float().transpose(1, 2)
        return torch.where(grid, y if heads == H else y.repeat_interleave(rep, 1), 0.0)

    Q, K, V = chunks(q, q.shape[1]), chunks(k, q.shape[1]), chunks(v, H)
    g = s["g"][0] if s["g"].dim() == 3 else s["g"].expand(T, H)
    G = torch.where(live[:, None], g[tok].transpose(1, 2), 0.0)            # [M, H, C]
    i = torch.arange(CHUNK, device=dev)
    # sums of the decays after j, up to i
    E = torch.cumsum(torch.where(i[:, None] > i[None, :], G[..., :, None], 0.0), -2)
    P = (Q @ K.transpose(-1, -2)) * torch.where(i[:, None] >= i[None, :], torch.exp(E), 0.0)
    o = P @ V
    dS = (V * torch.exp(E[..., -1, :])[..., None]).transpose(-1, -2) @ K   # [M, H, V, K]
    total = G.sum(-1)                                                      # [M, H]
    # decays from the end of chunk d to the start of chunk c, of one sequence
    m = torch.arange(M, device=dev)
    F = torch.cumsum(torch.where(m[:, None] > m[None, :], total.t()[:, :, None], 0.0), 1)
    F = torch.cat([torch.zeros_like(F[:, :1]), F[:, :-1]], 1)              # up to before c
    link = (m[:, None] > m[None, :]) & (seq[:, None] == seq[None, :])
    W = torch.where(link, torch.exp(torch.where(link, F, 0.0)), 0.0)       # [H, c, d]
    S = torch.bmm(W, dS.transpose(0, 1).reshape(H, M, D * D)).view(H, M, D, D).transpose(0, 1)
    start = torch.where(link, total.t()[:, None, :], 0.0).sum(-1).t()      # [M, H]
    S = S + torch.exp(start)[..., None, None] * S0[seq]
    o = o + torch.exp(torch.cumsum(G, -1))[..., None] * (Q @ S.transpose(-1, -2))
    o = o * (D ** -0.5)
    out = s["out"]
    out[0, tok[live]] = o.transpose(1, 2)[live].to(out.dtype)
    if M:
        at_end = last.clamp(min=0)
        end = torch.exp(total[at_end])[..., None, None] * S[at_end] + dS[at_end]
        S0 = torch.where(some[:, None, None, None], end, S0)
    pool[idx] = S0.to(pool.dtype)
    return {"out": out, "pool": pool}


# --------------------------------------------------------------------------
# What a pass cannot do without, and what it should give
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["k_heads"])
        return {"bytes": 2 * n * case["dim"] * BYTES[case["dtype"]] + 4 * case["tokens"],
                "flops": 3 * n * case["rot"]}
    if case["op"] == "gated_norm":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 3 * n * BYTES[case["dtype"]], "flops": 8 * n}
    lens = _lengths(case)
    T, N, H = sum(lens), len(lens), case["heads"]
    state = H * D * D * BYTES[case["pool"]]
    decays = 4 * H * (T if case["decay"] == "token" else 1)
    return {"bytes": 2 * T * D * 2 * (case["qk_heads"] + H) + decays + N * state * (1 + case["init"]),
            "flops": 4 * T * H * D * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        r, lay = case["rot"], case["layout"]
        pairs = torch.arange(r // 2, device="cuda")
        one = pairs if lay == "half" else 2 * pairs
        two = pairs + r // 2 if lay == "half" else 2 * pairs + 1
        turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["inv_freq"])[None, :, None]
        res = {}
        for name in ("q", "k"):
            y = s[name].double()
            z = torch.complex(y[..., one], y[..., two]) * turn
            y[..., one], y[..., two] = z.real, z.imag
            res[name] = y
        return res
    if case["op"] == "gated_norm":
        x, z = s["x"].double(), s["gate"].double()
        y = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + s["eps"]) * s["weight"].double()
        return y * torch.sigmoid(z) * (z if case["gate"] == "silu" else 1.0)
    # token by token, all sequences at once, longest first
    lens = _lengths(case)
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    rep = case["heads"] // case["qk_heads"]
    pool = s["pool"].double()
    out = torch.zeros(1, sum(lens), case["heads"], D, dtype=torch.float64, device="cuda")
    slot = s["idx"].long()[order]
    S = pool[slot] * s["has"][order].double()[:, None, None, None]
    start = s["cu"].long()[:-1][order]
    for t in range(max(lens, default=0)):
        n = sum(1 for a in lens if a > t)
        at = start[:n] + t
        q = s["q"][0, at].double().repeat_interleave(rep, 1)
        k = s["k"][0, at].double().repeat_interleave(rep, 1)
        v = s["v"][0, at].double()
        g = (s["g"][0, at] if case["decay"] == "token" else s["g"][None]).double()
        S[:n] *= torch.exp(g)[..., None, None]
        S[:n] += v[..., :, None] * k[..., None, :]
        out[0, at] = (S[:n] @ q[..., None]).squeeze(-1) * D ** -0.5
    pool[slot] = S
    return {"out": out, "pool": pool}
