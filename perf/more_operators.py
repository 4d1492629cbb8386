"""More operators of a linear-attention stack, as cases to be measured: the gated delta rule
with a decay for each head (packed prompts and single tokens over a paged pool of states), and
the norms of queries and keys for each head with the rotary positions in the same pass.

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is set,
by the calls a user makes of this package.
"""
import math
import random

import torch

own = False

D = 128     # head size of q, k and v of the delta rule
CHUNK = 64  # tokens per chunk of the delta rule's plain form, at most
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _delta(name, *, ones=0, seqs=0, lo=1, hi=1, empty=0.0, heads=12, qk_heads=12, decay="token",
           pool="fp32", fused=False, init=0.5, lens_seed=0):
    c = dict(op="gated_delta", ones=ones, seqs=seqs, lo=lo, hi=hi, empty=empty, heads=heads,
             qk_heads=qk_heads, decay=decay, pool=pool, fused=fused, init=init,
             lens_seed=lens_seed)
    return dict(c, name=name) if name else c


def _turn(name, *, tokens, heads=12, k_heads=12, dim=D, rot=D, layout="half", far=0,
          weights="dim", fused=False, dtype="bf16"):
    c = dict(op="qk_norm_rope", tokens=tokens, heads=heads, k_heads=k_heads, dim=dim, rot=rot,
             layout=layout, far=far, weights=weights, fused=fused, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request answering: the latency of a single token
        _delta("delta_step_1", ones=1, init=1.0),
        # a full decode batch, one token for each of 512 requests
        _delta("delta_step_512", ones=512, init=1.0),
        # one prompt, one token over a round length
        _delta("delta_prompt_4097", seqs=1, lo=4097, hi=4097, init=1.0),
        # one long prompt
        _delta("delta_prompt_16384", seqs=1, lo=16384, hi=16384, init=0.0),
        # the same on a shard with few heads, one decay a head for all tokens
        _delta("delta_prompt_16384_h2", seqs=1, lo=16384, hi=16384, heads=2, qk_heads=2,
               decay="head", init=0.0),
        # a prompt batch of ragged requests, q and k heads shared by groups of three v heads,
        # all three views of one projection's output
        _delta("delta_varlen_128", seqs=128, lo=1, hi=2048, empty=0.05, qk_heads=4, fused=True,
               lens_seed=3),
        # decode and prompts in one batch, 2-byte states
        _delta("delta_mixed", ones=512, seqs=4, lo=2048, hi=2048, pool="bf16", lens_seed=4),
        # a decode batch deep in long contexts, q and k in one projection's output
        _turn("turn_step_512", tokens=512, far=131072, fused=True),
        # a long prompt, every dimension turned
        _turn("turn_prompt_16384", tokens=16384),
        # the same with few k heads, a weight for each head, half of each head turned by
        # interleaved pairs
        _turn("turn_prompt_16384_grouped", tokens=16384, k_heads=2, rot=64, layout="interleaved",
              weights="head"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "prompt", "batch", "mixed", "turn", "turn"])
    if kind == "turn":
        dim = rng.choice([64, 128, 192])
        rot = rng.choice([dim, dim // 2])
        return _turn(None, tokens=_log_int(rng, 1, 16384), heads=rng.randint(1, 12),
                     k_heads=rng.randint(1, 12), dim=dim, rot=rot,
                     layout=rng.choice(["half", "interleaved"]),
                     far=rng.choice([0, _log_int(rng, 4096, 131072)]),
                     weights=rng.choice(["none", "dim", "head"]), fused=rng.random() < 0.5,
                     dtype=rng.choice(["bf16", "bf16", "fp16"]))
    groups, per = rng.choice([1, 2, 4]), rng.choice([1, 2, 3])
    kw = dict(heads=groups * per, qk_heads=groups, decay=rng.choice(["head", "token"]),
              pool=rng.choice(["fp32", "fp32", "bf16", "fp16"]), fused=rng.random() < 0.5,
              init=rng.choice([0.0, 0.5, 1.0]), lens_seed=rng.randrange(1 << 20))
    if kind == "step":
        return _delta(None, ones=_log_int(rng, 1, 512), **kw)
    if kind == "prompt":
        n = _log_int(rng, 2, 16384)
        return _delta(None, seqs=1, lo=n, hi=n, **kw)
    if kind == "batch":
        return _delta(None, seqs=_log_int(rng, 2, 96), lo=1, hi=_log_int(rng, 9, 2048), empty=0.05,
                      **kw)
    hi = _log_int(rng, 64, 2048)
    return _delta(None, ones=_log_int(rng, 1, 512), seqs=rng.randint(1, 8), lo=max(1, hi // 2),
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

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev).to(dtype)

    if case["op"] == "qk_norm_rope":
        T, H, Hk, dim = case["tokens"], case["heads"], case["k_heads"], case["dim"]
        dt = DTYPES[case["dtype"]]
        if case["fused"]:
            qk = normal(1, T, H + Hk, dim, dtype=dt)
            q, k = qk[:, :, :H], qk[:, :, H:]
        else:
            q, k = normal(1, T, H, dim, dtype=dt), normal(1, T, Hk, dim, dtype=dt)
        if case["far"]:  # requests at their own places
            pos = torch.randint(0, case["far"], (T,), generator=gen, device=dev)
        else:            # one prompt from its start
            pos = torch.arange(T, device=dev)
        shapes = {"none": (None, None), "dim": ((dim,), (dim,)), "head": ((H, dim), (Hk, dim))}
        w = [None if s is None else 1.0 + 0.1 * normal(*s, dtype=torch.float32)
             for s in shapes[case["weights"]]]
        freq = [10000.0 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
        return dict(case=case, q=q, k=k, q_weight=w[0], k_weight=w[1], pos=pos.to(torch.int32),
                    inv_freq=torch.tensor(freq, dtype=torch.float64, device=dev), eps=1e-6,
                    q_out=torch.empty_like(q, memory_format=torch.contiguous_format),
                    k_out=torch.empty_like(k, memory_format=torch.contiguous_format))

    lens = _lengths(case)
    N, T, H, Hk = len(lens), sum(lens), case["heads"], case["qk_heads"]
    if case["fused"]:
        qkv = normal(1, T, 2 * Hk + H, D)
        q, k, v = qkv[:, :, :Hk], qkv[:, :, Hk:2 * Hk], qkv[:, :, 2 * Hk:]
    else:
        q, k, v = normal(1, T, Hk, D), normal(1, T, Hk, D), normal(1, T, H, D)
    # rates from one token to 256, over the heads, as fixed slopes or as the middle of what
    # the tokens ask for; writes of any strength
    slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)
    if case["decay"] == "head":
        g = -slope
    else:
        g = -slope * torch.exp(torch.randn(1, T, H, generator=gen, device=dev))
    beta = torch.sigmoid(2.0 * torch.randn(1, T, H, generator=gen, device=dev))
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0).to(torch.int32)
    slots = N + 3
    pool = (0.1 * torch.randn(slots, H, D, D, generator=gen, device=dev)).to(DTYPES[case["pool"]])
    idx = torch.randperm(slots, generator=gen, device=dev)[:N].to(torch.int32)
    has = torch.rand(N, generator=gen, device=dev) < case["init"]
    return dict(case=case, q=q, k=k, v=v, g=g, beta=beta, cu=cu.to(dev), cu_cpu=cu, pool=pool,
                idx=idx, has=has, out=torch.empty(1, T, H, D, dtype=torch.bfloat16, device=dev))


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import kda_prefill_gb300 as kda
        if op == "qk_norm_rope":
            kda.qk_norm_rope(state["q"], state["k"], state["q_weight"], state["k_weight"],
                             state["pos"], state["inv_freq"], layout=state["case"]["layout"],
                             eps=state["eps"], q_out=state["q_out"], k_out=state["k_out"])
            return {"q": state["q_out"], "k": state["k_out"]}
        kda.gated_delta_fwd(state["q"], state["k"], state["v"], state["g"], state["beta"],
                            state["cu"], state_cache=state["pool"], state_indices=state["idx"],
                            has_initial_state=state["has"], out=state["out"],
                            cu_seqlens_cpu=state["cu_cpu"])
        return {"out": state["out"], "pool": state["pool"]}
    if op == "qk_norm_rope":
        return _plain_turn(state)
    return _plain_delta(state)


def _plain_turn(s):
    c = s["case"]
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[None, :, None], torch.sin(angle).float()[None, :, None]

    def one(x, w):
        r, y = c["rot"], x.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + s["eps"])
        y = y if w is None else y * w
        if c["layout"] == "half":
            a, b = y[..., :r // 2], y[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([turned, y[..., r:]], -1).to(x.dtype)

    return {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"])}


def _plain_delta(s):
    """The sequences cut into chunks: what a chunk's tokens write, by a triangular inverse made of
    ever larger blocks, for all chunks at once; then the chunks in their order, all sequences
    at once. Sums of log decays start at the place they are counted from."""
    pool, dev, H = s["pool"], s["q"].device, s["v"].shape[2]
    has, idx, T = s["has"], s["idx"].long(), s["v"].shape[1]
    rep = H // s["q"].shape[2]
    cu = s["cu_cpu"].long()
    lens = cu[1:] - cu[:-1]
    longest = int(lens.max()) if len(lens) else 0
    C = min(CHUNK, 1 << max(0, longest - 1).bit_length())
    n_chunks = (lens + C - 1) // C
    seq = torch.repeat_interleave(torch.arange(len(lens)), n_chunks)       # of each chunk
    first = torch.cumsum(n_chunks, 0) - n_chunks                           # of each sequence
    M = len(seq)
    tok = (cu[seq] + (torch.arange(M) - first[seq]) * C)[:, None] + torch.arange(C)
    live = (tok < cu[seq + 1][:, None]).to(dev)                            # [M, C]
    tok = tok.clamp(max=max(0, T - 1)).to(dev)

    def chunks(x):  # [M, H, C, d]
        y = x[0][tok].float().transpose(1, 2)
        y = y if y.shape[1] == H else y.repeat_interleave(rep, 1)
        return torch.where(live[:, None, :, None], y, 0.0)

    def unit(x):
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)

    Q, K, V = unit(chunks(s["q"])) * D ** -0.5, unit(chunks(s["k"])), chunks(s["v"])
    g = s["g"] if s["g"].dim() == 3 else s["g"].expand(1, T, H)
    G, B = chunks(g[..., None])[..., 0], chunks(s["beta"][..., None])      # [M, H, C], [M, H, C, 1]
    i = torch.arange(C, device=dev)
    below = i[:, None] > i[None, :]
    # e to the sums of the decays after j, up to i
    L = torch.exp(torch.cumsum(torch.where(below, G[..., :, None], 0.0), -2))
    A = torch.where(below, B * L * (K @ K.transpose(-1, -2)), 0.0)
    X = torch.eye(C, device=dev).expand_as(A).contiguous()                 # (1 + A)^-1
    w = 1
    while w < C:
        a, b = i[(i // w) % 2 == 1].view(-1, w), i[(i // w) % 2 == 0].view(-1, w)
        at, before = a[:, :, None], b[:, None, :]
        X[:, :, at, before] = -(X[:, :, at, a[:, None, :]] @ A[:, :, at, before]
                                @ X[:, :, b[:, :, None], before])
        w *= 2
    from_start = torch.exp(torch.cumsum(G, -1))[..., None]
    P = torch.where(below | (i[:, None] == i[None, :]), L * (Q @ K.transpose(-1, -2)), 0.0)
    W, U0 = X @ (B * from_start * K), X @ (B * V)
    Qs, Ke = from_start * Q, L[..., -1, :, None] * K
    kept = from_start[:, :, -1:]
    order = torch.argsort(n_chunks, descending=True, stable=True)
    S = torch.where(has[:, None, None, None], pool[idx].float(), 0.0)[order.to(dev)]
    O = torch.empty_like(V)
    for c in range(int(n_chunks.max()) if len(lens) else 0):
        n = int((n_chunks > c).sum())
        m = (first[order[:n]] + c).to(dev)
        St = S[:n].transpose(-1, -2)
        U = U0[m] - W[m] @ St
        O[m] = Qs[m] @ St + P[m] @ U
        S[:n] = kept[m] * S[:n] + U.transpose(-1, -2) @ Ke[m]
    out = s["out"]
    out[0, tok[live]] = O.transpose(1, 2)[live].to(out.dtype)
    pool[idx[order.to(dev)]] = S.to(pool.dtype)
    return {"out": out, "pool": pool}


# --------------------------------------------------------------------------
# What a pass cannot do without, and what it should give
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "qk_norm_rope":
        n = case["tokens"] * (case["heads"] + case["k_heads"])
        return {"bytes": 2 * n * case["dim"] * BYTES[case["dtype"]] + 4 * case["tokens"],
                "flops": n * (4 * case["dim"] + 3 * case["rot"])}
    lens = _lengths(case)
    T, N, H = sum(lens), len(lens), case["heads"]
    state = H * D * D * BYTES[case["pool"]]
    scalars = 4 * H * (2 * T if case["decay"] == "token" else T + 1)
    return {"bytes": 2 * T * D * 2 * (case["qk_heads"] + H) + scalars + N * state * (1 + case["init"]),
            "flops": 6 * T * H * D * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk_norm_rope":
        r = case["rot"]
        pairs = torch.arange(r // 2, device="cuda")
        one = pairs if case["layout"] == "half" else 2 * pairs
        two = pairs + r // 2 if case["layout"] == "half" else 2 * pairs + 1
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["inv_freq"])[None, :, None]
        res = {}
        for name in ("q", "k"):
            y = s[name].double()
            y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + s["eps"])
            if s[name + "_weight"] is not None:
                y = y * s[name + "_weight"].double()
            z = torch.complex(y[..., one], y[..., two]) * turn
            y[..., one], y[..., two] = z.real, z.imag
            res[name] = y
        return res
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
        q, k = (x[0, at].double().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
        q = q * torch.rsqrt(q.pow(2).sum(-1, keepdim=True) + 1e-6) * D ** -0.5
        k = k * torch.rsqrt(k.pow(2).sum(-1, keepdim=True) + 1e-6)
        g = (s["g"][0, at] if case["decay"] == "token" else s["g"][None]).double()
        S[:n] *= torch.exp(g)[..., None, None]
        new = s["v"][0, at].double() - (S[:n] @ k[..., None]).squeeze(-1)
        S[:n] += (s["beta"][0, at].double()[..., None] * new)[..., :, None] * k[..., None, :]
        out[0, at] = (S[:n] @ q[..., None]).squeeze(-1)
    pool[slot] = S
    return {"out": out, "pool": pool}
