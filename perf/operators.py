"""The serving operators around the chunked forward, as cases to measure.

Five operators: linear attention with one decay per head over prompts (``la_fwd``) and for single
tokens (``la_step``), the KDA recurrence for single tokens (``step``), and the two norms of a
layer: RMS norm and gate of the heads' outputs (``norm_gate``), and the norms around the residual
addition with its gate and scale (``add_norm``).

``run`` makes the library's calls where ``own`` is true and computes the same results with
elementary torch operations in fp32 where it is false. ``exact`` gives them in fp64, token by token.
"""
import math
import random

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda", torch.cuda.current_device())
else:
    DEV = torch.device("cpu")

PLAIN_CHUNK = 64   # tokens per chunk of the plain form


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt on a small model, its two value heads sharing one query / key head
        {"name": "la-prompt-tiny", "op": "la_fwd", "B": 1, "T": 128, "N": 0, "Hk": 1, "H": 2, "K": 64, "V": 64,
         "decay": "head", "init": True, "state": "fp32", "layout": "vk", "fused": False, "len_seed": 0},
        # prompts of equal length, as the library's fixed workload has them
        {"name": "la-prompt-fixed", "op": "la_fwd", "B": 2, "T": 2048, "N": 0, "Hk": 32, "H": 32, "K": 128, "V": 128,
         "decay": "head", "init": False, "state": "fp32", "layout": "vk", "fused": False, "len_seed": 0},
        # a packed batch of ragged prompts that go on from stored states, with a decay per token;
        # q, k and v are views of one projection
        {"name": "la-prompt-varlen", "op": "la_fwd", "B": 1, "T": 8192, "N": 16, "Hk": 32, "H": 32, "K": 128, "V": 128,
         "decay": "token", "init": True, "state": "fp32", "layout": "vk", "fused": True, "len_seed": 0},
        # one long document
        {"name": "la-prompt-long", "op": "la_fwd", "B": 1, "T": 65536, "N": 0, "Hk": 16, "H": 16, "K": 128, "V": 128,
         "decay": "head", "init": False, "state": "fp32", "layout": "vk", "fused": False, "len_seed": 0},
        # one request's next token: latency
        {"name": "la-step-1", "op": "la_step", "N": 1, "slots": 8, "Hk": 32, "H": 32, "K": 128, "V": 128,
         "decay": "head", "state": "fp32", "layout": "vk", "fused": True},
        # a full decoding batch over a pool of states
        {"name": "la-step-256", "op": "la_step", "N": 256, "slots": 288, "Hk": 32, "H": 32, "K": 128, "V": 128,
         "decay": "token", "state": "fp32", "layout": "vk", "fused": True},
        # a few requests' next tokens of a KDA layer
        {"name": "kda-step-4", "op": "kda_step", "N": 4, "slots": 16, "H": 32, "K": 128, "V": 128, "gate": "channel",
         "beta": "bf16", "state": "fp32", "layout": "vk", "fused": True},
        # a full decoding batch of a KDA layer whose pool of states is kept in bf16
        {"name": "kda-step-200", "op": "kda_step", "N": 200, "slots": 256, "H": 32, "K": 128, "V": 128,
         "gate": "channel", "beta": "bf16", "state": "bf16", "layout": "vk", "fused": True},
        # the heads' outputs of a decoding batch
        {"name": "norm-gate-step", "op": "norm_gate", "R": 8, "H": 32, "D": 128, "act": "sigmoid", "weight": True,
         "fused": True},
        # the heads' outputs of a prompt
        {"name": "norm-gate-prompt", "op": "norm_gate", "R": 16384, "H": 32, "D": 128, "act": "sigmoid",
         "weight": True, "fused": False},
        # residual addition and the next block's norm in a decoding batch
        {"name": "add-norm-step", "op": "add_norm", "R": 8, "D": 4096, "residual": "bf16", "post": False,
         "gate": False, "scale": "one"},
        # a prompt's residual stream in fp32, with the block's own output norm, gate and channel scale
        {"name": "add-norm-prompt", "op": "add_norm", "R": 16384, "D": 4096, "residual": "fp32", "post": True,
         "gate": True, "scale": "channel"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_step", "kda_step", "norm_gate", "add_norm"])
    K, V = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    H = rng.choice([1, 2, 3, 5, 8, 12, 16, 24, 32, 48, 64])
    Hk = rng.choice([d for d in (H, H, H // 2, H // 4, 1) if d >= 1 and H % d == 0])
    state, layout = rng.choice(["fp32", "fp32", "bf16"]), rng.choice(["vk", "vk", "kv"])
    if op == "la_fwd":
        N = rng.choice([0, 0, _spread(rng, 1, 64)])
        B = 1 if N else rng.choice([1, 1, 2, 3, 8])
        T = _spread(rng, 1, 65536)
        most = 16 * 65536 * 128   # the long document's value elements
        while max(B, (N + 1) // 2) * T * H * max(K, V) > most:
            T = max(1, T // 2 - rng.randrange(2))
        return {"op": op, "B": B, "T": T + (T == 3072), "N": N, "Hk": Hk, "H": H, "K": K, "V": V,
                "decay": rng.choice(["head", "token"]), "init": rng.random() < 0.6, "state": state, "layout": layout,
                "fused": rng.random() < 0.5, "len_seed": rng.randrange(1 << 20)}
    if op in ("la_step", "kda_step"):
        N = _spread(rng, 1, 512)
        while N * H * K * V > 256 * 32 * 128 * 128:
            N = max(1, N // 2 - rng.randrange(2))
        case = {"op": op, "N": N, "slots": N + rng.randrange(1, 33), "H": H, "K": K, "V": V, "state": state,
                "layout": layout, "fused": rng.random() < 0.5}
        if op == "la_step":
            return {**case, "Hk": Hk, "decay": rng.choice(["head", "token"])}
        return {**case, "gate": rng.choice(["channel", "channel", "head"]), "beta": rng.choice(["bf16", "fp32"])}
    if op == "norm_gate":
        R = _spread(rng, 1, 16384)
        while R * H * V > 16384 * 32 * 128:
            R = max(1, R // 2 - rng.randrange(2))
        return {"op": op, "R": R + (R == 3072), "H": H, "D": V, "act": rng.choice(["sigmoid", "silu"]),
                "weight": rng.random() < 0.7, "fused": rng.random() < 0.5}
    D = rng.choice([64, 100, 1000, 1023, 2048, 2880, 4096, 5120, 6144, 8192, 16384])
    R = _spread(rng, 1, 16384)
    while R * D > 16384 * 4096:
        R = max(1, R // 2 - rng.randrange(2))
    return {"op": op, "R": R + (R == 3072), "D": D, "residual": rng.choice(["bf16", "fp32"]),
            "post": rng.random() < 0.5, "gate": rng.random() < 0.5, "scale": rng.choice(["one", "number", "channel"])}


def _lengths(case):
    """Sequence lengths of a prompt case: `N` ragged ones, up to T tokens, or B equal ones."""
    if not case["N"]:
        return [case["T"]] * case["B"]
    rng = random.Random(case["len_seed"])
    least = min(64, case["T"]) if case["len_seed"] == 0 else 0
    lens = [rng.randint(least, case["T"]) for _ in range(case["N"])]
    return lens if sum(lens) else [1] + lens[1:]


# ---------------------------------------------------------------------------------- inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _split(lead, widths, fused, randn):
    """bf16 tensors [*lead, *w] for each w of `widths`: views of one projection's output, or each its own."""
    sizes = [math.prod(w) for w in widths]
    if not fused:
        return [randn(*lead, *w).to(torch.bfloat16) for w in widths]
    whole = randn(*lead, sum(sizes)).to(torch.bfloat16)
    parts = torch.split(whole, sizes, dim=-1)
    return [p.unflatten(-1, w) for p, w in zip(parts, widths)]


def _head_decay(H):
    """Log decays of the heads: memories from about two tokens to about 256."""
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)

    def randn_per_token(*shape):   # log of a decay that the token sets: about -0.05, at times much lower
        return torch.nn.functional.logsigmoid(1.5 * randn(*shape) + 3.0)

    op, s = case["op"], {"case": dict(case)}
    if op in ("la_fwd", "la_step", "kda_step"):
        H, K, V = case["H"], case["K"], case["V"]
        s["scale"] = K ** -0.5
        tail = (H, V, K) if case["layout"] == "vk" else (H, K, V)
        sdt = _dtype(case["state"])
    if op == "la_fwd":
        lens = _lengths(case)
        n = len(lens)
        B, T = (1, sum(lens)) if case["N"] else (case["B"], case["T"])
        Hk = case["Hk"]
        s["q"], s["k"], s["v"] = _split((B, T), [(Hk, K), (Hk, K), (H, V)], case["fused"], randn)
        s["decay"] = _head_decay(H) if case["decay"] == "head" else randn_per_token(B, T, H)
        s["init"] = (0.5 * randn(n, *tail)).to(sdt) if case["init"] else None
        s["cu"], s["longest"] = None, max(lens)
        if case["N"]:
            ends = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
            s["cu"] = ends.to(torch.int32).to(DEV)
    elif op == "la_step":
        N, Hk = case["N"], case["Hk"]
        s["q"], s["k"], s["v"] = _split((N,), [(Hk, K), (Hk, K), (H, V)], case["fused"], randn)
        s["decay"] = _head_decay(H) if case["decay"] == "head" else randn_per_token(N, H)
    elif op == "kda_step":
        N = case["N"]
        per_head = case["gate"] == "head"
        s["q"], s["k"], s["v"] = _split((N,), [(H, K), (H, K), (H, V)], case["fused"], randn)
        s["g"] = randn(N, H).to(torch.bfloat16) if per_head else randn(N, H, K).to(torch.bfloat16)
        s["beta"] = randn(N, H).to(_dtype(case["beta"]))
        s["A_log"] = 0.3 * randn(H)
        s["dt_bias"] = 0.5 * randn(H) - 1.0 if per_head else 0.5 * randn(H, K) - 1.0
    elif op == "norm_gate":
        R, H, D = case["R"], case["H"], case["D"]
        s["x"] = (2.0 * randn(R, H, D)).to(torch.bfloat16)
        # fused: the gate is the second half of a projection that another part of the layer reads too
        s["gate"] = _split((R,), [(H, D), (H, D)], case["fused"], randn)[1]
        s["weight"] = 1.0 + 0.1 * randn(D) if case["weight"] else None
    else:
        R, D = case["R"], case["D"]
        s["x"] = randn(R, D).to(torch.bfloat16)
        s["residual"] = (4.0 * randn(R, D)).to(_dtype(case["residual"]))
        s["weight"] = 1.0 + 0.1 * randn(D)
        s["post"] = 1.0 + 0.1 * randn(D) if case["post"] else None
        s["gate"] = randn(R, D).to(torch.bfloat16) if case["gate"] else None
        s["scale"] = {"one": 1.0, "number": 0.35}.get(case["scale"])
        if s["scale"] is None:
            s["scale"] = 0.5 + 0.1 * randn(D)
    if op in ("la_step", "kda_step"):
        # each request's state lies anywhere in the pool
        s["state"] = (0.5 * randn(case["slots"], *tail)).to(sdt)
        s["slots"] = torch.randperm(case["slots"], generator=gen, device=DEV)[:N].to(torch.int32)
    return s


# ---------------------------------------------------------------------------------- the operators

def run(state):
    op = state["case"]["op"]
    return (_run_own if own else _run_plain)[op](state)


def _own_la_fwd(s):
    import chunked_gated_delta_02_gb300 as kda
    c = s["case"]
    return kda.la_fwd(s["q"], s["k"], s["v"], s["decay"], scale=s["scale"], initial_state=s["init"],
                      output_final_state=True, cu_seqlens=s["cu"], state_layout=c["layout"],
                      state_dtype=_dtype(c["state"]))


def _own_la_step(s):
    import chunked_gated_delta_02_gb300 as kda
    o = kda.la_step(s["q"], s["k"], s["v"], s["decay"], s["state"], state_indices=s["slots"], scale=s["scale"],
                    state_layout=s["case"]["layout"])
    return o, s["state"]


def _own_kda_step(s):
    import chunked_gated_delta_02_gb300 as kda
    o = kda.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["A_log"], s["state"], dt_bias=s["dt_bias"],
                 lower_bound=-5.0, scale=s["scale"], state_indices=s["slots"], state_layout=s["case"]["layout"])
    return o, s["state"]


def _own_norm_gate(s):
    import chunked_gated_delta_02_gb300 as kda
    return kda.norm_gate(s["x"], s["gate"], s["weight"], activation=s["case"]["act"])


def _own_add_norm(s):
    import chunked_gated_delta_02_gb300 as kda
    return kda.add_norm(s["x"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                        residual_scale=s["scale"])


_run_own = {"la_fwd": _own_la_fwd, "la_step": _own_la_step, "kda_step": _own_kda_step, "norm_gate": _own_norm_gate,
            "add_norm": _own_add_norm}


# ---- plain forms

def _shared_heads(x, H, dim):
    """Each query / key head once for every value head that reads it."""
    n = x.shape[dim]
    return x if n == H else x.repeat_interleave(H // n, dim=dim)


def _sums_between(x):
    """[..., n] -> [..., n, n]: the sum of x over (j, i] at (i, j), -inf above the diagonal."""
    n = x.shape[-1]
    i = torch.arange(n, device=x.device)
    rows = torch.where(i[:, None] > i, x[..., :, None], torch.zeros((), device=x.device)).cumsum(-2)
    return torch.where(i[:, None] >= i, rows, torch.full((), -math.inf, device=x.device))


def _plain_la_fwd(s):
    c, cu = s["case"], s["cu"]
    H, K, V, C = c["H"], c["K"], c["V"], PLAIN_CHUNK
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    B, T = q.shape[:2]
    a = s["decay"].expand(B, T, H) if s["decay"].dim() == 1 else s["decay"]
    n, longest = (B, T) if cu is None else (cu.numel() - 1, s["longest"])
    P = -(-max(longest, 1) // C) * C
    if cu is not None:   # ragged sequences as rows of equal length
        at = torch.arange(P, device=DEV)
        rows = cu[:-1, None].long() + at
        inside = at < (cu[1:] - cu[:-1])[:, None]
        rows = rows.clamp(max=max(T - 1, 0))
        q, k, v, a = ((x[0][rows] * inside[(...,) + (None,) * (x.dim() - 2)]) if T else
                      torch.zeros(n, P, *x.shape[2:], device=DEV) for x in (q, k, v, a))
    else:
        q, k, v, a = (torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, P - T)) for x in (q, k, v, a))
    # [n, H, chunks, C, .]
    q, k, v = (_shared_heads(x, H, 2).unflatten(1, (P // C, C)).permute(0, 3, 1, 2, 4) for x in (q, k, v))
    a = a.unflatten(1, (P // C, C)).permute(0, 3, 1, 2)
    between = _sums_between(a)
    to_end = a.flip(-1).cumsum(-1).flip(-1) - a
    scores = (q @ k.transpose(-1, -2)) * torch.exp(between)
    o = scores @ v
    local = (k * torch.exp(to_end)[..., None]).transpose(-1, -2) @ v      # [n, H, chunks, K, V]
    first = torch.zeros(n, H, 1, K, V, device=DEV)
    if s["init"] is not None:
        init = s["init"].float() if c["layout"] == "kv" else s["init"].float().transpose(-1, -2)
        first = init[:, :, None]
    # state after chunk i: decays over chunks (j, i] times what chunk j adds, the first state before all
    total = torch.nn.functional.pad(a.sum(-1), (1, 0))
    states = (torch.exp(_sums_between(total)) @ torch.cat([first, local], 2).flatten(-2)).unflatten(-1, (K, V))
    o = o + torch.exp(a.cumsum(-1))[..., None] * (q @ states[:, :, :-1])
    o = (s["scale"] * o).permute(0, 2, 3, 1, 4).reshape(n, P, H, V).to(torch.bfloat16)
    if cu is None:
        o = o[:, :T].contiguous()
    else:   # the packed rows again
        seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(T, device=DEV, dtype=torch.int32), right=True)
        o = o[seq, torch.arange(T, device=DEV) - cu[:-1].long()[seq]][None]
    last = states[:, :, -1]
    return o, (last if c["layout"] == "kv" else last.transpose(-1, -2)).contiguous().to(_dtype(c["state"]))


def _plain_update(s, decayed_and_new):
    """Reads the requests' states of the pool as [N, H, K, V], writes the new ones back."""
    slots, kv = s["slots"].long(), s["case"]["layout"] == "kv"
    old = s["state"][slots].float()
    new, o = decayed_and_new(old if kv else old.transpose(-1, -2))
    s["state"][slots] = (new if kv else new.transpose(-1, -2)).to(s["state"].dtype)
    return (s["scale"] * o).to(torch.bfloat16), s["state"]


def _plain_la_step(s):
    H = s["case"]["H"]
    q, k, v = _shared_heads(s["q"].float(), H, 1), _shared_heads(s["k"].float(), H, 1), s["v"].float()

    def update(S):
        a = torch.exp(s["decay"])[..., None, None]
        S = a * S + k[..., :, None] * v[..., None, :]
        return S, (q[..., :, None] * S).sum(-2)

    return _plain_update(s, update)


def _plain_kda_step(s):
    q, k, v, g = s["q"].float(), s["k"].float(), s["v"].float(), s["g"].float()
    beta = torch.sigmoid(s["beta"].float())

    def update(S):
        ea = torch.exp(s["A_log"])
        if g.dim() == 2:
            a = torch.exp(-5.0 * torch.sigmoid(ea * (g + s["dt_bias"])))[..., None]
        else:
            a = torch.exp(-5.0 * torch.sigmoid(ea[:, None] * (g + s["dt_bias"])))
        qn = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        kn = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
        S = a[..., None] * S
        u = beta[..., None] * (v - (kn[..., :, None] * S).sum(-2))
        S = S + kn[..., :, None] * u[..., None, :]
        return S, (qn[..., :, None] * S).sum(-2)

    return _plain_update(s, update)


def _plain_rms(x, weight):
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return y if weight is None else y * weight


def _plain_norm_gate(s):
    g = s["gate"].float()
    act = torch.sigmoid(g) if s["case"]["act"] == "sigmoid" else g * torch.sigmoid(g)
    return (_plain_rms(s["x"].float(), s["weight"]) * act).to(torch.bfloat16)


def _plain_add_norm(s):
    z = s["x"].float()
    if s["post"] is not None:
        z = _plain_rms(z, s["post"])
    if s["gate"] is not None:
        z = z * torch.sigmoid(s["gate"].float())
    h = s["residual"].float() + s["scale"] * z
    return _plain_rms(h, s["weight"]).to(torch.bfloat16), h.to(s["residual"].dtype)


_run_plain = {"la_fwd": _plain_la_fwd, "la_step": _plain_la_step, "kda_step": _plain_kda_step,
              "norm_gate": _plain_norm_gate, "add_norm": _plain_add_norm}


# ---------------------------------------------------------------------------------- fp64

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    op = case["op"]
    if op == "norm_gate":
        x, g, w = d["x"], d["gate"], d["weight"]
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
        y = y if w is None else y * w
        return y / (1 + torch.exp(-g)) * (g if case["act"] == "silu" else 1.0)
    if op == "add_norm":
        z = d["x"]
        if d["post"] is not None:
            z = z / torch.sqrt((z ** 2).sum(-1, keepdim=True) / z.shape[-1] + 1e-6) * d["post"]
        if d["gate"] is not None:
            z = z / (1 + torch.exp(-d["gate"]))
        h = d["residual"] + d["scale"] * z
        return h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / h.shape[-1] + 1e-6) * d["weight"], h
    H, K, V = case["H"], case["K"], case["V"]
    vk = case["layout"] == "vk"
    if op == "la_fwd":
        return _exact_la_fwd(case, d, vk)
    slots = s["slots"].long()
    S = d["state"][slots]
    S = S.transpose(-1, -2).clone() if vk else S.clone()           # [N, H, K, V]
    if op == "la_step":
        q, k = (x[:, torch.arange(H, device=DEV) // (H // x.shape[1])] for x in (d["q"], d["k"]))
        S = S * torch.exp(d["decay"]).reshape(-1, H, 1, 1) + torch.einsum("nhk,nhv->nhkv", k, d["v"])
    else:
        z = d["g"] if d["g"].dim() == 3 else d["g"][..., None]
        bias = d["dt_bias"] if d["dt_bias"].dim() == 2 else d["dt_bias"][:, None]
        a = torch.exp(-5.0 / (1 + torch.exp(-torch.exp(d["A_log"])[:, None] * (z + bias))))
        q, k = (x / torch.sqrt((x ** 2).sum(-1, keepdim=True) + 1e-6) for x in (d["q"], d["k"]))
        S = S * a[..., None]
        miss = d["v"] - torch.einsum("nhk,nhkv->nhv", k, S)
        S = S + torch.einsum("nhk,nhv,nh->nhkv", k, miss, 1 / (1 + torch.exp(-d["beta"])))
    o = d["scale"] * torch.einsum("nhk,nhkv->nhv", q, S)
    pool = d["state"].clone()
    pool[slots] = S.transpose(-1, -2) if vk else S
    return o, pool


def _exact_la_fwd(case, d, vk):
    """Token after token, the sequences side by side."""
    H, K, V = case["H"], case["K"], case["V"]
    lens = _lengths(case)
    n = len(lens)
    q, k, v = d["q"], d["k"], d["v"]
    group = torch.arange(H, device=DEV) // (H // q.shape[2])
    first = [0] * n if not case["N"] else [sum(lens[:i]) for i in range(n)]
    row = list(range(n)) if not case["N"] else [0] * n
    S = torch.zeros(n, H, K, V, device=DEV, dtype=torch.float64)
    if d["init"] is not None:
        S += d["init"].transpose(-1, -2) if vk else d["init"]
    o = torch.zeros(*v.shape[:3], V, device=DEV, dtype=torch.float64)
    order = sorted(range(n), key=lambda i: -lens[i])               # those still running come first
    S = S[order]
    rows = torch.tensor([row[i] for i in order], device=DEV)
    starts = torch.tensor([first[i] for i in order], device=DEV)
    live = n
    per_head = torch.exp(d["decay"]) if d["decay"].dim() == 1 else None
    for t in range(max(lens, default=0)):
        while live and lens[order[live - 1]] <= t:
            live -= 1
        r, at = rows[:live], starts[:live] + t
        a = per_head if per_head is not None else torch.exp(d["decay"][r, at])
        X = S[:live]
        X *= a[..., None, None]
        X += k[r, at][:, group, :, None] * v[r, at][:, :, None, :]
        o[r, at] = torch.matmul(q[r, at][:, group, None, :], X)[:, :, 0] * d["scale"]
    back = torch.empty_like(S)
    back[order] = S
    return o, (back.transpose(-1, -2) if vk else back).contiguous()


# ---------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "norm_gate":
        n = case["R"] * case["H"] * case["D"]
        return {"bytes": 6 * n + 4 * case["D"] * case["weight"], "flops": 8 * n}
    if op == "add_norm":
        n, D = case["R"] * case["D"], case["D"]
        size = 2 if case["residual"] == "bf16" else 4
        weights = 4 * D * (1 + case["post"] + (case["scale"] == "channel"))
        return {"bytes": n * (4 + 2 * size + 2 * case["gate"]) + weights, "flops": n * (8 + 4 * case["post"] + 4 * case["gate"])}
    H, K, V = case["H"], case["K"], case["V"]
    size = 2 if case["state"] == "bf16" else 4
    if op == "la_fwd":
        lens = _lengths(case)
        tokens, n = sum(lens), len(lens)
        moved = tokens * (4 * case["Hk"] * K + 4 * H * V) + n * H * K * V * size * (1 + case["init"])
        moved += 4 * (tokens * H if case["decay"] == "token" else H)
        return {"bytes": moved, "flops": tokens * H * 4 * K * V}       # state update and read, token by token
    N = case["N"]
    moved = 2 * N * H * K * V * size + 4 * N
    if op == "la_step":
        moved += N * (4 * case["Hk"] * K + 4 * H * V) + 4 * H * (N if case["decay"] == "token" else 1)
        return {"bytes": moved, "flops": 5 * N * H * K * V}
    gate = K if case["gate"] == "channel" else 1
    moved += N * H * (4 * K + 4 * V + 2 * gate + (4 if case["beta"] == "fp32" else 2)) + 4 * H * (1 + gate)
    return {"bytes": moved, "flops": 7 * N * H * K * V}
