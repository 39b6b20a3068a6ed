"""Measured cases of the gated delta rule with one decay per head and of the norm and rotation of
queries and keys before it.

Three operators, each in its plain form (elementary torch operations in 32 bits, 64 for the decay
sums and the angles, rounded once at the end) and as the calls a user makes of the binding:

``prefill``  the gated delta rule over packed sequences, per sequence and value head h with
             query/key head h // (H // Hk):
             S' = e^{g_t} S_{t-1},  u = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u^T,
             o_t = scale S_t^T q_t. ``binding.delta_prefill``.
``decode``   one token of the same recurrence for B sequences, states updated in place.
             ``binding.delta_decode``.
``rotate``   the norm of each query and key head (w x / rms(x), x / |x| or none), then rotary
             positions: the channel pair i of the first ``rot`` channels turns by
             position[axis(i)] * inv_freq[i]. ``binding.norm_rotate``.
"""

import math

import torch

own = False

_CHUNK = 64  # tokens per chunk of the plain prefill
_EPS = 1e-6
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    def prefill(name, lens, H, Hk, d_k, d_v, types, per_token=True):
        return {"name": name, "op": "prefill", "lens": lens, "H": H, "Hk": Hk, "d_k": d_k, "d_v": d_v, "in": types[0],
                "out": types[1], "per_token": per_token}

    b, f = ("bf16", "bf16"), ("fp32", "fp32")
    return [
        # three short prompts of a server that has nothing else to do: latency
        prefill("prefill_short", "1,17,46", 8, 8, 128, 128, b),
        # one layer's prompt at this repository's headline sizes (T = 4096, H = 96, d = 128)
        prefill("prefill_layer", "4096", 96, 96, 128, 128, b),
        # ragged prompts packed together, query/key heads shared by two value heads, fp32 read-out
        prefill("prefill_packed", "3001,0,517,1024,129,4096,1,2222", 32, 16, 128, 128, ("bf16", "fp32")),
        # one long document on few heads, shared by four
        prefill("prefill_long", "65536", 16, 4, 128, 128, b),
        # many short requests admitted at once, value heads of 64 channels
        prefill("prefill_many", ",".join(str(40 + 37 * i % 211) for i in range(64)), 16, 8, 128, 64, b),
        # reference accuracy: fp32 in and out, odd head sizes, a constant decay for each head
        prefill("prefill_fp32", "700,333", 6, 2, 100, 72, f, False),
        # one user's next token
        {"name": "decode_one", "op": "decode", "B": 1, "H": 96, "Hk": 96, "d_k": 128, "d_v": 128, "in": "bf16",
         "out": "bf16", "per_token": True},
        # a full batch at this repository's decode sizes (B = 256, H = 96)
        {"name": "decode_batch", "op": "decode", "B": 256, "H": 96, "Hk": 96, "d_k": 128, "d_v": 128, "in": "bf16",
         "out": "fp32", "per_token": True},
        # an odd batch, shared query/key heads, fp32, a constant decay for each head
        {"name": "decode_shared", "op": "decode", "B": 37, "H": 24, "Hk": 8, "d_k": 100, "d_v": 72, "in": "fp32",
         "out": "fp32", "per_token": False},
        # the queries and keys of one token far into a document
        {"name": "rotate_one", "op": "rotate", "T": 1, "Hq": 96, "Hk": 96, "d": 128, "rot": 128, "norm": "rms",
         "pairs": "halves", "axes": 1, "far": 1 << 20, "fused": True, "in": "bf16", "out": "bf16"},
        # a prompt's queries and keys at this repository's headline sizes, a quarter of the channels turned
        {"name": "rotate_prompt", "op": "rotate", "T": 4096, "Hq": 96, "Hk": 96, "d": 128, "rot": 32, "norm": "l2",
         "pairs": "halves", "axes": 1, "far": 1 << 17, "fused": False, "in": "bf16", "out": "bf16"},
        # a video's patches: time, height and width, neighbouring channels, shared keys, an odd number of
        # rows out of a fused projection
        {"name": "rotate_video", "op": "rotate", "T": 10007, "Hq": 16, "Hk": 4, "d": 72, "rot": 72, "norm": "rms",
         "pairs": "neighbours", "axes": 3, "far": 4096, "fused": True, "in": "bf16", "out": "fp32"},
    ]


def draw(rng):
    def spread(lo, hi):  # over the logarithm
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "rotate", "rotate"])
    if op == "rotate":
        d = rng.choice([64, 128, 256, 8 * spread(2, 32), spread(4, 256)])
        Hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
        Hq = Hk * rng.choice([1, 1, 2, 4, 7])
        rot = rng.choice([d - d % 2, d - d % 2, 2 * spread(1, d // 2)])
        return {"op": op, "T": spread(1, max(1, 4096 * 192 * 128 // ((Hq + Hk) * d))), "Hq": Hq, "Hk": Hk, "d": d, "rot": rot,
                "norm": rng.choice(["rms", "rms", "l2", "none"]), "pairs": rng.choice(["halves", "neighbours"]),
                "axes": rng.choice([1, 1, 2, 3]), "far": spread(1, 1 << 22), "fused": rng.random() < 0.5,
                "in": rng.choice(["bf16", "bf16", "fp32"]), "out": rng.choice(["bf16", "bf16", "fp32"])}
    Hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
    H = Hk * rng.choice([1, 1, 2, 3, 4])
    d_k, d_v = (rng.choice([128, 128, 64, 8 * spread(2, 16), spread(5, 128)]) for _ in range(2))
    types = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
    c = {"op": op, "H": H, "Hk": Hk, "d_k": d_k, "d_v": d_v, "in": types[0], "out": types[1],
         "per_token": rng.random() < 0.7}
    if op == "decode":
        return {**c, "B": spread(1, max(1, 24576 // H))}
    total, n = spread(1, min(32768, 393216 // H if types[0] == "bf16" else 16384 // H + 1)), spread(1, 48)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if max(lens) * n > 8 * total + 4096:  # keep the padded plain form near the others' cost
        lens = [total // n + (1 if i < total % n else 0) for i in range(n)]
    return {**c, "lens": ",".join(str(x) for x in lens)}


def _axis_of_pair(case):
    """Which row of the positions turns each channel pair: the axes one after the other, the first
    with what does not divide."""
    pairs, axes = case["rot"] // 2, case["axes"]
    return [max(0, (i - pairs % axes) // (pairs // axes)) if pairs >= axes else 0 for i in range(pairs)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = dict(case)
    dt = _TYPES[case["in"]]
    if case["op"] == "rotate":
        T, Hq, Hk, d, rot = case["T"], case["Hq"], case["Hk"], case["d"], case["rot"]
        if case["fused"]:  # queries and keys are parts of one projection's rows, the values behind them
            rows = (1.5 * normal(T, (Hq + 2 * Hk) * d)).to(dt)
            s["q"] = rows[:, :Hq * d].view(T, Hq, d)
            s["k"] = rows[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
        else:
            s["q"], s["k"] = (1.5 * normal(T, Hq, d)).to(dt), (1.5 * normal(T, Hk, d)).to(dt)
        rms = case["norm"] == "rms"
        s["wq"], s["wk"] = (1.0 + 0.1 * normal(d), 1.0 + 0.1 * normal(d)) if rms else (None, None)
        s["inv_freq"] = torch.exp(torch.arange(rot // 2, device="cuda") * (-2.0 / rot * math.log(1e4 if case["axes"] > 1 else 1e6)))
        start = torch.randint(0, case["far"], (1,), device="cuda", generator=g)
        t = torch.arange(T, device="cuda")
        grid = [t] if case["axes"] == 1 else [t // 64, t // 8 % 8, t % 8][:case["axes"]]
        s["positions"] = torch.stack([start + x for x in grid]) if case["axes"] > 1 else start + t
        s["axis"] = _axis_of_pair(case) if case["axes"] > 1 else None
        s["row"] = torch.tensor(s["axis"] or [0] * (rot // 2), device="cuda")
        return s
    H, Hk, d_k, d_v = case["H"], case["Hk"], case["d_k"], case["d_v"]
    if case["op"] == "prefill":
        lens = [int(x) for x in case["lens"].split(",")]
        n, rows = len(lens), sum(lens)
        cu = [sum(lens[:i]) for i in range(n + 1)]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["longest"] = max(lens)
    else:
        n = rows = case["B"]

    def unit(x):  # queries and keys come out of Swish and an L2 norm
        x = x / (1.0 + torch.exp(-x))
        return (x / (x.square().sum(-1, keepdim=True) + _EPS).sqrt()).to(dt)

    s["q"], s["k"] = unit(normal(rows, Hk, d_k)), unit(normal(rows, Hk, d_k))
    s["v"] = normal(rows, H, d_v).to(dt)
    # retention: the first half of the heads forgets within tens of tokens, the others within
    # thousands
    head = torch.where(torch.arange(H, device="cuda") < (H + 1) // 2, 0.1, 0.001)
    s["g"] = -head * torch.log1p(torch.exp(normal(rows, H))) if case["per_token"] else -head * (0.5 + torch.rand(H, device="cuda", generator=g))
    s["beta"] = 1.0 / (1.0 + torch.exp(-normal(rows, H)))
    s["state"] = 0.5 * normal(n, H, d_k, d_v)
    s["scale"] = d_k ** -0.5 * 4.0
    return s


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "rotate": _plain_rotate}[state["op"]](state)


def _own(s):
    from kimi_delta_attention_02_gb300 import binding
    if s["op"] == "prefill":
        return binding.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], s["state"], scale=s["scale"],
                                     out_dtype=_TYPES[s["out"]])
    if s["op"] == "decode":
        out = binding.delta_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"],
                                   out_dtype=_TYPES[s["out"]])
        return out, s["state"]
    return binding.norm_rotate(s["q"], s["k"], s["positions"], s["inv_freq"],
                               norm=None if s["norm"] == "none" else s["norm"], q_weight=s["wq"], k_weight=s["wk"],
                               eps=_EPS, interleaved=s["pairs"] == "neighbours", pair_axis=s["axis"],
                               out_dtype=_TYPES[s["out"]])


def _plain_rotate(s):
    half = s["rot"] // 2
    pos = s["positions"].double().view(s["axes"], -1)[s["row"]].t()
    angle = (pos * s["inv_freq"].double())[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def one(x, w):
        x = x.float()
        if s["norm"] == "rms":
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w
        elif s["norm"] == "l2":
            x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) + _EPS)
        y = x.clone()
        even = s["pairs"] == "neighbours"
        first, second = (slice(0, s["rot"], 2), slice(1, s["rot"], 2)) if even else (slice(0, half), slice(half, s["rot"]))
        y[..., first] = x[..., first] * cos - x[..., second] * sin
        y[..., second] = x[..., second] * cos + x[..., first] * sin
        return y.to(_TYPES[s["out"]])

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _heads(x, H):
    """Query/key heads [rows, Hk, d] as the H value heads read them, in 32 bits."""
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def _plain_decode(s):
    H = s["H"]
    S = s["state"] * torch.exp(s["g"].double()).float()[..., None, None]
    k = _heads(s["k"], H)
    u = s["beta"][..., None] * (s["v"].float() - (k[..., :, None] * S).sum(-2))
    S = S + k[..., :, None] * u[..., None, :]
    out = s["scale"] * (_heads(s["q"], H)[..., :, None] * S).sum(-2)
    s["state"].copy_(S)
    return out.to(_TYPES[s["out"]]), s["state"]


def _plain_prefill(s):
    """The chunked form on sequences padded to the longest: within chunks the triangular system by
    forward substitution, all chunks at once; then the states, a chunk at a time."""
    cu, H, C = s["cu"].long(), s["H"], _CHUNK
    n, N = cu.shape[0] - 1, max(1, -(-s["longest"] // C))
    pos = torch.arange(N * C, device="cuda")
    valid = pos < (cu[1:] - cu[:-1])[:, None]
    tok = torch.where(valid, cu[:-1, None] + pos, 0)

    def padded(x):  # [rows, H, d] -> [n, H, N, C, d], zero behind each sequence
        return (x[tok] * valid[..., None, None]).reshape(n, N, C, H, x.shape[-1]).permute(0, 3, 1, 2, 4)

    q, k, v = padded(_heads(s["q"], H)), padded(_heads(s["k"], H)), padded(s["v"].float())
    beta = padded(s["beta"][..., None])
    g = s["g"].double()
    g = (g[tok] if g.ndim == 2 else g.expand(n, N * C, H)) * valid[..., None]
    G = g.permute(0, 2, 1).reshape(n, H, N, C).cumsum(-1)
    i = torch.arange(C, device="cuda")
    D = torch.exp(torch.where(i[:, None] >= i, G[..., :, None] - G[..., None, :], -math.inf)).float()
    A = beta * (k @ k.transpose(-1, -2)) * D * (i[:, None] > i)
    eG = torch.exp(G).float()[..., None]
    rest = torch.exp(G[..., -1:] - G).float()[..., None]
    end = torch.exp(G[..., -1]).float()[..., None, None]
    # (I + A) [Uv, W] = beta [v, e^G k], a row at a time
    X = torch.cat([v, eG * k], -1) * beta
    for t in range(1, C):
        X[..., t, :] -= (A[..., t, None, :t] @ X[..., :t, :])[..., 0, :]
    Uv, W = X[..., :s["d_v"]], X[..., s["d_v"]:]
    P = (q @ k.transpose(-1, -2)) * D
    q, k = eG * q, rest * k
    S = s["state"]
    out = torch.empty_like(v)
    for c in range(N):
        u = Uv[:, :, c] - W[:, :, c] @ S
        out[:, :, c] = q[:, :, c] @ S + P[:, :, c] @ u
        S = end[:, :, c] * S + k[:, :, c].transpose(-1, -2) @ u
    t = torch.arange(s["v"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    out = (s["scale"] * out).permute(0, 2, 3, 1, 4).reshape(n, N * C, H, -1)[seq, t - cu[seq]]
    return out.to(_TYPES[s["out"]]), S


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "rotate":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
        return {"bytes": n * (size[case["in"]] + size[case["out"]]) + 8 * case["axes"] * case["T"] + 2 * case["rot"]
                + (8 * case["d"] if case["norm"] == "rms" else 0),
                "flops": n * (4 if case["norm"] != "none" else 0) + 3 * case["T"] * (case["Hq"] + case["Hk"]) * case["rot"]}
    n, rows = (case["B"],) * 2 if case["op"] == "decode" else (case["lens"].count(",") + 1, sum(int(x) for x in case["lens"].split(",")))
    H, Hk, d_k, d_v = case["H"], case["Hk"], case["d_k"], case["d_v"]
    return {"bytes": rows * (2 * Hk * d_k + H * d_v) * size[case["in"]] + rows * H * d_v * size[case["out"]]
            + 4 * H * (rows if case["per_token"] else 1) + 4 * H * rows + 2 * n * H * d_k * d_v * 4,
            "flops": 6.0 * rows * H * d_k * d_v}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        d, rot = case["d"], case["rot"]
        axis = torch.tensor(_axis_of_pair(case), device="cuda")
        pos = s["positions"].double().reshape(case["axes"], -1)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[axis].T * s["inv_freq"].double())

        def one(x, w):
            x = x.double()
            if case["norm"] != "none":
                power = (x * x).sum(-1, keepdim=True) / (d if case["norm"] == "rms" else 1)
                x = x / torch.sqrt(power + _EPS)
            if w is not None:
                x = x * w.double()
            z, rest = x[..., :rot], x[..., rot:]
            if case["pairs"] == "neighbours":
                z = torch.view_as_complex(z.reshape(*z.shape[:-1], rot // 2, 2).contiguous()) * turn[:, None]
                return torch.cat([torch.view_as_real(z).flatten(-2), rest], -1)
            z = torch.complex(z[..., :rot // 2], z[..., rot // 2:]) * turn[:, None]
            return torch.cat([z.real, z.imag, rest], -1)

        return one(s["q"], s["wq"]), one(s["k"], s["wk"])
    # the recurrence itself, a token at a time: decode is n sequences of one token
    H, d_k, d_v = case["H"], case["d_k"], case["d_v"]
    rows = s["v"].shape[0]
    lens = [1] * rows if case["op"] == "decode" else [int(x) for x in case["lens"].split(",")]
    first = torch.tensor([sum(lens[:i]) for i in range(len(lens))], device="cuda")
    length = torch.tensor(lens, device="cuda")
    group = torch.arange(H, device="cuda") // (H // case["Hk"])
    S = s["state"].double()
    out = torch.zeros(rows, H, d_v, dtype=torch.float64, device="cuda")
    alpha = torch.exp(s["g"].double()).expand(rows, H)
    for t in range(max(lens)):
        on = (length > t).nonzero()[:, 0] if len(lens) > 1 else slice(None)
        row = (first + t)[on]
        k = s["k"][row].double()[:, group]
        S_on = S[on] * alpha[row][..., None, None]
        miss = s["v"][row].double() - torch.einsum("bhk,bhkv->bhv", k, S_on)
        S_on += k[..., :, None] * (s["beta"][row].double()[..., None] * miss)[..., None, :]
        out[row] = s["scale"] * torch.einsum("bhk,bhkv->bhv", s["q"][row].double()[:, group], S_on)
        S[on] = S_on
    return out, S
