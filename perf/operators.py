"""Measured cases of the linear-attention operators and of the block norm.

Three operators, each in its plain form (elementary torch operations in 32 bits, 64 for the decay
sums, rounded once at the end) and as the calls a user makes of the binding:

``prefill``  linear attention with one decay per head over packed sequences, per sequence and head
             S_t = a_t S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  a_t = e^{g_t};
             head h reads query/key head h // (H // Hk). ``binding.linear_prefill``.
``decode``   one token of the same recurrence for B sequences, states updated in place.
             ``binding.linear_decode``.
``norm``     between two blocks of a residual stream x with block output y:
             x' = x + scale c (*) Sigmoid(r) (*) (w_post (*) y / rms(y)),  h = w_pre (*) x' / rms(x').
             ``binding.block_norm``.
"""

import math

import torch

own = False

_CHUNK = 128  # tokens per chunk of the plain prefill
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    def prefill(name, lens, H, Hk, d_k, d_v, types, per_token):
        return {"name": name, "op": "prefill", "lens": lens, "H": H, "Hk": Hk, "d_k": d_k, "d_v": d_v, "in": types[0],
                "out": types[1], "per_token": per_token}

    b, f = ("bf16", "bf16"), ("fp32", "fp32")
    return [
        # three short prompts of a server that has nothing else to do: latency
        prefill("prefill_short", "1,17,46", 8, 8, 128, 128, b, True),
        # one layer's prompt at this repository's headline sizes (T = 4096, H = 96, d = 128)
        prefill("prefill_layer", "4096", 96, 96, 128, 128, b, True),
        # ragged prompts packed together, query/key heads shared by four value heads of 64
        # channels, fp32 read-out
        prefill("prefill_packed", "3001,0,517,1024,129,4096,1,2222", 32, 8, 128, 64, ("bf16", "fp32"), True),
        # one long document on few heads, a constant decay for each head
        prefill("prefill_long", "65536", 16, 16, 128, 128, b, False),
        # many short requests admitted at once
        prefill("prefill_many", ",".join(str(40 + 37 * i % 211) for i in range(64)), 16, 4, 128, 128, b, True),
        # reference accuracy: fp32 in and out, odd head sizes
        prefill("prefill_fp32", "700,333", 6, 2, 100, 72, f, True),
        # one user's next token
        {"name": "decode_one", "op": "decode", "B": 1, "H": 96, "Hk": 96, "d_k": 128, "d_v": 128, "in": "bf16",
         "out": "bf16", "per_token": True},
        # a full batch at this repository's decode sizes (B = 256, H = 96)
        {"name": "decode_batch", "op": "decode", "B": 256, "H": 96, "Hk": 96, "d_k": 128, "d_v": 128, "in": "bf16",
         "out": "fp32", "per_token": True},
        # an odd batch, shared query/key heads, fp32, a constant decay for each head
        {"name": "decode_shared", "op": "decode", "B": 37, "H": 24, "Hk": 8, "d_k": 100, "d_v": 72, "in": "fp32",
         "out": "fp32", "per_token": False},
        # one token between two blocks of the 7168-channel residual stream
        {"name": "norm_one", "op": "norm", "T": 1, "D": 7168, "x": "bf16", "y": "bf16", "gate": "channel",
         "post": True, "channel_scale": True},
        # a prompt: fp32 residual stream, bf16 blocks, channel gate
        {"name": "norm_prompt", "op": "norm", "T": 4096, "D": 7168, "x": "fp32", "y": "bf16", "gate": "channel",
         "post": True, "channel_scale": True},
        # odd row length (rows that start off 16-byte boundaries), one gate per token, no norm after the block
        {"name": "norm_odd", "op": "norm", "T": 777, "D": 1001, "x": "bf16", "y": "bf16", "gate": "token",
         "post": False, "channel_scale": False},
    ]


def draw(rng):
    def spread(lo, hi):  # over the logarithm
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "norm", "norm"])
    if op == "norm":
        D = rng.choice([spread(17, 8192), 8 * spread(8, 1024)])
        return {"op": op, "T": spread(1, max(1, 29360128 // D)), "D": D, "x": rng.choice(["bf16", "fp32"]),
                "y": rng.choice(["bf16", "bf16", "fp32"]), "gate": rng.choice(["channel", "token", "none"]),
                "post": rng.random() < 0.7, "channel_scale": rng.random() < 0.5}
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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = dict(case)
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        # the residual stream has grown over the layers below; block outputs are about one
        s["x"] = (4.0 * normal(T, D)).to(_TYPES[case["x"]])
        s["y"] = normal(T, D).to(_TYPES[case["y"]])
        s["r"] = {"channel": lambda: normal(T, D), "token": lambda: normal(T), "none": lambda: None}[case["gate"]]()
        s["r"] = None if s["r"] is None else s["r"].to(_TYPES[case["y"]])
        s["w_post"] = 1.0 + 0.1 * normal(D) if case["post"] else None
        s["c"] = 0.5 + 0.1 * normal(D) if case["channel_scale"] else None
        s["w_pre"] = 1.0 + 0.1 * normal(D)
        return s
    H, Hk, d_k, d_v, dt = case["H"], case["Hk"], case["d_k"], case["d_v"], _TYPES[case["in"]]
    if case["op"] == "prefill":
        lens = [int(x) for x in case["lens"].split(",")]
        n, rows = len(lens), sum(lens)
        cu = [sum(lens[:i]) for i in range(n + 1)]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["longest"] = max(lens)
    else:
        n = rows = case["B"]
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    s["q"], s["k"] = unit(normal(rows, Hk, d_k)).to(dt), unit(normal(rows, Hk, d_k)).to(dt)
    s["v"] = normal(rows, H, d_v).to(dt)
    # retention: the first half of the heads forgets within tens of tokens, the others within
    # thousands
    head = torch.where(torch.arange(H, device="cuda") < (H + 1) // 2, 0.1, 0.001)
    s["g"] = -head * torch.log1p(torch.exp(normal(rows, H))) if case["per_token"] else -head * (0.5 + torch.rand(H, device="cuda", generator=g))
    s["state"] = 0.5 * normal(n, H, d_k, d_v)
    s["scale"] = d_k ** -0.5 * 4.0
    return s


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "norm": _plain_norm}[state["op"]](state)


def _own(s):
    from kimi_delta_attention_02_gb300 import binding
    if s["op"] == "prefill":
        return binding.linear_prefill(s["q"], s["k"], s["v"], s["g"], s["cu"], s["state"], scale=s["scale"],
                                      out_dtype=_TYPES[s["out"]])
    if s["op"] == "decode":
        out = binding.linear_decode(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"],
                                    out_dtype=_TYPES[s["out"]])
        return out, s["state"]
    return binding.block_norm(s["x"], s["y"], gate=s["r"], post_norm=s["post"], post_weight=s["w_post"], scale=0.7,
                              channel_scale=s["c"], pre_weight=s["w_pre"], eps=1e-6, out_dtype=_TYPES["bf16"])


def _plain_norm(s):
    u = s["y"].float()
    if s["post"]:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-6) * s["w_post"]
    if s["r"] is not None:
        r = s["r"].float()
        u = u / (1.0 + torch.exp(-(r if r.ndim == 2 else r[:, None])))
    if s["c"] is not None:
        u = u * s["c"]
    x = s["x"].float() + 0.7 * u
    h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["w_pre"]
    return x.to(s["x"].dtype), h.to(torch.bfloat16)


def _heads(x, H):
    """Query/key heads [rows, Hk, d] as the H value heads read them, in 32 bits."""
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def _plain_decode(s):
    H = s["H"]
    a = torch.exp(s["g"].double()).float()
    S = s["state"] * a[..., None, None] + _heads(s["k"], H)[..., :, None] * s["v"].float()[..., None, :]
    out = s["scale"] * (_heads(s["q"], H)[..., :, None] * S).sum(-2)
    s["state"].copy_(S)
    return out.to(_TYPES[s["out"]]), s["state"]


def _plain_prefill(s):
    """The chunked form on sequences padded to the longest: products within chunks, the chunks'
    states joined through the matrix of decays between chunks."""
    cu, H, C = s["cu"].long(), s["H"], _CHUNK
    n, N = cu.shape[0] - 1, max(1, -(-s["longest"] // C))
    pos = torch.arange(N * C, device="cuda")
    valid = pos < (cu[1:] - cu[:-1])[:, None]
    tok = torch.where(valid, cu[:-1, None] + pos, 0)

    def padded(x):  # [rows, H, d] -> [n, H, N, C, d], zero behind each sequence
        return (x[tok] * valid[..., None, None]).reshape(n, N, C, H, x.shape[-1]).permute(0, 3, 1, 2, 4)

    q, k, v = padded(_heads(s["q"], H)), padded(_heads(s["k"], H)), padded(s["v"].float())
    g = s["g"].double()
    g = (g[tok] if g.ndim == 2 else g.expand(n, N * C, H)) * valid[..., None]
    G = g.permute(0, 2, 1).cumsum(-1).reshape(n, H, N, C)
    end = G[..., -1]
    start = torch.cat([torch.zeros_like(end[..., :1]), end[..., :-1]], -1)
    i = torch.arange(max(C, N), device="cuda")
    low = i[:C, None] >= i[:C]
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
    out = ((q @ k.transpose(-1, -2)) * D) @ v
    U = ((k * torch.exp(end[..., None] - G).float()[..., None]).transpose(-1, -2) @ v).flatten(-2)
    W = torch.exp(torch.where(i[:N, None] > i[:N], start[..., :, None] - end[..., None, :], -math.inf)).float()
    S0 = s["state"].flatten(-2)
    S = (W @ U + torch.exp(start).float()[..., None] * S0[:, :, None]).unflatten(-1, (s["d_k"], s["d_v"]))
    out = out + (q * torch.exp(G - start[..., None]).float()[..., None]) @ S
    last = torch.exp(end[..., -1:] - end).float()
    final = torch.exp(end[..., -1]).float()[..., None] * S0 + (last[..., None, :] @ U)[..., 0, :]
    t = torch.arange(s["v"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    out = (s["scale"] * out).permute(0, 2, 3, 1, 4).reshape(n, N * C, H, -1)[seq, t - cu[seq]]
    return out.to(_TYPES[s["out"]]), final.reshape(s["state"].shape)


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        rows = 2 * size[case["x"]] + size[case["y"]] * (2 if case["gate"] == "channel" else 1) + 2
        return {"bytes": T * D * rows + (T * size[case["y"]] if case["gate"] == "token" else 0) + 12 * D,
                "flops": 12 * T * D}
    n, rows = (case["B"],) * 2 if case["op"] == "decode" else (case["lens"].count(",") + 1, sum(int(x) for x in case["lens"].split(",")))
    H, Hk, d_k, d_v = case["H"], case["Hk"], case["d_k"], case["d_v"]
    return {"bytes": rows * (2 * Hk * d_k + H * d_v) * size[case["in"]] + rows * H * d_v * size[case["out"]]
            + 4 * H * (rows if case["per_token"] else 1) + 2 * n * H * d_k * d_v * 4,
            "flops": 4.0 * rows * H * d_k * d_v}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        y, x = s["y"].double(), s["x"].double()
        if case["post"]:
            y = s["w_post"].double() * y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["D"] + 1e-6)
        if case["gate"] != "none":
            y = torch.sigmoid(s["r"].double().reshape(case["T"], -1)) * y
        if case["channel_scale"]:
            y = y * s["c"].double()
        x = x + 0.7 * y
        return x, s["w_pre"].double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + 1e-6)
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
        S_on = S[on] * alpha[row][..., None, None]
        S_on += s["k"][row].double()[:, group][..., :, None] * s["v"][row].double()[..., None, :]
        out[row] = s["scale"] * torch.einsum("bhk,bhkv->bhv", s["q"][row].double()[:, group], S_on)
        S[on] = S_on
    return out, S
