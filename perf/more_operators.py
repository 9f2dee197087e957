"""Measured cases of linear attention with a decay a head and of the norms around a block.

Operators that a serving engine calls beside the recurrent-state calls, for the layers whose state
decays by one factor a head and token, and for the norms that join any two layers:

  prefill   chunked linear attention of packed sequences, states read from and written to a pool
  decode    the recurrent form: 1..16 positions a request over that pool; as a step (outputs and new
            states), as a speculative verify (outputs only) or as its commit (states only)
  gated     each head's row normalised and multiplied by its activated gate
  residual  norm after a block, gate, residual sum, norm before the next block

run() with own = False computes the definitions with elementary torch operations in fp32;
with own = True it makes the library's calls on the same state.
"""
import math

import torch

own = False

D = 128  # key and value channels of a head
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6
ALPHA, BETA = 1.0, 0.25  # of the residual sum
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def _spread(n, mean, low=0.5):
    """n ragged lengths around mean, from low*mean to (2-low)*mean, the same for every seed."""
    return [max(1, int(mean * (low + (2 - 2 * low) * math.modf((i + 1) * 0.6180339887)[0]))) for i in range(n)]


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # three short prompts on a tensor-parallel head slice: latency of one layer
        dict(name="prefill_3x70_h2", op="prefill", seqs=3, length=70, heads=2, key_heads=2, decay="head", init=False,
             dtype="bf16", state="f32"),
        # a packed batch of ragged prompts that continue cached prefixes, gated per token
        dict(name="prefill_8x5182_h32", op="prefill", seqs=8, length=5182, heads=32, key_heads=32, decay="token",
             init=True, dtype="bf16", state="f32"),
        # one long prompt, fixed slopes a head
        dict(name="prefill_1x131072_h16", op="prefill", seqs=1, length=131072, heads=16, key_heads=16, decay="head",
             init=False, dtype="bf16", state="f32"),
        # long prompts on a head slice whose heads share one key head
        dict(name="prefill_4x32768_h4_k1", op="prefill", seqs=4, length=32768, heads=4, key_heads=1, decay="token",
             init=True, dtype="f16", state="f32"),
        # a single user's token: latency of one layer
        dict(name="decode_1_h16", op="decode", mode="step", requests=1, k=1, heads=16, key_heads=16, decay="token",
             dtype="bf16", state="f32"),
        # a full decode batch
        dict(name="decode_256_h32", op="decode", mode="step", requests=256, k=1, heads=32, key_heads=32, decay="token",
             dtype="bf16", state="f32"),
        # the verify step of speculative decoding, seven positions a request
        dict(name="verify_64x7_h32", op="decode", mode="verify", requests=64, k=7, heads=32, key_heads=32,
             decay="token", dtype="bf16", state="f32"),
        # the commit of its accepted tokens
        dict(name="commit_64x7_h32", op="decode", mode="commit", requests=64, k=7, heads=32, key_heads=32,
             decay="token", dtype="bf16", state="f32"),
        # the attention's rows of a full decode batch
        dict(name="gated_256x32x128", op="gated", rows=256, heads=32, dim=128, gate="sigmoid", dtype="bf16"),
        # and of a packed prefill
        dict(name="gated_41460x32x128", op="gated", rows=41460, heads=32, dim=128, gate="silu", dtype="bf16"),
        # between two blocks of a single token
        dict(name="residual_1x4096", op="residual", rows=1, dim=4096, post=True, gate="none", dtype="bf16"),
        # and of a packed prefill, with a learned scale a channel
        dict(name="residual_41460x4096", op="residual", rows=41460, dim=4096, post=True, gate="channel", dtype="bf16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "decode", "gated", "residual"])
    heads = rng.choice([1, 2, 3, 4, 8, 16, 24, 32, 40, 64])
    key_heads = rng.choice([heads, heads, 1, heads // 2 if heads % 2 == 0 else heads])
    decay, state = rng.choice(["head", "token", "both"]), rng.choice(["f32", "f32", "bf16", "f16"])
    if op == "prefill":
        seqs = _log(rng, 1, 16)
        length = _log(rng, 1, max(1, min(131072, (1 << 21) // heads) // seqs))
        return dict(op=op, seqs=seqs, length=length, heads=heads, key_heads=key_heads, decay=decay,
                    init=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f16"]), state=state)
    if op == "decode":
        k = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
        return dict(op=op, mode=rng.choice(["step", "verify", "commit"]) if k > 1 else "step",
                    requests=_log(rng, 1, 8192 // heads), k=k, heads=heads, key_heads=key_heads, decay=decay,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), state=state)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "gated":
        dim = rng.choice([D, D, 64, 80, 256, 129, _log(rng, 8, 8192)])
        heads = heads if dim <= 512 else 1
        rows = _log(rng, 1, min(41460, (41460 * 32 * D) // (2 * heads * dim)))
        return dict(op=op, rows=rows, heads=heads, dim=dim, gate=rng.choice(["none", "sigmoid", "silu"]), dtype=dtype)
    dim = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 8, 2048)])
    return dict(op=op, rows=_log(rng, 1, min(41460, (41460 * 2048) // dim)), dim=dim, post=rng.random() < 0.6,
                gate=rng.choice(["none", "channel", "token"]), dtype=dtype)


def _lengths(case):
    return _spread(case["seqs"], case["length"]) if case["seqs"] > 1 else [case["length"]]


# ------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, std=1.0, unit=False):
    """Normal values, or rows of unit length, drawn in pieces."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    rows = out.view(-1, shape[-1])
    step = max(1, (1 << 27) // shape[-1])
    for i in range(0, rows.shape[0], step):
        x = torch.randn(rows[i:i + step].shape, generator=g, device="cuda")
        rows[i:i + step] = x / x.norm(dim=1, keepdim=True) if unit else x.mul_(std)
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _decays(case, g, rows):
    """(log decay a head, log decay a row and head), either None."""
    H = case["heads"]
    head = token = None
    if case["decay"] != "token":  # slopes in a geometric series over the heads
        head = -torch.exp2(-8 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)
    if case["decay"] != "head":  # a gate that mostly keeps, and now and then lets go
        x = torch.randn(rows, H, generator=g, device="cuda")
        token = -torch.nn.functional.softplus(1.5 * x - 3)
        token[torch.rand(rows, H, generator=g, device="cuda") < 1e-3] = -20.0
    return head, token


def prepare(case, seed):
    return globals()["_prepare_" + case["op"]](case, _gen(seed))


def _rows_of_heads(case, g, rows, s):
    dt, H, Hk = TYPES[case["dtype"]], case["heads"], case["key_heads"]
    s["q"] = _randn(g, (rows, Hk, D), dt, unit=True)
    s["k"] = _randn(g, (rows, Hk, D), dt, unit=True)
    s["v"] = _randn(g, (rows, H, D), dt)
    s["head"], s["token"] = _decays(case, g, rows)
    s["out"] = torch.zeros(rows, H, D, dtype=dt, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _prepare_prefill(case, g):
    lens = _lengths(case)
    N, T = len(lens), sum(lens)
    s = dict(case=case, cu=_i32([sum(lens[:i]) for i in range(N + 1)]), lens=lens)
    _rows_of_heads(case, g, T, s)
    # slots of the cached prefixes first, in another order than the sequences, then the new states'
    order = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    s["pool"] = _randn(g, (2 * N, case["heads"], D, D), TYPES[case["state"]], 0.1)
    s["init"] = order if case["init"] else None
    s["final"] = N + order
    return s


def _prepare_decode(case, g):
    R, K = case["requests"], case["k"]
    s = dict(case=case)
    _rows_of_heads(case, g, R * K, s)
    s["pool"] = _randn(g, (R + 2, case["heads"], D, D), TYPES[case["state"]], 0.1)
    s["slot"] = torch.randperm(R + 2, generator=g, device="cuda")[:R].to(torch.int32)
    s["commit"] = torch.randint(1, K + 1, (R,), generator=g, device="cuda").to(torch.int32)
    s["nothing"] = torch.zeros(R, dtype=torch.int32, device="cuda")
    return s


def _prepare_gated(case, g):
    R, H, d, dt = case["rows"], case["heads"], case["dim"], TYPES[case["dtype"]]
    return dict(case=case, x=_randn(g, (R, H, d), dt, 0.3), weight=1 + _randn(g, (d,), dt, 0.1),
                gate=None if case["gate"] == "none" else _randn(g, (R, H, d), dt, 1.5),
                out=torch.empty(R, H, d, dtype=dt, device="cuda"))


def _prepare_residual(case, g):
    R, d, dt = case["rows"], case["dim"], TYPES[case["dtype"]]
    gate = {"none": None, "channel": (1, d), "token": (R, d)}[case["gate"]]
    return dict(case=case, x=_randn(g, (R, d), dt, 0.5), residual=_randn(g, (R, d), dt, 2.0),
                post=1 + _randn(g, (d,), dt, 0.1) if case["post"] else None, weight=1 + _randn(g, (d,), dt, 0.1),
                gate=None if gate is None else _randn(g, gate, dt),
                hidden=torch.empty(R, d, dtype=dt, device="cuda"), out=torch.empty(R, d, dtype=dt, device="cuda"))


# ------------------------------------------------------------------------------ one pass


def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _log_decay(s, rows):
    """Log decays [rows, H], not above 0."""
    H = s["case"]["heads"]
    g = torch.zeros(rows, H, device=s["v"].device)
    if s["head"] is not None:
        g = g + s["head"]
    if s["token"] is not None:
        g = g + s["token"]
    return g.clamp_max(0)


def _plain_prefill(s, C=128):
    c = s["case"]
    N, H, rep, dev = c["seqs"], c["heads"], c["heads"] // c["key_heads"], s["q"].device
    T, longest = s["q"].shape[0], max(s["lens"])
    cu = s["cu"].long()
    g = _log_decay(s, T)
    at = torch.arange(C, device=dev)
    causal = at[:, None] >= at[None, :]
    S = torch.zeros(N, H, D, D, device=dev)  # transposed: [value, key], as the pool holds it
    if s["init"] is not None:
        S = s["pool"][s["init"].long()].float()
    for first in range(0, longest, C):
        row = cu[:-1, None] + first + at
        live = row < cu[1:, None]
        row = row.clamp_max(T - 1)
        q, k, v = (s[n][row].float().transpose(1, 2) for n in "qkv")  # [N, heads, C, D]
        if rep > 1:
            q, k = q.repeat_interleave(rep, dim=1), k.repeat_interleave(rep, dim=1)
        keep = live[:, None, :, None]
        k, v = k * keep, v * keep
        # differences of long sums: in 64 bits
        G = (g[row] * live[:, :, None]).transpose(1, 2).double().cumsum(2)
        w = torch.exp((G[..., :, None] - G[..., None, :]).clamp_max(0).float()) * causal
        e, f = torch.exp(G.float())[..., None], torch.exp((G[..., -1:] - G).float())[..., None]
        o = torch.matmul(torch.matmul(q, k.transpose(2, 3)) * w, v) + torch.matmul(q, S.transpose(2, 3)) * e
        s["out"][row[live]] = (o.transpose(1, 2)[live] * SCALE).to(s["out"].dtype)
        S = S * e[..., -1:, :] + torch.matmul(v.transpose(2, 3), k * f)
    s["pool"][s["final"].long()] = S.to(s["pool"].dtype)
    return {"out": s["out"], "pool": s["pool"]}


def _plain_decode(s):
    c = s["case"]
    R, K, H, rep = c["requests"], c["k"], c["heads"], c["heads"] // c["key_heads"]
    q, k, v = (s[n].float().view(R, K, -1, D) for n in "qkv")
    if rep > 1:
        q, k = q.repeat_interleave(rep, dim=2), k.repeat_interleave(rep, dim=2)
    a = torch.exp(_log_decay(s, R * K)).view(R, K, H)
    slot = s["slot"].long()
    S = s["pool"][slot].float()
    new = S
    out = torch.empty(R, K, H, D, device=S.device)
    for t in range(K):
        S = S * a[:, t, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
        if c["mode"] != "commit":
            out[:, t] = (S * q[:, t, :, None, :]).sum(-1) * SCALE
        if c["mode"] != "verify":
            new = torch.where((s["commit"] > t)[:, None, None, None], S, new) if c["mode"] == "commit" else S
    res = {}
    if c["mode"] != "commit":
        s["out"].copy_(out.view(R * K, H, D))
        res["out"] = s["out"]
    if c["mode"] != "verify":
        s["pool"][slot] = new.to(s["pool"].dtype)
        res["pool"] = s["pool"]
    return res


def _norm(x, weight):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()


def _plain_gated(s):
    y = _norm(s["x"].float(), s["weight"])
    if s["gate"] is not None:
        z = s["gate"].float()
        act = 1 / (1 + torch.exp(-z))
        y = y * (act * z if s["case"]["gate"] == "silu" else act)
    return {"out": y.to(s["out"].dtype)}


def _plain_residual(s):
    z = s["x"].float()
    if s["post"] is not None:
        z = _norm(z, s["post"])
    if s["gate"] is not None:
        z = z * s["gate"].float()
    h = ALPHA * s["residual"].float() + BETA * z
    return {"hidden": h.to(s["hidden"].dtype), "out": _norm(h, s["weight"]).to(s["out"].dtype)}


def _own_prefill(s):
    import serving_kda_chunk_gb300 as kda

    if "workspace" not in s:  # kept by the program from call to call
        s["workspace"] = torch.empty(kda.kda_decay_prefill_workspace_size(s["q"].shape[0], s["case"]["seqs"],
                                                                          s["case"]["heads"]),
                                     dtype=torch.uint8, device="cuda")
    kda.kda_decay_prefill(s["q"], s["k"], s["v"], s["cu"], s["out"], head_decay=s["head"], log_decay=s["token"],
                          state_pool=s["pool"], init_slot=s["init"], final_slot=s["final"], scale=SCALE,
                          workspace=s["workspace"], dev_status=s["status"])
    return {"out": s["out"], "pool": s["pool"]}


def _own_decode(s):
    import serving_kda_chunk_gb300 as kda

    mode = s["case"]["mode"]
    kda.kda_decay_decode(s["q"], s["k"], s["v"], s["pool"], s["slot"], None if mode == "commit" else s["out"],
                         K=s["case"]["k"], n_commit={"step": None, "verify": s["nothing"], "commit": s["commit"]}[mode],
                         head_decay=s["head"], log_decay=s["token"], scale=SCALE, dev_status=s["status"])
    res = {} if mode == "commit" else {"out": s["out"]}
    if mode != "verify":
        res["pool"] = s["pool"]
    return res


def _own_gated(s):
    import serving_kda_chunk_gb300 as kda

    kda.kda_gated_norm(s["x"], s["out"], gate=s["gate"], weight=s["weight"], eps=EPS,
                       act=kda.KDA_ACT_SILU if s["case"]["gate"] == "silu" else kda.KDA_ACT_SIGMOID)
    return {"out": s["out"]}


def _own_residual(s):
    import serving_kda_chunk_gb300 as kda

    kda.kda_residual_norm(s["x"], s["residual"], hidden=s["hidden"], out=s["out"], post_weight=s["post"],
                          gate=s["gate"], weight=s["weight"], residual_scale=ALPHA, branch_scale=BETA, eps=EPS)
    return {"hidden": s["hidden"], "out": s["out"]}


# ------------------------------------------------------------------------------ what a pass cannot do without


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] in ("prefill", "decode"):
        H, Hk, state = case["heads"], case["key_heads"], D * D * SIZE[case["state"]]
        gate = 4 * H if case["decay"] != "head" else 0
    if case["op"] == "prefill":
        T, units = sum(_lengths(case)), case["seqs"] * H
        return {"bytes": T * ((2 * Hk + 2 * H) * D * b + gate) + units * state * (2 if case["init"] else 1),
                "flops": T * H * 4 * D * D}
    if case["op"] == "decode":
        R, rows, mode = case["requests"], case["requests"] * case["k"], case["mode"]
        tokens = rows if mode != "commit" else R * (case["k"] + 1) // 2  # of a commit, those accepted on average
        acts = tokens * ((2 * Hk + 2 * H) * D * b + gate) if mode != "commit" else tokens * ((Hk + H) * D * b + gate)
        return {"bytes": acts + R * H * state * (1 if mode == "verify" else 2) + 4 * R,
                "flops": tokens * H * 2 * D * D * (2 if mode == "step" else 1)}
    rows = case["rows"] * case.get("heads", 1)
    d = case["dim"]
    if case["op"] == "gated":
        return {"bytes": rows * d * b * (2 if case["gate"] == "none" else 3) + d * b, "flops": 8 * rows * d}
    gate = {"none": 0, "channel": 1, "token": rows}[case["gate"]]
    return {"bytes": (4 * rows + gate + 1 + case["post"]) * d * b, "flops": 12 * rows * d}


# ------------------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _recur(S, q, k, v, g):
    """The recurrence over axis 1 of [batch, steps, heads, D]: outputs and the last state [.., key, value]."""
    outs, a = [], g.exp()
    for t in range(q.shape[1]):
        S = torch.addcmul(S * a[:, t, :, None, None], k[:, t, :, :, None], v[:, t, :, None, :])
        outs.append((S * q[:, t, :, :, None]).sum(-2))
    return torch.stack(outs, 1) * SCALE, S


def _wide(s, name, rows):
    x = s[name][rows].double()
    return x if name == "v" else x.repeat_interleave(s["case"]["heads"] // s["case"]["key_heads"], dim=-2)


def _gates(s, rows):
    g = torch.zeros(*rows.shape, s["case"]["heads"], dtype=torch.float64, device="cuda")
    for x in (s["head"], None if s["token"] is None else s["token"][rows]):
        if x is not None:
            g = g + x.double()
    return g.clamp_max(0)


def _exact_prefill(s):
    N, H = s["case"]["seqs"], s["case"]["heads"]
    cu, lens = s["cu"].tolist(), torch.tensor(s["lens"], device="cuda")
    pool = s["pool"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    S = torch.zeros(N, H, D, D, dtype=torch.float64, device="cuda")
    if s["init"] is not None:
        S = pool[s["init"].long()].transpose(2, 3).contiguous()
    start = torch.tensor(cu[:-1], device="cuda")
    for first in range(0, max(s["lens"]), 256):
        steps = first + torch.arange(min(256, max(s["lens"]) - first), device="cuda")
        inside = steps[None, :] < lens[:, None]
        rows = torch.where(inside, start[:, None] + steps, 0)
        m = inside[:, :, None]
        o, S = _recur(S, _wide(s, "q", rows), _wide(s, "k", rows) * m[..., None], _wide(s, "v", rows), _gates(s, rows) * m)
        out[rows[inside]] = o[inside]
    pool[s["final"].long()] = S.transpose(2, 3)
    return {"out": out, "pool": pool}


def _exact_decode(s):
    c = s["case"]
    R, K = c["requests"], c["k"]
    rows = torch.arange(R * K, device="cuda").view(R, K)
    slot, pool = s["slot"].long(), s["pool"].double()
    S = pool[slot].transpose(2, 3)
    parts = [_wide(s, n, rows) for n in "qkv"]
    g = _gates(s, rows)
    res = {}
    if c["mode"] != "commit":
        o, last = _recur(S, *parts, g)
        res["out"] = o.reshape(R * K, c["heads"], D)
    else:  # rows past the accepted ones change nothing
        taken = (torch.arange(K, device="cuda")[None, :] < s["commit"].long()[:, None])[:, :, None]
        _, last = _recur(S, parts[0], parts[1] * taken[..., None], parts[2], g * taken)
    if c["mode"] != "verify":
        pool[slot] = last.transpose(2, 3)
        res["pool"] = pool
    return res


def _unit(x):
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()


def _exact_gated(s):
    out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    for i in range(0, out.shape[0], 4096):
        y = _unit(s["x"][i:i + 4096].double()) * s["weight"].double()
        if s["gate"] is not None:
            z = s["gate"][i:i + 4096].double()
            y = y * torch.sigmoid(z)
            if s["case"]["gate"] == "silu":
                y = y * z
        out[i:i + 4096] = y
    return {"out": out}


def _exact_residual(s):
    hidden, out = (torch.empty(s["x"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, hidden.shape[0], 4096):
        z = s["x"][i:i + 4096].double()
        if s["post"] is not None:
            z = _unit(z) * s["post"].double()
        if s["gate"] is not None:
            z = z * (s["gate"] if s["gate"].shape[0] == 1 else s["gate"][i:i + 4096]).double()
        hidden[i:i + 4096] = ALPHA * s["residual"][i:i + 4096].double() + BETA * z
        out[i:i + 4096] = _unit(hidden[i:i + 4096]) * s["weight"].double()
    return {"hidden": hidden, "out": out}
