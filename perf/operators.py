"""Measured cases of the latent-attention and token-log-probability operators.

Four operators that a serving engine with recurrent-state layers calls next to them, for the
full-attention layers of the same model and for what it answers with:

  append    one latent vector and rope key a token, normalised, written into a paged cache
  decode    absorbed latent attention of 1..16 query positions a request over that cache
  prefill   expanded latent attention of packed sequences, causal behind an earlier context
  logprobs  log probability of given tokens, entropy and the top alternatives of each row

run() with own = False computes the definitions with elementary torch operations in fp32;
with own = True it makes the library's calls on the same state.
"""
import math
import random

import torch

own = False

RANK, ROPE, NOPE, DV = 512, 64, 128, 128  # latent, rope key, per-head key and value widths
WIDTH = RANK + ROPE
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _bytes(case):
    return 4 if case["dtype"] == "f32" else 2


def _spread(n, mean, low=0.5):
    """n ragged lengths around mean, from low*mean to (2-low)*mean, the same for every seed."""
    return [max(1, int(mean * (low + (2 - 2 * low) * math.modf((i + 1) * 0.6180339887)[0]))) for i in range(n)]


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step's tokens of a full batch, appended to the cache
        dict(name="append_decode_256", op="append", tokens=256, page=64, dtype="bf16"),
        # the tokens of a packed prefill of eight sequences
        dict(name="append_prefill_41460", op="append", tokens=41460, page=64, dtype="bf16"),
        # a single user early in a conversation: latency of one layer
        dict(name="decode_1x900_h16", op="decode", requests=1, heads=16, k=1, length=900, page=64, dtype="bf16"),
        # a full decode batch with ragged contexts
        dict(name="decode_256x4096_h32", op="decode", requests=256, heads=32, k=1, length=4096, page=64, dtype="bf16"),
        # the verify step of speculative decoding, seven positions a request
        dict(name="verify_64x7x6000_h32", op="decode", requests=64, heads=32, k=7, length=6000, page=32, dtype="f16"),
        # few very long contexts on small pages: the work has to be split along the tokens
        dict(name="decode_4x131072_h16", op="decode", requests=4, heads=16, k=1, length=131072, page=16, dtype="bf16"),
        # three short prompts on a tensor-parallel head slice
        dict(name="prefill_3x70_h2", op="prefill", seqs=3, heads=2, new=70, context=0, dtype="bf16"),
        # a mixed batch of prompt chunks behind earlier contexts
        dict(name="prefill_8x1500_c3000_h32", op="prefill", seqs=8, heads=32, new=1500, context=3000, dtype="bf16"),
        # one long prompt
        dict(name="prefill_1x16384_h16", op="prefill", seqs=1, heads=16, new=16384, context=0, dtype="bf16"),
        # one answer token with its alternatives
        dict(name="logprobs_1x32768", op="logprobs", rows=1, vocab=32768, top=5, masked=False, dtype="bf16"),
        # every position of a speculative verify batch over a large vocabulary
        dict(name="logprobs_448x160000", op="logprobs", rows=448, vocab=160000, top=20, masked=True, dtype="bf16"),
        # the prompt's log probabilities, an odd vocabulary, fp32 logits
        dict(name="logprobs_4096x100003", op="logprobs", rows=4096, vocab=100003, top=8, masked=False, dtype="f32"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "logprobs", "logprobs"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 41460), page=rng.choice([16, 32, 48, 64, 128]), dtype=dtype)
    if op == "decode":
        r, k = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 7, 8, 16])
        h = rng.choice([1, 2, 4, 8, 12, 16, 24, 32, 40, 64, 128])
        r = max(1, min(r, 65536 // (h * k)))  # query rows
        most = min(131072, (1 << 20) // r, int(1.2e12 / (2 * r * h * k * (WIDTH + RANK))))
        length = _log(rng, 1, max(1, most))
        return dict(op=op, requests=r, heads=h, k=k, length=length,
                    page=rng.choice([16, 32, 48, 64, 128]), dtype=dtype)
    if op == "prefill":
        n, h = _log(rng, 1, 12), rng.choice([1, 2, 3, 4, 8, 16, 32])
        new = _log(rng, 1, 12288 // n)
        context = rng.choice([0, 0, _log(rng, 1, 6000)])
        while n * h * new * (new + context) > (1 << 31):
            h = max(1, h // 2)
            if h == 1:
                new = max(1, new // 2)
        return dict(op=op, seqs=n, heads=h, new=new, context=context, dtype=dtype)
    vocab = _log(rng, 1000, 200000)
    return dict(op=op, rows=_log(rng, 1, max(1, min(4096, 400_000_000 // vocab))), vocab=vocab,
                top=rng.choice([0, 1, 5, 8, 20, 32]), masked=rng.random() < 0.3,
                dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))


def _lengths(case):
    """(lengths of the queries, lengths of the keys) of each sequence or request."""
    if case["op"] == "decode":
        lens = [n + case["k"] - 1 for n in _spread(case["requests"], case["length"])] if case["requests"] > 1 \
            else [case["length"] + case["k"] - 1]
        return [case["k"]] * case["requests"], lens
    if case["seqs"] == 1:
        return [case["new"]], [case["new"] + case["context"]]
    new = _spread(case["seqs"], case["new"])
    ctx = _spread(case["seqs"], case["context"], 0.25)[::-1] if case["context"] else [0] * case["seqs"]
    return new, [a + b for a, b in zip(new, ctx)]


# ------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, std=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(std))
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return globals()["_prepare_" + case["op"]](case, _gen(seed))


def _prepare_append(case, g):
    T, page, dt = case["tokens"], case["page"], TYPES[case["dtype"]]
    pages = -(-2 * T // page)
    s = dict(case=case, kv=_randn(g, (T, WIDTH), dt, 3.0), weight=1 + _randn(g, (RANK,), dt, 0.1),
             cache=_randn(g, (pages, page, WIDTH), dt))
    s["slot"] = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _prepare_decode(case, g):
    R, K, H, page, dt = case["requests"], case["k"], case["heads"], case["page"], TYPES[case["dtype"]]
    _, lens = _lengths(case)
    width = max(-(-n // page) for n in lens)
    need = sum(-(-n // page) for n in lens)
    pages = need + 8
    cache = _randn(g, (pages, page, WIDTH), dt)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(R, width, dtype=torch.int32, device="cuda")
    used = torch.tensor([-(-n // page) for n in lens], device="cuda")
    held = torch.arange(width, device="cuda")[None, :] < used[:, None]
    table[held] = order[:need]
    return dict(case=case, q_latent=_randn(g, (R * K, H, RANK), dt), q_rope=_randn(g, (R * K, H, ROPE), dt),
                cache=cache, table=table, seq_len=_i32(lens),
                out=torch.empty(R * K, H, RANK, dtype=dt, device="cuda"),
                lse=torch.empty(R * K, H, dtype=torch.float32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_prefill(case, g):
    H, dt = case["heads"], TYPES[case["dtype"]]
    lq, lk = _lengths(case)
    Tq, Tk = sum(lq), sum(lk)
    # keys and values of a head side by side, as one up-projection of the latent vectors leaves them
    kv = _randn(g, (Tk, H, NOPE + DV), dt)
    cum = lambda v: _i32([sum(v[:i]) for i in range(len(v) + 1)])  # noqa: E731
    return dict(case=case, q=_randn(g, (Tq, H, NOPE + ROPE), dt), kv=kv, k_rope=_randn(g, (Tk, ROPE), dt),
                cu_q=cum(lq), cu_k=cum(lk), max_q=max(lq), max_k=max(lk),
                out=torch.empty(Tq, H, DV, dtype=dt, device="cuda"),
                lse=torch.empty(Tq, H, dtype=torch.float32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_logprobs(case, g):
    R, V, dt = case["rows"], case["vocab"], TYPES[case["dtype"]]
    logits = _randn(g, (R, V), dt, 2.5)
    if case["masked"]:  # a grammar leaves a part of the vocabulary
        cut = torch.rand(V, generator=g, device="cuda") < 0.4
        cut[: max(case["top"], 64)] = False
        logits.masked_fill_(cut[None, :], float("-inf"))
    tokens = torch.randint(0, min(V, max(case["top"], 64)), (R,), generator=g, device="cuda").to(torch.int32)
    # the model's favourite of each row stands clear of the rest in half of the rows
    best = torch.randint(0, V, (R,), generator=g, device="cuda")
    rows = torch.arange(0, R, 2, device="cuda")
    logits[rows, best[::2]] = 14.0
    top = case["top"]
    f = lambda *n: torch.empty(*n, dtype=torch.float32, device="cuda")  # noqa: E731
    return dict(case=case, logits=logits, tokens=tokens, logprob=f(R), entropy=f(R), top_logprobs=f(R, top),
                top_ids=torch.empty(R, top, dtype=torch.int32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------------------ one pass


def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _plain_append(s):
    x = s["kv"].float()
    c = x[:, :RANK]
    c = c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    rows = torch.cat([c, x[:, RANK:]], dim=1).to(s["cache"].dtype)
    s["cache"].view(-1, WIDTH)[s["slot"].long()] = rows
    return {"cache": s["cache"]}


def _softmax_parts(x):
    """exp(x - max) with its sum and log-sum-exp over the last axis; a row of -inf has sum 0."""
    m = x.amax(dim=-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = x.sub_(m0).exp_()
    z = e.sum(dim=-1, keepdim=True)
    return e, z, (m0 + z.log()).squeeze(-1)


def _plain_decode(s):
    R, K, H = s["case"]["requests"], s["case"]["k"], s["case"]["heads"]
    kv = s["cache"][s["table"].long()].reshape(R, -1, WIDTH).float()
    q = torch.cat([s["q_latent"], s["q_rope"]], dim=2).float().reshape(R, K * H, WIDTH)
    x = torch.matmul(q, kv.transpose(1, 2)).mul_(SCALE).view(R, K, H, -1)
    pos = torch.arange(x.shape[-1], device=x.device)
    last = s["seq_len"].long()[:, None] - K + torch.arange(K, device=x.device)[None, :]
    x.masked_fill_((pos[None, None, :] > last[:, :, None])[:, :, None, :], float("-inf"))
    e, z, lse = _softmax_parts(x)
    o = torch.matmul(e.view(R, K * H, -1), kv[..., :RANK]).view(R, K, H, RANK) / z.clamp_min(1e-30)
    return {"out": o.reshape(R * K, H, RANK).to(s["out"].dtype), "lse": lse.reshape(R * K, H)}


def _plain_prefill(s):
    N, dev = s["case"]["seqs"], s["q"].device
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    iq, ik = torch.arange(s["max_q"], device=dev), torch.arange(s["max_k"], device=dev)
    at_q = (cu_q[:-1, None] + iq).clamp_max(s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp_max(s["kv"].shape[0] - 1)
    q = s["q"][at_q].float().transpose(1, 2)
    kv = s["kv"][at_k].float().transpose(1, 2)
    rope = s["k_rope"][at_k].float()[:, None]
    x = torch.matmul(q[..., :NOPE], kv[..., :NOPE].transpose(2, 3))
    x.add_(torch.matmul(q[..., NOPE:], rope.transpose(2, 3))).mul_(SCALE)
    last = iq[None, :] + (lk - lq)[:, None]
    x.masked_fill_((ik[None, None, :] > last[:, :, None])[:, None], float("-inf"))
    e, z, lse = _softmax_parts(x)
    o = torch.matmul(e, kv[..., NOPE:]) / z.clamp_min(1e-30)
    t = torch.arange(s["q"].shape[0], device=dev)
    n = torch.searchsorted(cu_q, t, right=True).sub_(1).clamp_max(N - 1)
    i = t - cu_q[n]
    return {"out": o[n, :, i].to(s["out"].dtype), "lse": lse[n, :, i]}


def _plain_logprobs(s):
    top = s["case"]["top"]
    x = s["logits"].float() + 0.0
    m = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(dim=1, keepdim=True)
    lse = m + z.log()
    moment = torch.where(e > 0, e * (x - m), torch.zeros_like(x)).sum(dim=1, keepdim=True)
    out = {"logprob": (x.gather(1, s["tokens"].long()[:, None]) - lse)[:, 0], "entropy": (z.log() - moment / z)[:, 0]}
    if top:
        # order by value, then by the lower index, as one whole number
        b = x.view(torch.int32).long()
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        key = b * (1 << 20) + ((1 << 20) - 1 - torch.arange(x.shape[1], device=x.device))
        ids = (1 << 20) - 1 - (key.topk(top, dim=1).values & ((1 << 20) - 1))
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = x.gather(1, ids) - lse
    return out


def _own_append(s):
    import serving_kda_chunk_gb300 as kda

    kda.kda_latent_append(s["kv"], s["cache"], s["slot"], weight=s["weight"], eps=EPS, dev_status=s["status"])
    return {"cache": s["cache"]}


def _own_decode(s):
    import serving_kda_chunk_gb300 as kda

    c = s["case"]
    if "workspace" not in s:  # kept by the program from call to call
        s["workspace"] = torch.empty(kda.kda_latent_decode_workspace_size(c["requests"], c["k"], c["heads"]),
                                     dtype=torch.uint8, device="cuda")
    kda.kda_latent_decode(s["q_latent"], s["q_rope"], s["cache"], s["table"], s["seq_len"], s["out"],
                          s["workspace"], K=c["k"], scale=SCALE, lse=s["lse"], dev_status=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prefill(s):
    import serving_kda_chunk_gb300 as kda

    kda.kda_latent_prefill(s["q"], s["kv"][..., :NOPE], s["k_rope"], s["kv"][..., NOPE:], s["cu_q"], s["cu_k"],
                           s["out"], scale=SCALE, lse=s["lse"], dev_status=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_logprobs(s):
    import serving_kda_chunk_gb300 as kda

    top = s["case"]["top"]
    kda.kda_token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"],
                           top_ids=s["top_ids"] if top else None,
                           top_logprobs=s["top_logprobs"] if top else None, dev_status=s["status"])
    out = {"logprob": s["logprob"], "entropy": s["entropy"]}
    if top:
        out["top_ids"], out["top_logprobs"] = s["top_ids"], s["top_logprobs"]
    return out


# ------------------------------------------------------------------------------ what a pass cannot do without


def work(case):
    b = _bytes(case)
    if case["op"] == "append":
        T = case["tokens"]
        return {"bytes": T * (2 * WIDTH * b + 4) + RANK * b, "flops": 4 * T * RANK}
    if case["op"] == "decode":
        lq, lk = _lengths(case)
        rows = case["requests"] * case["k"] * case["heads"]
        pairs = sum(sum(n - case["k"] + t + 1 for t in range(case["k"])) for n in lk) * case["heads"]
        return {"bytes": sum(lk) * WIDTH * b + rows * ((WIDTH + RANK) * b + 4) + 4 * sum(-(-n // case["page"]) for n in lk),
                "flops": 2 * pairs * (WIDTH + RANK)}
    if case["op"] == "prefill":
        lq, lk = _lengths(case)
        H = case["heads"]
        pairs = sum(a * (c - a) + a * (a + 1) // 2 for a, c in zip(lq, lk)) * H
        return {"bytes": (sum(lq) * H * (NOPE + ROPE + DV) + sum(lk) * (H * (NOPE + DV) + ROPE)) * b + sum(lq) * H * 4,
                "flops": 2 * pairs * (NOPE + ROPE + DV)}
    R, V = case["rows"], case["vocab"]
    return {"bytes": R * V * b + R * (12 + 8 * case["top"]), "flops": 5 * R * V}


# ------------------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _exact_append(s):
    cache = s["cache"].double().view(-1, WIDTH)
    for i in range(0, s["kv"].shape[0], 1 << 16):
        x = s["kv"][i:i + (1 << 16)].double()
        norm = x[:, :RANK].square().sum(1).div(RANK).add(EPS).sqrt()
        x[:, :RANK] = x[:, :RANK] / norm[:, None] * s["weight"].double()
        cache[s["slot"][i:i + (1 << 16)].long()] = x
    return {"cache": cache.view(s["cache"].shape)}


def _attend(q, k, v, last):
    """softmax(SCALE q k^T) v in 64 bits over keys 0 .. last[i] of query row i, and its log-sum-exp."""
    x = q @ k.T * SCALE
    x = torch.where(torch.arange(k.shape[0], device=q.device)[None, :] <= last[:, None], x, float("-inf"))
    lse = torch.logsumexp(x, dim=1)
    p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[:, None])
    return p @ v, lse


def _exact_decode(s):
    R, K, H = s["case"]["requests"], s["case"]["k"], s["case"]["heads"]
    out = torch.zeros(R * K, H, RANK, dtype=torch.float64, device="cuda")
    lse = torch.zeros(R * K, H, dtype=torch.float64, device="cuda")
    page = s["case"]["page"]
    for r, n in enumerate(s["seq_len"].tolist()):
        c = s["cache"][s["table"][r, : -(-n // page)].long()].reshape(-1, WIDTH)[:n].double()
        rows = slice(r * K, (r + 1) * K)
        q = torch.cat([s["q_latent"][rows], s["q_rope"][rows]], 2).double().reshape(K * H, WIDTH)
        last = n - K + torch.arange(K, device="cuda").repeat_interleave(H)
        o, z = _attend(q, c, c[:, :RANK], last)
        out[rows], lse[rows] = o.view(K, H, RANK), z.view(K, H)
    return {"out": out, "lse": lse}


def _exact_prefill(s):
    H = s["case"]["heads"]
    lq, lk = _lengths(s["case"])
    if 4 * H * sum(a * c for a, c in zip(lq, lk)) * (NOPE + ROPE + DV) > 2e13:
        return None
    out = torch.zeros(sum(lq), H, DV, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(lq), H, dtype=torch.float64, device="cuda")
    a = c = 0
    for nq, nk in zip(lq, lk):
        last = nk - nq + torch.arange(nq, device="cuda")
        for h in range(H):
            k = torch.cat([s["kv"][c:c + nk, h, :NOPE], s["k_rope"][c:c + nk]], 1).double()
            out[a:a + nq, h], lse[a:a + nq, h] = _attend(s["q"][a:a + nq, h].double(), k,
                                                         s["kv"][c:c + nk, h, NOPE:].double(), last)
        a, c = a + nq, c + nk
    return {"out": out, "lse": lse}


def _exact_logprobs(s):
    R, top = s["logits"].shape[0], s["case"]["top"]
    parts = []
    for i in range(0, R, 256):
        x = s["logits"][i:i + 256].double()
        logp = x - torch.logsumexp(x, dim=1, keepdim=True)
        part = {"logprob": logp.gather(1, s["tokens"][i:i + 256].long()[:, None])[:, 0],
                "entropy": -torch.where(logp.isinf(), 0.0, logp.exp() * logp).sum(1)}
        if top:
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
            part["top_ids"], part["top_logprobs"] = ids.to(torch.int32), logp.gather(1, ids)
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
