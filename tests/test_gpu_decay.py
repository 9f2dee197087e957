"""Linear attention with a decay a head: the calls against the recurrence itself in 64 bits.

Tolerances are relative 2-norms over a (sequence or request, head).  u = eps / 2 is the most that a rounding to
a type changes a value.
  Decode rounds its outputs and states once; the rest is fp32 sums of at most 128 + 16 terms (each rounding 2^-24,
  random in sign: below 1e-5 of the result's norm, exponentials included).
  Prefill rounds three things to the input type or the output's: weights of a chunk, the state for the product with
  the queries, the output.  Each rounding error is spread over +-u of its value, u / sqrt(3) in the mean square, and
  the three are independent: u in all; 1.5 u allows for values that lie low in their binade alike.
  A prefill's fp32 state adds keys split in two 16-bit parts: 2 u^2 relative for bf16, 3.1e-5, and no more for fp16.
"""
import pytest
import torch

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
D = 128
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NINF = float("-inf")


def half_step(dt):
    return torch.finfo(dt).eps / 2


def rel(got, want):
    """Largest relative 2-norm error over the leading dimension's blocks; blocks of zeros have to be zeros."""
    got, want = got.double().flatten(1), want.double().flatten(1)
    n, e = want.norm(dim=1), (got - want).norm(dim=1)
    assert not torch.isnan(got).any() and not (e[n == 0] != 0).any()
    return (e[n > 0] / n[n > 0]).max().item() if (n > 0).any() else 0.0


def gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dt=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gates(g, kind, n, H):
    """(head_decay, log_decay)."""
    head = -torch.exp2(-8 * torch.arange(1, H + 1, device="cuda", dtype=F32) / H)
    token = -torch.nn.functional.softplus(1.5 * torch.randn(n, H, generator=g, device="cuda") - 3)
    if kind == "resets":  # forgotten states, at neighbouring tokens too, and values that count as 0
        x = torch.rand(n, H, generator=g, device="cuda")
        token[x < 0.05] = NINF
        token[x > 0.97] = -300.0
        token[(x > 0.5) & (x < 0.55)] = 2.0
        token[1::7] = -1e-7
    if kind == "none":
        return torch.zeros(H, device="cuda"), None
    return (head if kind in ("head", "both") else None), (token if kind != "head" else None)


def log_decay(head, token, n, H):
    x = torch.zeros(n, H, dtype=torch.float64, device="cuda")
    for t in (head, token):
        if t is not None:
            x = x + t.double()
    return x.clamp_max(0)


def recur(S, q, k, v, g):
    """Outputs [n, H, D] and states after each row [n + 1, H, value, key] of one sequence in 64 bits."""
    H, rep = v.shape[1], v.shape[1] // k.shape[1]
    q, k, v = q.double().repeat_interleave(rep, 1), k.double().repeat_interleave(rep, 1), v.double()
    states, outs = [S], []
    for t in range(v.shape[0]):
        S = S * g[t].exp()[:, None, None] + v[t, :, :, None] * k[t, :, None, :]
        states.append(S)
        outs.append((S * q[t, :, None, :]).sum(-1))
    return (torch.stack(outs) if outs else torch.zeros(0, H, D, device="cuda", dtype=torch.float64)), torch.stack(states)


def prefill_case(lens, H, Hk, dt, kind, st=F32, seed=0, extra=3, std=1.0):
    """Packed sequences with `extra` rows behind the last; q, k and v are views of one projection's rows."""
    g = gen(seed)
    T = sum(lens) + extra
    qkv = randn(g, T, 2 * Hk + H, D, dt=dt)
    q, k, v = qkv[:, :Hk], qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
    k.mul_(D ** -0.5)
    v.mul_(std)
    head, token = gates(g, kind, T, H)
    N = len(lens)
    pool = randn(g, 2 * N + 1, H, D, D, dt=st, std=0.3 * std)
    cu = i32([sum(lens[:i]) for i in range(N + 1)])
    return dict(q=q, k=k, v=v, head=head, token=token, pool=pool, cu=cu, lens=lens, H=H, T=T, dt=dt)


def call_prefill(c, out, pool, init, final, ws=True, scale=D ** -0.5, **kw):
    status = i32([0])
    if ws is True:
        ws = torch.full((kda.kda_decay_prefill_workspace_size(c["T"], len(c["lens"]), c["H"]),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    kda.kda_decay_prefill(c["q"], c["k"], c["v"], c["cu"], out, head_decay=c["head"], log_decay=c["token"],
                          state_pool=pool, init_slot=init, final_slot=final, scale=scale, workspace=ws,
                          dev_status=status, **kw)
    torch.cuda.synchronize()
    return int(status)


def want_prefill(c, init, scale=D ** -0.5):
    """Per sequence (outputs, states after each of its rows)."""
    g = log_decay(c["head"], c["token"], c["T"], c["H"])
    res, a = [], 0
    for n, L in enumerate(c["lens"]):
        S = torch.zeros(c["H"], D, D, dtype=torch.float64, device="cuda")
        if init is not None and int(init[n]) >= 0:
            S = c["pool"][int(init[n])].double()
        o, s = recur(S, c["q"][a:a + L], c["k"][a:a + L], c["v"][a:a + L], g[a:a + L])
        res.append((o * scale, s))
        a += L
    return res


def check_prefill(c, out, pool, want, final, out_dt):
    # an fp32 output leaves the weights' and the state's roundings; a 16-bit state its own on top
    u, us, a = half_step(c["dt"]), half_step(pool.dtype) if pool.dtype != F32 else 0.0, 0
    for n, (o, s) in enumerate(want):
        got = out[a:a + len(o)]
        if len(o):
            assert rel(got.transpose(0, 1), o.transpose(0, 1)) <= 1.5 * max(u, half_step(out_dt)), n
        if final is not None and int(final[n]) >= 0:
            assert rel(pool[int(final[n])], s[-1]) <= us + 3.1e-5, n
        a += len(o)


LENS = [[1], [2, 1, 3], [127], [128], [129], [5, 0, 128, 300, 64], [700, 1, 257], [0], [1500]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("kind", ["head", "token", "both", "resets", "none"])
def test_prefill(lens, kind):
    c = prefill_case(lens, 2, 2, BF16, kind)
    N = len(lens)
    init = i32([n if n % 3 != 1 else -1 for n in range(N)])
    final = i32([N + n if n % 3 != 2 else n for n in range(N)])  # some in place
    want = want_prefill(c, init)
    pool, out = c["pool"].clone(), torch.full((c["T"], 2, D), 7.0, dtype=BF16, device="cuda")
    assert call_prefill(c, out, pool, init, final) == 0
    check_prefill(c, out, pool, want, final, BF16)
    assert (out[sum(lens):] == 7.0).all()  # rows of no sequence
    kept = [i for i in range(2 * N + 1) if i not in final.tolist()]
    assert torch.equal(pool[kept], c["pool"][kept])


@pytest.mark.parametrize("dt,out_dt,st", [(BF16, BF16, BF16), (BF16, F32, F16), (F16, F16, F32), (F16, BF16, F16), (F16, F32, BF16),
                                          (BF16, F16, F32)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (4, 2), (5, 5)])
def test_prefill_types_and_heads(dt, out_dt, st, H, Hk):
    lens = [130, 41, 256]
    c = prefill_case(lens, H, Hk, dt, "both", st)
    init, final = i32([0, -1, 2]), i32([3, 4, 2])
    want = want_prefill(c, init)
    # heads outside rows: the output is a view of [H, T, D]
    pool, wide = c["pool"].clone(), torch.zeros(H, c["T"], D + 8, dtype=out_dt, device="cuda")
    out = wide[:, :, :D].transpose(0, 1)
    assert call_prefill(c, out, pool, init, final) == 0
    check_prefill(c, out, pool, want, final, out_dt)
    assert (wide[:, :, D:] == 0).all()


@pytest.mark.parametrize("std", [1e-3, 30.0])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_prefill_small_and_large_values(dt, std):
    """Scores and states that fp16 could not hold unscaled, and ones near its smallest."""
    lens = [300, 129]
    c = prefill_case(lens, 2, 1, dt, "none", std=std)
    c["q"].mul_(std)
    if std > 1:
        c["k"].mul_(std)
    init, final = i32([0, 1]), i32([2, 3])
    want = want_prefill(c, init)
    pool, out = c["pool"].clone(), torch.zeros(c["T"], 2, D, device="cuda")
    assert call_prefill(c, out, pool, init, final) == 0
    check_prefill(c, out, pool, want, final, F32)


def test_prefill_continues_where_it_stopped():
    """A prompt in two calls, the state through the pool, answers as in one."""
    c = prefill_case([1000], 2, 2, BF16, "token", extra=0)
    pool = c["pool"].clone()
    whole, parts = (torch.zeros(1000, 2, D, device="cuda") for _ in range(2))
    assert call_prefill(c, whole, pool, None, i32([0])) == 0
    for a, b in ((0, 384), (384, 1000)):
        d = {**c, "q": c["q"][a:b], "k": c["k"][a:b], "v": c["v"][a:b], "token": c["token"][a:b].contiguous(),
             "cu": i32([0, b - a]), "T": b - a}
        assert call_prefill(d, parts[a:b], pool, i32([1]) if a else None, i32([1])) == 0
    assert rel(parts.transpose(0, 1), whole.transpose(0, 1)) <= 3 * half_step(BF16)
    assert rel(pool[1], pool[0]) <= 6.2e-5


def test_prefill_snapshots():
    lens = [500, 128, 60]
    c = prefill_case(lens, 3, 3, BF16, "token")
    init, final = i32([0, -1, 2]), i32([3, 4, 5])
    want = want_prefill(c, init)
    track = i32([[3, -1, 0], [0, 1, -1], [0, -7, -1]])  # 1 of one chunk, and -7, do not exist
    snap = torch.full((3, 3, 3, D, D), 5.0, device="cuda")
    pool, out = c["pool"].clone(), torch.zeros(c["T"], 3, D, dtype=BF16, device="cuda")
    assert call_prefill(c, out, pool, init, final, track_chunk_idx=track, track_state=snap) == kda.KDA_DEV_BAD_TRACK
    for n, m, t in ((0, 0, 384), (0, 2, 0), (1, 0, 0), (2, 0, 0)):
        assert rel(snap[n, m], want[n][1][t]) <= 3.1e-5
    for n, m in ((0, 1), (1, 1), (1, 2), (2, 1), (2, 2)):
        assert (snap[n, m] == 5.0).all()
    check_prefill(c, out, pool, want, final, BF16)


@pytest.mark.parametrize("shape", [([5000], 1), ([3000, 17], 3), ([9000, 2000, 1], 2), ([200] * 40, 8), ([4000, 100, 6000], 16)],
                         ids=str)
def test_prefill_cut_between_sms(shape):
    """Long sequences with few heads, with and without a workspace, against the chunked definition in 64 bits."""
    lens, H = shape
    c = prefill_case(lens, H, 1, BF16, "both", seed=3)
    c["head"].mul_(0.01)  # states that outlive many chunks
    c["token"].mul_(0.02)
    N = len(lens)
    init, final = i32(list(range(N))), i32([N + n for n in range(N)])
    want = want_prefill(c, init)
    results = []
    for ws in (True, None):
        pool, out = c["pool"].clone(), torch.zeros(c["T"], H, D, dtype=BF16, device="cuda")
        assert call_prefill(c, out, pool, init, final, ws=ws) == 0
        # rounding errors of keys are alike in sign for no reason, and a state sums up to 9000 of them
        check_prefill(c, out, pool, want, final, BF16)
        results.append((out, pool))
    again_pool, again = c["pool"].clone(), torch.zeros(c["T"], H, D, dtype=BF16, device="cuda")
    call_prefill(c, again, again_pool, init, final)
    assert torch.equal(again, results[0][0]) and torch.equal(again_pool, results[0][1])  # the same bits each time


def test_prefill_bad_bounds_and_slots():
    c = prefill_case([100, 100, 100], 2, 2, BF16, "head", extra=0)
    good = torch.zeros(300, 2, D, dtype=BF16, device="cuda")
    call_prefill(c, good, c["pool"].clone(), None, None)
    for cu in ([0, 100, 250, 200], [0, 100, 200, 301], [-5, 100, 200, 300]):
        out = torch.full((300, 2, D), 9.0, dtype=BF16, device="cuda")
        status = call_prefill({**c, "cu": i32(cu)}, out, c["pool"].clone(), None, None)
        assert status == kda.KDA_DEV_BAD_SEQLEN
        if cu[0] == 0:
            assert torch.equal(out[:100], good[:100])
    pool, out = c["pool"].clone(), torch.full((300, 2, D), 9.0, dtype=BF16, device="cuda")
    assert call_prefill(c, out, pool, i32([-1, 99, -1]), i32([-1, 0, 7])) == kda.KDA_DEV_BAD_SLOT
    assert torch.equal(pool, c["pool"]) and (out[100:] == 9.0).all() and torch.equal(out[:100], good[:100])


def test_prefill_without_rows_passes_states_on():
    pool = randn(gen(), 4, 2, D, D)
    q = torch.zeros(0, 2, D, dtype=BF16, device="cuda")
    before = pool.clone()
    kda.kda_decay_prefill(q, q, q, i32([0, 0, 0]), q, head_decay=torch.zeros(2, device="cuda"), state_pool=pool,
                          init_slot=i32([0, -1]), final_slot=i32([2, 3]))
    assert torch.equal(pool[2], before[0]) and (pool[3] == 0).all() and torch.equal(pool[:2], before[:2])


def test_prefill_bits_behind_a_sequence_reach_nothing():
    """NaN rows behind the last sequence, and an unwritten neighbour's, leave the others' results as they are."""
    c = prefill_case([70, 130], 2, 2, BF16, "token", extra=200)
    a, b = (torch.zeros(c["T"], 2, D, dtype=BF16, device="cuda") for _ in range(2))
    p, r = c["pool"].clone(), c["pool"].clone()
    call_prefill(c, a, p, None, i32([0, 1]))
    for t in (c["q"], c["k"], c["v"]):
        t[200:] = float("nan")
    c["token"][200:] = float("nan")
    call_prefill(c, b, r, None, i32([0, 1]))
    assert torch.equal(a, b) and torch.equal(p, r)
    c["v"][70:200] = float("inf")  # the second sequence's values
    call_prefill(c, b, r, None, i32([0, 1]))
    assert torch.equal(a[:70], b[:70]) and torch.equal(p[0], r[0])


def test_prefill_in_graphs_and_on_two_streams():
    """Two captured calls with workspaces of their own, replayed at once."""
    cs = [prefill_case([2000, 300], 2, 2, BF16, "token", seed=s) for s in (1, 2)]
    wants, runs = [], []
    for c in cs:
        pool, out = c["pool"].clone(), torch.zeros(c["T"], 2, D, dtype=BF16, device="cuda")
        call_prefill(c, out, pool, i32([0, 1]), i32([2, 3]))
        wants.append((out, pool))
    for c in cs:
        pool, out = c["pool"].clone(), torch.zeros(c["T"], 2, D, dtype=BF16, device="cuda")
        ws = torch.empty(kda.kda_decay_prefill_workspace_size(c["T"], 2, 2), dtype=torch.uint8, device="cuda")
        args = dict(head_decay=c["head"], log_decay=c["token"], state_pool=pool, init_slot=i32([0, 1]),
                    final_slot=i32([2, 3]), scale=D ** -0.5, workspace=ws)
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kda.kda_decay_prefill(c["q"], c["k"], c["v"], c["cu"], out, **args)
        runs.append((g, s, out, pool, args))  # a graph keeps no tensor alive
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, *_ in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, _, out, pool, _), (wo, wp) in zip(runs, wants):
        assert torch.equal(out, wo) and torch.equal(pool, wp)


# ------------------------------------------------------------------------------ decode


def decode_case(R, K, H, Hk, dt, kind, st=F32, seed=0):
    g = gen(seed)
    qkv = randn(g, R * K, 2 * Hk + H, D, dt=dt)
    k = qkv[:, Hk:2 * Hk]
    k.mul_(D ** -0.5)
    head, token = gates(g, kind, R * K, H)
    pool = randn(g, 2 * R + 2, H, D, D, dt=st, std=0.3)
    slot = torch.randperm(2 * R + 2, generator=g, device="cuda").to(torch.int32)
    return dict(q=qkv[:, :Hk], k=k, v=qkv[:, 2 * Hk:], head=head, token=token, pool=pool, slot=slot[:R].contiguous(),
                spare=slot[R:2 * R].contiguous(), R=R, K=K, H=H)


def call_decode(c, pool, out, scale=D ** -0.5, **kw):
    status = i32([0])
    kda.kda_decay_decode(c["q"], c["k"], c["v"], pool, kw.pop("slot", c["slot"]), out, K=c["K"], head_decay=c["head"],
                         log_decay=c["token"], scale=scale, dev_status=status, **kw)
    return int(status)


def want_decode(c, r, ql):
    rows = slice(r * c["K"], r * c["K"] + ql)
    g = log_decay(c["head"], c["token"], c["R"] * c["K"], c["H"])
    return recur(c["pool"][int(c["slot"][r])].double(), c["q"][rows], c["k"][rows], c["v"][rows], g[rows])


def tol(dt):
    return (half_step(dt) if dt != F32 else 0.0) + 1e-5


@pytest.mark.parametrize("K", [1, 2, 3, 5, 8, 16])
@pytest.mark.parametrize("kind", ["head", "token", "both", "resets"])
def test_decode_step_verify_commit(K, kind):
    R, H = 5, 3
    c = decode_case(R, K, H, 1 if K % 2 else 3, BF16, kind)
    ql = i32([K, max(K - 1, 0), 1, 0, K])
    nc = i32([K // 2, max(K - 1, 0), 1, 0, 0])
    pool, out = c["pool"].clone(), torch.full((R * K, H, D), 7.0, dtype=BF16, device="cuda")
    assert call_decode(c, pool, out, q_len=ql, n_commit=i32([0] * R)) == 0  # verify
    assert torch.equal(pool, c["pool"])
    assert call_decode({**c, "q": None}, pool, None, q_len=ql, n_commit=nc) == 0  # commit
    step_pool, step_out = c["pool"].clone(), torch.zeros_like(out)
    assert call_decode(c, step_pool, step_out, q_len=ql) == 0  # all positions at once
    assert torch.equal(step_out, out)
    one = c["pool"].clone()
    assert call_decode(c, one, step_out, q_len=ql, n_commit=nc) == 0  # outputs and part of the states
    assert torch.equal(step_out, out) and torch.equal(one, pool)
    for r in range(R):
        o, s = want_decode(c, r, int(ql[r]))
        rows = out[r * K:r * K + int(ql[r])]
        if len(o):
            assert rel(rows.reshape(-1, D), (o * D ** -0.5).reshape(-1, D)) <= tol(BF16)
        assert (out[r * K + int(ql[r]):(r + 1) * K] == 0).all()
        at = int(c["slot"][r])
        assert rel(pool[at], s[int(nc[r])]) <= 1e-5
        assert rel(step_pool[at], s[int(ql[r])]) <= 1e-5
    others = [i for i in range(len(pool)) if i not in c["slot"].tolist()]
    assert torch.equal(pool[others], c["pool"][others])


@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("dt,out_dt,st", [(BF16, F32, F16), (F16, F16, F32), (F32, F32, F32), (F32, BF16, BF16), (F16, F32, BF16)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (5, 1)])
def test_decode_types_and_heads(K, dt, out_dt, st, H, Hk):
    c = decode_case(3, K, H, Hk, dt, "token", st)
    pool, wide = c["pool"].clone(), torch.zeros(H, 3 * K, D + 8, dtype=out_dt, device="cuda")
    assert call_decode(c, pool, wide[:, :, :D].transpose(0, 1)) == 0
    for r in range(3):
        o, s = want_decode(c, r, K)
        assert rel(wide[:, r * K:(r + 1) * K, :D].reshape(-1, D), (o * D ** -0.5).transpose(0, 1).reshape(-1, D)) <= tol(out_dt)
        assert rel(pool[int(c["slot"][r])], s[-1]) <= tol(st)
    assert (wide[:, :, D:] == 0).all()


@pytest.mark.parametrize("K", [1, 3])
def test_decode_destination_slots_and_refused_requests(K):
    c = decode_case(6, K, 2, 2, BF16, "both")
    P = len(c["pool"])
    slot, dst = c["slot"].clone(), c["spare"].clone()
    slot[1], slot[2] = -1, P
    dst[3], dst[4] = -1, P
    nc = i32([0, 0, 0, K, K, K])
    pool, out = c["pool"].clone(), torch.full((6 * K, 2, D), 7.0, dtype=BF16, device="cuda")
    assert call_decode(c, pool, out, slot=slot, dst_slot=dst, n_commit=nc) == kda.KDA_DEV_BAD_SLOT
    o, s = want_decode(c, 5, K)
    assert torch.equal(pool[int(dst[0])], c["pool"][int(slot[0])])  # nothing committed: a copy
    assert rel(pool[int(dst[5])], s[-1]) <= 1e-5
    for r in (1, 2, 4):
        assert (out[r * K:(r + 1) * K] == 0).all()
    for r in (0, 3, 5):
        o, _ = want_decode(c, r, K)
        assert rel(out[r * K:(r + 1) * K].reshape(-1, D), (o * D ** -0.5).reshape(-1, D)) <= tol(BF16)
    others = [i for i in range(P) if i not in (int(dst[0]), int(dst[5]))]
    assert torch.equal(pool[others], c["pool"][others])
    pool = c["pool"].clone()
    bad = call_decode(c, pool, out, q_len=i32([K, K + 1, -1, K, K, K]), n_commit=i32([0, 0, 0, -1, K + 1, K]))
    assert bad == kda.KDA_DEV_BAD_ACCEPT
    for r in range(1, 5):
        assert (out[r * K:(r + 1) * K] == 0).all() and torch.equal(pool[int(c["slot"][r])], c["pool"][int(c["slot"][r])])


def test_decode_padding_reads_nothing():
    """Rows past q_len and padding requests may hold anything."""
    c = decode_case(3, 4, 2, 2, BF16, "token")
    ql, slot = i32([2, 4, 0]), c["slot"].clone()
    slot[1] = -1
    a, b = (torch.zeros(12, 2, D, dtype=BF16, device="cuda") for _ in range(2))
    p, r = c["pool"].clone(), c["pool"].clone()
    call_decode(c, p, a, q_len=ql, slot=slot)
    for t in (c["q"], c["k"], c["v"], c["token"]):
        t[2:] = float("nan")
    assert call_decode(c, r, b, q_len=ql, slot=slot) == 0
    assert torch.equal(a, b) and torch.equal(p, r)


def test_decode_follows_the_prefill():
    """Tokens decoded one by one, or verified and committed, behind a prefilled prompt answer as the prefill
    of the longer prompt does."""
    n, extra = 200, 6
    c = prefill_case([n + extra], 4, 2, BF16, "token", extra=0)
    whole = torch.zeros(n + extra, 4, D, device="cuda")
    pool = c["pool"].clone()
    assert call_prefill(c, whole, pool, None, i32([0])) == 0
    cut = {**c, "q": c["q"][:n], "k": c["k"][:n], "v": c["v"][:n], "token": c["token"][:n], "cu": i32([0, n]), "T": n}
    part = torch.zeros(n, 4, D, device="cuda")
    assert call_prefill(cut, part, pool, None, i32([1])) == 0
    pool[2].copy_(pool[1])
    got = torch.zeros(extra, 4, D, device="cuda")
    for t in range(n, n + extra):
        row = dict(q=c["q"][t:t + 1], k=c["k"][t:t + 1], v=c["v"][t:t + 1], head=None, token=c["token"][t:t + 1], K=1)
        assert call_decode({**row, "slot": i32([1])}, pool, got[t - n:t - n + 1]) == 0
    assert rel(got.transpose(0, 1), whole[n:].transpose(0, 1)) <= 1.5 * half_step(BF16) + 1e-4
    assert rel(pool[1], pool[0]) <= 7e-5
    rows = dict(q=c["q"][n:], k=c["k"][n:], v=c["v"][n:], head=None, token=c["token"][n:], K=extra, slot=i32([2]))
    again = torch.zeros(extra, 4, D, device="cuda")
    assert call_decode(rows, pool, again, n_commit=i32([0])) == 0
    assert call_decode({**rows, "q": None}, pool, None, n_commit=i32([extra])) == 0
    assert rel(again.transpose(0, 1), got.transpose(0, 1)) <= 2e-5 and rel(pool[2], pool[1]) <= 2e-5


def test_decode_in_a_graph():
    c = decode_case(4, 3, 2, 2, BF16, "token")
    pool, out = c["pool"].clone(), torch.zeros(12, 2, D, dtype=BF16, device="cuda")
    for _ in range(3):
        call_decode(c, pool, out)
    gpool, gout = c["pool"].clone(), torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kda.kda_decay_decode(c["q"], c["k"], c["v"], gpool, c["slot"], gout, K=3, log_decay=c["token"], scale=D ** -0.5)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, out) and torch.equal(gpool, pool)
