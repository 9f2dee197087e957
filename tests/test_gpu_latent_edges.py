"""Latent attention at its edges, against its definition in 64 bits."""
import numpy as np
import pytest
import torch

from helpers import i32
from test_gpu_latent import DL, DR, SCALE, TYPES, UNIT, W, Decode, Prefill  # noqa: F401

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------- requests without positions


@pytest.mark.parametrize("K,H", [(1, 4), (2, 16), (3, 40)])
@pytest.mark.parametrize("n", [130, 40000])  # one block; split over many
def test_decode_without_positions_reads_no_key(n, K, H):
    # a padding request of a captured batch: its length, pages and what lies on them are left over
    d = Decode([n, 90], K, H, 16, seed=n + K)
    d.cache[d.table[0, : -(-n // 16)].long()] = float("nan")
    d.table[0, 1] = -1  # a page that is no longer there
    out, lse, st = d.run(q_len=[0, K])
    assert st == 0
    assert (out[:K] == 0).all() and (lse[:K] == -torch.inf).all()
    d.check((out, lse, st), q_len=[0, K], skip=(0,))


def test_decode_without_positions_still_reports_a_bad_length():
    d = Decode([100, 50], 2, 4, 16, seed=2)
    for bad in (-1, 16 * d.table.shape[1] + 1):
        out, lse, st = d.run(q_len=[0, 2], seq_len=i32([bad, 50]))
        assert st == kda.KDA_DEV_BAD_SEQLEN
        assert (out[:2] == 0).all() and (lse[:2] == -torch.inf).all()
        d.check((out, lse, st), q_len=[0, 2], skip=(0,))


# ----------------------------------------------------------- rows that see no key


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,K,H", [(70, 3, 4), (70, 4, 30), (30000, 3, 8), (30000, 16, 8)])
def test_decode_rows_past_the_query_length_are_zero_beside_keys_that_are_not_finite(n, K, H, out_dtype, dtype):
    d = Decode([n], K, H, 32, dtype, seed=K)
    d.cache[d.table[0, 0].long(), 3] = float("nan")  # seen by position 0, the only one
    d.cache[d.table[0, 1].long(), 5, :DL] = float("inf")
    out, lse, st = d.run(out_dtype=TYPES[out_dtype], q_len=[1])
    assert st == 0
    assert (out[1:] == 0).all() and (lse[1:] == -torch.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
def test_prefill_rows_without_keys_are_zero_beside_keys_that_are_not_finite(out_dtype, dtype):
    # 200 queries over 150 keys: the first 50 see none, the others see the first key
    p = Prefill([200, 40], [150, 40], 2, dtype, seed=4)
    p.kv[0, :, :128] = float("nan")
    p.kv[1, :, 128:] = float("inf")
    out, lse, st = p.run(out_dtype=TYPES[out_dtype])
    assert st == 0
    assert (out[:50] == 0).all() and (lse[:50] == -torch.inf).all()
    p.check((out, lse, st), skip=(0,))


# ----------------------------------------------------------- scores that are not numbers


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,K,H", [(1, 1, 1), (70, 1, 9), (90, 2, 20), (300, 3, 30), (30000, 1, 12), (30000, 4, 16)])
def test_decode_rows_that_see_a_nan_score_have_nan_results(n, K, H, dtype):
    d = Decode([n, 65], K, H, 16, dtype, seed=n)
    d.ql[0, 0, 7] = float("nan")  # every score of one row
    out, lse, st = d.run(out_dtype=torch.float32)
    assert st == 0 and torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0])
    out[0, 0], lse[0, 0], d.ql[0, 0, 7] = 0, 0, 0
    if H > 1:
        o, z, bo, bz = d.ref(0)  # the other rows of the request
        assert ((out[:K].double() - o).abs() <= bo + 2.0 ** -20).view(K * H, DL)[1:].all()
        assert ((lse[:K].double() - z).abs() <= bz).view(K * H)[1:].all()
    d.check((out, lse, st), skip=(0,))
    # one key: every row that sees it, whichever tile or part it lies in
    for at in {0, n // 2, n - 1}:
        e = Decode([n, 65], K, H, 16, dtype, seed=n)
        e.cache[e.table[0, at // 16].long(), at % 16, DL] = float("nan")  # in the rope part: no value holds it
        out, lse, st = e.run(out_dtype=torch.float32)
        sees = torch.tensor([at <= n - K + t for t in range(K)], device="cuda")
        assert torch.isnan(out[:K][sees]).all() and torch.isnan(lse[:K][sees]).all()
        assert torch.isfinite(out[:K][~sees]).all()
        e.check((out, lse, st), skip=(0,))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prefill_rows_that_see_a_nan_score_have_nan_results(dtype):
    p = Prefill([300, 40], [700, 40], 2, dtype, seed=5)
    p.q[70, 1, 3] = float("nan")
    p.kr[650] = float("nan")  # seen by the rows from 250 on
    out, lse, st = p.run()
    assert st == 0
    bad = torch.zeros(300, 2, dtype=torch.bool, device="cuda")
    bad[70, 1] = True
    bad[250:] = True
    assert torch.equal(torch.isnan(out[:300]), bad[..., None].expand(300, 2, 128))
    assert torch.equal(torch.isnan(lse[:300]), bad)
    p.check((out, lse, st), skip=(0,))


@pytest.mark.parametrize("n,K,H", [(70, 1, 9), (300, 3, 30), (30000, 1, 12)])
def test_decode_rows_that_see_an_infinite_score(n, K, H):
    d = Decode([n], K, H, 16, seed=n)
    at = n // 2
    d.cache[d.table[0, at // 16].long(), at % 16, DL] = float("inf")  # scores of +inf or -inf, by the query's sign
    up = (d.qr[..., 0] > 0) & (torch.arange(K, device="cuda") + n - K >= at)[:, None]
    assert up.any() and not up.all()
    out, lse, st = d.run()
    assert st == 0
    assert torch.equal(torch.isnan(out), up[..., None].expand(K, H, DL)) and torch.equal(torch.isnan(lse), up)


def test_prefill_rows_that_see_an_infinite_score():
    p = Prefill([300], [700], 2, seed=6)
    p.kr[500, 0] = float("inf")
    out, lse, _ = p.run()
    up = (p.q[..., 128] > 0) & (torch.arange(300, device="cuda") + 400 >= 500)[:, None]
    assert torch.equal(torch.isnan(out), up[..., None].expand(300, 2, 128)) and torch.equal(torch.isnan(lse), up)


# ----------------------------------------------------------- fp16 weights far below the largest
#
# One key scores `drop` above the others (in powers of two) and has value 0, the n others score 0 and
# have value 1.  The output is z / (1 + z) with z = n 2^-drop.  An fp16 weight (scaled by 2^7) is off by
# at most 2^-11 of it or, below the normal range, by 2^-25 / 2^7 = 2^-32 of the row's largest.  A score
# is one product of exact operands with a factor that is 2^-23 off, 2^-16 with the exponential's own
# error; the n / 16 sums of a product are 2^-23 off each.

DROPS = [12.0, 17.25, 21.375, 25.125]  # exact in bf16


def sink_check(out, lse, n, drop, dtype):
    z = n * 2.0 ** -drop
    o = z / (1 + z)
    lim = (UNIT[TYPES[dtype]] + 2.0 ** -15 + n / 16 * 2.0 ** -23) * o
    if dtype == "f16":
        lim += n * 2.0 ** -32 / (1 + z)
    err = (out.double() - o).abs().max().item()
    assert err <= lim, (err, lim, o)
    want = drop * np.log(2) + np.log1p(z)
    err = (lse.double() - want).abs().max().item()
    assert err <= 2.0 ** -16 + 2.0 ** -20 * (1 + want), (err, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,n", [(304, 2048), (1, 131072), (152, 131072)])
@pytest.mark.parametrize("H", [3, 24, 40])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("drop", DROPS)
def test_decode_keeps_small_weights_beside_a_large_one(drop, where, H, R, n, dtype):
    page, dt = 64, TYPES[dtype]
    pages = n // page + 1
    cache = torch.zeros(pages, page, W, dtype=dt, device="cuda")
    x = cache.view(-1, W)
    x[: n + 1, :DL] = 1
    sink = 0 if where == "first" else n
    x[sink, :DL] = 0
    x[sink, DL] = drop
    table = torch.arange(pages, device="cuda", dtype=torch.int32).expand(R, pages).contiguous()
    ql, qr = torch.zeros(R, H, DL, dtype=dt, device="cuda"), torch.zeros(R, H, DR, dtype=dt, device="cuda")
    qr[..., 0] = 1
    out, lse = torch.empty(R, H, DL, device="cuda"), torch.empty(R, H, device="cuda")
    ws = torch.empty(kda.kda_latent_decode_workspace_size(R, 1, H), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_latent_decode(ql, qr, cache, table, i32([n + 1] * R), out, ws, scale=float(np.log(2)), lse=lse,
                          dev_status=st)
    assert int(st) == 0
    sink_check(out, lse, n, drop, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("drop", DROPS)
def test_prefill_keeps_small_weights_beside_a_large_one(drop, where, dtype):
    n = 131072
    p = Prefill([3], [n + 1], 2, dtype, seed=1)
    sink = 0 if where == "first" else n
    p.q.zero_()
    p.q[..., 128] = 1
    p.kr.zero_()
    p.kr[sink, 0] = drop
    p.kv.zero_()
    p.kv[..., 128:] = 1
    p.kv[sink, :, 128:] = 0
    out, lse, st = p.run(out_dtype=torch.float32, scale=float(np.log(2)), flags=kda.KDA_LATENT_FULL)
    assert st == 0
    sink_check(out, lse, n, drop, dtype)


# ----------------------------------------------------------- joins of split requests
#
# With zero queries every weight is exactly 1 and the sum exactly the number of keys.  Channel j of key p
# is 1 where p falls into the j-th of 512 equal stretches of the request, else 0: the output is the share
# of seen keys in each stretch, and a part that is lost, doubled or left over from elsewhere moves whole
# channels by all they hold.  The counts are exact in fp32; the store, the reciprocal and a join's factors
# leave 2^-20 of each.
#
# Requests, positions and heads reach: one and several row tiles, more and fewer (request, row tile)s
# than blocks, and with more than 8 x 152 token tiles the turns between requests that count in the ranges
# (2 tiles up to 32 query rows, 6 above).

JOINS = [
    # R, K, H, longest, page
    (40, 1, 8, 6000, 16), (40, 1, 24, 6000, 64), (300, 1, 16, 800, 32), (300, 2, 16, 800, 64), (1300, 1, 4, 130, 16),
    (30, 3, 40, 4000, 16), (200, 7, 32, 500, 16), (100, 1, 128, 1600, 64), (1500, 1, 40, 90, 8),
    (3, 1, 16, 50000, 64), (2, 5, 24, 30000, 48), (1, 1, 128, 90000, 16), (5, 16, 16, 9000, 8),
]


def stretches(n, dtype):
    x = torch.zeros(n, W, dtype=dtype, device="cuda")
    p = torch.arange(n, device="cuda")
    x[p, p * DL // max(n, 1)] = 1
    x[:, DL:] = 1
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,K,H,longest,page", JOINS)
def test_decode_joins_every_part_once(R, K, H, longest, page, dtype):
    dt = TYPES[dtype]
    rng = np.random.Generator(np.random.PCG64(R + H))
    lens = rng.integers(0, longest + 1, R) if R > 1 else np.array([longest])
    lens[R // 2] = longest
    if R > 4:
        lens[1], lens[2] = 0, 1
    q_len = rng.integers(0, K + 1, R) if K > 1 else np.ones(R, np.int64)
    used = -(-lens // page)
    cache = torch.full((int(used.sum()) + 1, page, W), float("nan"), dtype=dt, device="cuda")
    table = torch.full((R, int(used.max()) + 1), -3, dtype=torch.int32, device="cuda")
    at = 0
    for r in range(R):
        n, u = int(lens[r]), int(used[r])
        cache[at:at + u].view(-1, W)[:n] = stretches(n, dt)
        table[r, :u] = torch.arange(at, at + u, device="cuda", dtype=torch.int32)
        at += u
    ql, qr = torch.zeros(R * K, H, DL, dtype=dt, device="cuda"), torch.zeros(R * K, H, DR, dtype=dt, device="cuda")
    out = torch.full((R * K, H, DL), float("nan"), device="cuda")
    lse = torch.full((R * K, H), float("nan"), device="cuda")
    ws = torch.full((kda.kda_latent_decode_workspace_size(R, K, H),), 255, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_latent_decode(ql, qr, cache, table, i32(lens), out, ws, K=K, q_len=i32(q_len), scale=SCALE, lse=lse,
                          dev_status=st)
    assert int(st) == 0
    n = torch.from_numpy(lens).cuda().double()
    qn = torch.from_numpy(q_len).cuda()
    t = torch.arange(K, device="cuda")
    seen = (n[:, None] - qn[:, None] + t[None] + 1).clamp(min=0)  # [R, K]: keys 0 .. seen - 1
    seen = torch.where(t[None] < qn[:, None], torch.minimum(seen, n[:, None]), 0.0).flatten()
    n = n.repeat_interleave(K)
    # keys below p that fall into stretches below j: ceil(j n / 512), so far as they are seen
    j = torch.arange(DL + 1, device="cuda", dtype=torch.float64)
    upto = torch.minimum(torch.ceil(j[None] * n[:, None] / DL), seen[:, None])
    want = torch.where(seen[:, None] > 0, (upto[:, 1:] - upto[:, :-1]) / seen.clamp(min=1)[:, None], 0.0)
    err = (out.double() - want[:, None]).abs()
    assert (err <= 2.0 ** -20 * want[:, None]).all(), err.max().item()
    some = seen > 0
    z = seen.clamp(min=1).log()
    assert ((lse.double() - z[:, None]).abs()[some] <= 2.0 ** -20 * (1 + z[:, None])[some]).all()
    assert (lse[~some] == -torch.inf).all()


@pytest.mark.parametrize("R,K,H,n", [(1, 1, 16, 40000), (3, 1, 32, 20011), (1, 7, 32, 30000), (40, 1, 8, 3000), (2, 2, 64, 9000)])
def test_decode_of_long_requests_is_as_close_as_rounded_weights_allow(R, K, H, n):
    # weights are rounded to bf16 independently of one another: over all channels and rows the outputs are
    # off by no more than u sqrt(sum p^2 v^2) in the mean square, and by 2 e A from scores that are e off.
    # One of 152 parts lost or doubled moves them several times as far.
    d = Decode([n - 37 * r for r in range(R)], K, H, 64, seed=R + H)
    out, lse, st = d.run(out_dtype=torch.float32)
    assert st == 0
    for r in range(0, R, 7):
        rows = slice(r * K, (r + 1) * K)
        x = d.tokens[r].double()
        q = torch.cat([d.ql, d.qr], 2)[rows].reshape(K * H, W).double()
        L = d.lens[r]
        t = torch.arange(K, device="cuda").repeat_interleave(H)
        seen = torch.arange(L, device="cuda")[None] <= (L - K + t)[:, None]
        p = torch.softmax((q @ x.T * SCALE).masked_fill(~seen, -torch.inf), 1)
        v = x[:, :DL]
        e = 64 * 2.0 ** -24 * SCALE * (q.abs() @ x.abs().T).amax()
        got, want = out[rows].double().view(K * H, DL), p @ v
        lim = 2.0 ** -8 * (p.square() @ v.square()).mean().sqrt() + 2 * e * (p @ v.abs()).square().mean().sqrt()
        err = (got - want).square().mean().sqrt()
        assert err <= lim, (r, err.item(), lim.item())


# ----------------------------------------------------------- a chunk behind an appended context


def test_prefill_of_a_chunk_behind_its_appended_context():
    # two chunks appended to a paged cache; the second's keys are expanded from the rows that the cache holds
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    H, page, lens = 3, 16, [(200, 90), (37, 140)]  # (context, chunk) of each sequence
    r = lambda *n: torch.randn(*n, generator=g, device="cuda").bfloat16()  # noqa: E731
    total = sum(a + b for a, b in lens)
    up = (torch.randn(DL, H * 256, generator=g, device="cuda") * DL ** -0.5).bfloat16()
    cache = torch.full((total // page + 4, page, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    places = torch.randperm(cache.shape[0] * page, generator=g, device="cuda")[:total].to(torch.int32)
    kv, st = r(total, W), torch.zeros(1, dtype=torch.int32, device="cuda")
    first, chunk, at = [], [], 0
    for a, b in lens:
        first += range(at, at + a)
        chunk += range(at + a, at + a + b)
        at += a + b
    q = r(len(chunk), H, 192)
    for part in (first, chunk):
        part = torch.tensor(part, device="cuda")
        kda.kda_latent_append(kv[part], cache, places[part], dev_status=st)
    rows = cache.view(-1, W)[places.long()]
    assert torch.equal(rows, kv)
    k = (rows[:, :DL] @ up).view(total, H, 256)
    out = torch.empty(len(chunk), H, 128, device="cuda")
    lse = torch.empty(len(chunk), H, device="cuda")
    kda.kda_latent_prefill(q, k[..., :128], rows[:, DL:], k[..., 128:], i32([0, 90, 230]), i32([0, 290, 467]), out,
                           scale=SCALE, lse=lse, dev_status=st)
    assert int(st) == 0
    p = Prefill([90, 140], [290, 177], H)
    p.q, p.kv, p.kr = q, k, rows[:, DL:]
    p.check((out, lse, 0))
