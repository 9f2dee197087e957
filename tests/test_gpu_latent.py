"""Latent attention (append, absorbed decode over a paged cache, expanded prefill) against its
definition in 64 bits.

Bound of an output channel, from the roundings of the computation: with u the unit roundoff of the
input type (2^-8 bf16, 2^-11 fp16), A = sum_p p |v| and e the error of a score,
  |o - o_ref| <= u A            (weights rounded once for the product with the values)
              + 2 e A           (softmax of scores that are e off)
              + u_out |o|       (the stored result)
              + n 2^-24 max|v|  (fp16 weights below its normal range; fp32 sums)
A score is a sum of at most 36 steps of 16 products accumulated in fp32, so
e <= 64 * 2^-24 * scale * sum |q||k|, and lse is off by at most e + 2^-20 (1 + |lse|)."""
import numpy as np
import pytest
import torch

from helpers import i32

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu

DL, DR, W = 512, 64, 576
SCALE = 192 ** -0.5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def attend(q, k, v, seen, scale):
    """Definition in 64 bits over rows q [n, d], keys k [L, d], values v [L, e], seen [n, L].
    Returns (o, lse, bound of o without the output rounding, bound of lse)."""
    n, u = k.shape[0], UNIT[q.dtype]
    q, k, v = q.double(), k.double(), v.double()
    seen_any = seen.any(1)
    v = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v)) if n else v
    k = torch.where(seen.any(0)[:, None], k, torch.zeros_like(k)) if n else k
    if n == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
        inf = torch.full((q.shape[0],), -torch.inf, dtype=torch.float64, device=q.device)
        return z, inf, z, torch.zeros_like(inf)
    s = (q @ k.T * scale).masked_fill(~seen, -torch.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - torch.where(seen_any, lse, 0.0)[:, None])
    e = 64 * 2.0 ** -24 * abs(scale) * (q.abs() @ k.abs().T).masked_fill(~seen, 0).amax(1)
    A = p @ v.abs()
    bound = (u + 2 * e[:, None]) * A + n * 2.0 ** -24 * v.abs().max()
    return p @ v, lse, bound, e + 2.0 ** -20 * (1 + torch.where(seen_any, lse.abs(), 0.0))


def close(out, lse, ref, where=""):
    o, z, bo, bz = ref
    err = (out.double() - o).abs()
    lim = bo + UNIT[out.dtype] * (o.abs() + bo) + 1e-30
    assert torch.isfinite(out).all(), where
    worst = (err / lim).max().item() if err.numel() else 0.0
    assert worst <= 1.0, (where, "out", worst)
    none = torch.isinf(z)
    assert torch.equal(lse[none], torch.full_like(lse[none], -torch.inf)), where
    worst = ((lse.double() - z).abs() / bz)[~none]
    assert worst.numel() == 0 or worst.max().item() <= 1.0, (where, "lse", worst.max().item())


# ------------------------------------------------------------------------------------ append


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,page,normed", [(1, 64, True), (7, 8, False), (257, 48, True), (1000, 16, True)])
def test_append(T, page, normed, dtype):
    g, dt = gen(T), TYPES[dtype]
    P = 2 * T // page + 2
    wide = randn(g, T, 600, dtype=dt, std=2.0)
    kv = wide[:, 8:8 + W]  # rows of a wider projection
    pool = randn(g, P, 2, page, W, dtype=dt)
    cache = pool[:, 1]  # pages of two layers side by side
    before = pool.clone()
    w = randn(g, DL, dtype=dt) if normed else None
    slot = torch.randperm(P * page, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 3:
        slot[2] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_latent_append(kv, cache, slot, weight=w, eps=1e-5, dev_status=st)
    want = before.double()
    for t in range(T):
        if slot[t] < 0:
            continue
        x = kv[t].double()
        if normed:
            x[:DL] *= w.double() / (x[:DL].square().mean() + 1e-5).sqrt()
        want[slot[t] // page, 1, slot[t] % page] = x
    # one rounding of an fp32 result that is within 2^-21 of the exact one
    assert ((pool.double() - want).abs() <= (UNIT[dt] + 2.0 ** -20) * want.abs() + 1e-7).all()
    assert torch.equal(pool[:, 0], before[:, 0])
    assert int(st) == 0


def test_append_reports_a_place_past_the_cache_and_skips_it():
    g = gen(1)
    kv, cache = randn(g, 3, W), randn(g, 2, 8, W)
    before = cache.clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_latent_append(kv, cache, i32([16, 3, 2 ** 31 - 1]), dev_status=st)
    assert int(st) == kda.KDA_DEV_BAD_SLOT
    before.view(-1, W)[3] = kv[1]
    assert torch.equal(cache, before)


def test_append_offsets_past_32_bits():
    cache = torch.zeros(60000, 64, W, dtype=torch.bfloat16, device="cuda")  # 2.2e9 elements
    kv = randn(gen(2), 2, W)
    kda.kda_latent_append(kv, cache, i32([60000 * 64 - 1, 0]))
    assert torch.equal(cache[-1, -1], kv[0]) and torch.equal(cache[0, 0], kv[1])
    assert int(cache.view(torch.int16).ne(0).any(2).sum()) == 2


# ------------------------------------------------------------------------------------ decode


class Decode:
    """A paged cache with requests of the given lengths; everything outside their tokens is NaN."""

    def __init__(self, lens, K, H, page, dtype="bf16", seed=0, std=1.0, extra=2, rising=False):
        g, dt = gen(seed), TYPES[dtype]
        self.lens, self.K, self.H, self.page, self.dt = lens, K, H, page, dt
        R = len(lens)
        used = [-(-n // page) for n in lens]
        self.cache = torch.full((sum(used) + extra, page, W), float("nan"), dtype=dt, device="cuda")
        order = torch.randperm(self.cache.shape[0], generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((R, max(used + [1]) + 1), -7, dtype=torch.int32, device="cuda")
        self.tokens, at = [], 0
        for r, n in enumerate(lens):
            x = randn(g, n, W, dtype=dt, std=std)
            if rising:  # later keys score higher: the running maximum keeps moving
                x = (x.float() * torch.linspace(0.05, 3, n, device="cuda")[:, None]).to(dt)
            self.table[r, : used[r]] = order[at:at + used[r]]
            at += used[r]
            for i in range(used[r]):
                part = x[i * page:(i + 1) * page]
                self.cache[self.table[r, i].long(), : part.shape[0]] = part
            self.tokens.append(x)
        self.ql, self.qr = randn(g, R * K, H, DL, dtype=dt), randn(g, R * K, H, DR, dtype=dt)
        self.seq_len = i32(lens)

    def run(self, out_dtype=None, q_len=None, scale=SCALE, stream=None, **kw):
        R = len(self.lens)
        out = torch.full((R * self.K, self.H, DL), float("nan"), dtype=out_dtype or self.dt, device="cuda")
        lse = torch.full((R * self.K, self.H), float("nan"), device="cuda")
        ws = torch.full((kda.kda_latent_decode_workspace_size(R, self.K, self.H),), 255, dtype=torch.uint8,
                        device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(ql=self.ql, qr=self.qr, cache=self.cache, table=self.table, seq_len=self.seq_len, out=out)
        args.update(kw)
        if stream is not None:
            torch.cuda.synchronize()
        kda.kda_latent_decode(args["ql"], args["qr"], args["cache"], args["table"], args["seq_len"],
                              args["out"], ws, K=self.K, q_len=None if q_len is None else i32(q_len),
                              scale=scale, lse=lse, dev_status=st, stream=stream)
        if stream is not None:
            stream.synchronize()
        return args["out"], lse, int(st)

    def ref(self, r, q_len=None, scale=SCALE, hole=None):
        K, H, n = self.K, self.H, self.lens[r]
        ql = K if q_len is None else q_len[r]
        t = torch.arange(K, device="cuda").repeat_interleave(H)
        seen = (torch.arange(n, device="cuda")[None] <= (n - ql + t)[:, None]) & (t < ql)[:, None]
        if hole is not None:
            seen[:, hole] = False
        q = torch.cat([self.ql, self.qr], 2)[r * K:(r + 1) * K].reshape(K * H, W)
        o, z, bo, bz = attend(q, self.tokens[r], self.tokens[r][:, :DL], seen, scale)
        return o.view(K, H, DL), z.view(K, H), bo.view(K, H, DL), bz.view(K, H)

    def check(self, got, q_len=None, scale=SCALE, skip=(), **kw):
        out, lse, _ = got
        for r in range(len(self.lens)):
            if r in skip:
                continue
            rows = slice(r * self.K, (r + 1) * self.K)
            close(out[rows], lse[rows], self.ref(r, q_len, scale, **kw), f"request {r}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,K,H,page", [
    ([1], 1, 1, 64), ([0], 1, 2, 16), ([5, 0, 64, 65, 63], 1, 16, 16), ([128, 127, 129, 1], 1, 32, 64),
    ([700, 3, 1500], 1, 24, 48), ([333, 64], 1, 128, 128), ([900], 2, 16, 8), ([2049, 70, 7], 7, 32, 32),
    ([1000, 40], 16, 5, 256), ([3], 7, 12, 64), ([100, 20, 6000], 3, 40, 24), ([15], 16, 128, 40),
])
def test_decode(lens, K, H, page, dtype):
    d = Decode(lens, K, H, page, dtype, seed=len(lens) * 31 + K)
    got = d.run()
    assert got[2] == 0
    d.check(got)


@pytest.mark.parametrize("R,H,L,page", [(1, 16, 40000, 64), (3, 32, 20011, 16), (200, 8, 300, 32), (700, 3, 40, 8)])
def test_decode_split_over_many_blocks(R, H, L, page):
    rng = np.random.Generator(np.random.PCG64(R))
    lens = [int(x) for x in rng.integers(0, 2 * L, R)] if R > 1 else [L]
    d = Decode(lens, 1, H, page, seed=R)
    got = d.run()
    assert got[2] == 0
    d.check(got)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("std,scale", [(4.0, SCALE), (1.0, 0.0), (2.0, -SCALE), (0.01, SCALE)])
def test_decode_moving_maximum(std, scale, dtype):
    d = Decode([1300, 200], 2, 20, 64, dtype, seed=5, std=std, rising=True)
    d.check(d.run(scale=scale), scale=scale)


def test_decode_query_lengths():
    d = Decode([300, 64, 10, 5, 130], 4, 9, 16, seed=6)
    q_len = [4, 1, 0, 3, 2]
    got = d.run(q_len=q_len)
    assert got[2] == 0
    d.check(got, q_len=q_len)


def test_decode_more_positions_than_tokens_leaves_empty_rows():
    d = Decode([2, 0, 1], 5, 7, 16, seed=7)
    got = d.run()
    d.check(got)
    out, lse, _ = got
    assert (out[5:10] == 0).all() and torch.isinf(lse[5:10]).all()
    assert (out[:3] == 0).all() and not (out[3:5] == 0).all()


@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
def test_decode_output_types(out_dtype):
    d = Decode([257, 40], 2, 33, 32, seed=8)
    d.check(d.run(out_dtype=TYPES[out_dtype]))


def test_decode_strided_queries_output_and_pages():
    d = Decode([500, 77, 64], 2, 12, 16, seed=9)
    R2, H = 6, 12
    plain = d.run()
    # head-major products, as a batched matrix product over heads leaves and takes them
    ql = d.ql.transpose(0, 1).contiguous().transpose(0, 1)
    qr = torch.cat([d.qr, d.qr], 2)[..., DR:]
    out = torch.full((H, R2, DL), float("nan"), dtype=d.dt, device="cuda").transpose(0, 1)
    layers = torch.full((d.cache.shape[0], 3, d.page, W), float("nan"), dtype=d.dt, device="cuda")
    layers[:, 1] = d.cache
    got = d.run(ql=ql, qr=qr, out=out, cache=layers[:, 1])
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


def test_decode_reports_bad_lengths_and_query_lengths():
    d = Decode([100, 50, 60, 70], 2, 4, 16, seed=10)
    bad = i32([100, -1, 16 * d.table.shape[1] + 1, 70])
    out, lse, st = d.run(seq_len=bad)
    assert st == kda.KDA_DEV_BAD_SEQLEN
    d.check((out, lse, st), skip=(1, 2))
    assert (out[2:6] == 0).all() and torch.isinf(lse[2:6]).all()
    out, lse, st = d.run(q_len=[2, 3, -1, 1])
    assert st == kda.KDA_DEV_BAD_ACCEPT
    d.check((out, lse, st), q_len=[2, 0, 0, 1])
    assert (out[2:6] == 0).all() and torch.isinf(lse[2:6]).all()


def test_decode_with_an_empty_table_or_cache():
    d = Decode([0, 0], 2, 6, 16, seed=17)
    out, lse, st = d.run(table=torch.empty(2, 0, dtype=torch.int32, device="cuda"))
    assert st == 0 and (out == 0).all() and torch.isinf(lse).all()
    empty = torch.empty(0, 16, W, dtype=d.dt, device="cuda")
    out, lse, st = d.run(cache=empty, table=i32([[0, 0], [1, 1]]), seq_len=i32([20, 0]))
    assert st == kda.KDA_DEV_BAD_SLOT and (out == 0).all() and torch.isinf(lse).all()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_latent_append(torch.zeros(2, W, dtype=d.dt, device="cuda"), empty, i32([-1, 0]), dev_status=st)
    assert int(st) == kda.KDA_DEV_BAD_SLOT


def test_decode_masks_the_tokens_of_a_bad_page():
    d = Decode([200, 90], 1, 10, 16, seed=11)
    for bad in (-1, d.cache.shape[0], 2 ** 31 - 1):
        table = d.table.clone()
        table[0, 3] = bad
        out, lse, st = d.run(table=table)
        assert st == kda.KDA_DEV_BAD_SLOT
        close(out[:1], lse[:1], d.ref(0, hole=slice(48, 64)), "with a hole")
        close(out[1:], lse[1:], d.ref(1), "untouched")


def test_decode_repeats_bit_for_bit_and_on_another_stream():
    d = Decode([3000, 10, 777], 3, 16, 64, seed=12)
    a = d.run()
    b = d.run(stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_offsets_past_32_bits():
    d = Decode([150], 1, 16, 64, seed=13)
    big = torch.full((60000, 64, W), float("nan"), dtype=d.dt, device="cuda")  # 2.2e9 elements
    table = torch.tensor([[59999, 3, 59998, 0]], dtype=torch.int32, device="cuda")
    for i in range(3):
        big[table[0, i].long()] = d.cache[d.table[0, i].long()]
    d.check(d.run(cache=big, table=table))


def test_decode_is_captured_and_replayed():
    d = Decode([800, 33], 1, 16, 64, seed=14)
    R = 2
    out, lse = torch.zeros(R, 16, DL, dtype=d.dt, device="cuda"), torch.zeros(R, 16, device="cuda")
    ws = torch.empty(kda.kda_latent_decode_workspace_size(R, 1, 16), dtype=torch.uint8, device="cuda")

    def step():
        kda.kda_latent_decode(d.ql, d.qr, d.cache, d.table, d.seq_len, out, ws, scale=SCALE, lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # another state of the same buffers: shorter requests
    d.seq_len.copy_(i32([500, 12]))
    d.lens = [500, 12]
    d.tokens = [d.tokens[0][:500], d.tokens[1][:12]]
    graph.replay()
    torch.cuda.synchronize()
    d.check((out, lse, 0))


# ------------------------------------------------------------------------------------ prefill


class Prefill:
    def __init__(self, lq, lk, H, dtype="bf16", seed=0, std=1.0, rising=False, pad=0):
        g, dt = gen(seed), TYPES[dtype]
        self.lq, self.lk, self.H, self.dt = lq, lk, H, dt
        Tq, Tk = sum(lq) + pad, sum(lk) + pad
        self.q = randn(g, Tq, H, 192, dtype=dt)
        self.kv = randn(g, Tk, H, 256, dtype=dt, std=std)
        self.kr = randn(g, Tk, 64, dtype=dt, std=std)
        if rising:
            f = torch.linspace(0.05, 4, Tk, device="cuda")
            self.kv[..., :128] = (self.kv[..., :128].float() * f[:, None, None]).to(dt)
        self.cu_q = i32(np.concatenate([[0], np.cumsum(lq)]))
        self.cu_k = i32(np.concatenate([[0], np.cumsum(lk)]))

    def run(self, out_dtype=None, scale=SCALE, flags=0, stream=None, **kw):
        out = torch.full((self.q.shape[0], self.H, 128), float("nan"), dtype=out_dtype or self.dt, device="cuda")
        lse = torch.full((self.q.shape[0], self.H), float("nan"), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        a = dict(q=self.q, k=self.kv[..., :128], v=self.kv[..., 128:], kr=self.kr, cu_q=self.cu_q,
                 cu_k=self.cu_k, out=out)
        a.update(kw)
        if stream is not None:
            torch.cuda.synchronize()
        kda.kda_latent_prefill(a["q"], a["k"], a["kr"], a["v"], a["cu_q"], a["cu_k"], a["out"], scale=scale,
                               flags=flags, lse=lse, dev_status=st, stream=stream)
        if stream is not None:
            stream.synchronize()
        return a["out"], lse, int(st)

    def check(self, got, scale=SCALE, full=False, skip=()):
        out, lse, _ = got
        a = c = 0
        for n, (nq, nk) in enumerate(zip(self.lq, self.lk)):
            if n not in skip and nq:
                i, j = torch.arange(nq, device="cuda"), torch.arange(nk, device="cuda")
                seen = torch.ones(nq, nk, dtype=torch.bool, device="cuda") if full else \
                    j[None] <= (nk - nq + i)[:, None]
                for h in {0, self.H // 2, self.H - 1}:
                    k = torch.cat([self.kv[c:c + nk, h, :128], self.kr[c:c + nk]], 1)
                    ref = attend(self.q[a:a + nq, h], k, self.kv[c:c + nk, h, 128:], seen, scale)
                    close(out[a:a + nq, h], lse[a:a + nq, h], ref, f"sequence {n} head {h}")
            a, c = a + nq, c + nk


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lq,lk,H", [
    ([1], [1], 1), ([70, 129, 5], [70, 129, 5], 2), ([256], [256], 3), ([255, 257, 1], [300, 257, 4000], 4),
    ([128, 127], [128, 1000], 5), ([1000], [1000], 2), ([511, 64, 700], [1023, 65, 2500], 3),
    ([1, 1, 1, 1], [1, 64, 127, 513], 16), ([2049], [4100], 1),
])
def test_prefill(lq, lk, H, dtype):
    p = Prefill(lq, lk, H, dtype, seed=sum(lq))
    got = p.run()
    assert got[2] == 0
    p.check(got)


@pytest.mark.parametrize("N,most,H", [(900, 40, 2), (350, 700, 3), (33, 1100, 8)])
def test_prefill_many_sequences(N, most, H):
    # more sequences than one scan step holds, more blocks than pairs of SMs, some without rows or keys
    rng = np.random.Generator(np.random.PCG64(N))
    lq = [int(x) for x in rng.integers(0, most, N)]
    lk = [max(0, n + int(x)) for n, x in zip(lq, rng.integers(-3, 50, N))]
    p = Prefill(lq, lk, H, seed=N)
    got = p.run()
    assert got[2] == 0
    p.check(got)


def test_prefill_rows_without_keys():
    # fewer keys than queries leave the first rows empty; sequences without queries or keys
    p = Prefill([300, 0, 10, 40, 3], [170, 50, 0, 1, 3], 2, seed=3)
    got = p.run()
    assert got[2] == 0
    p.check(got)
    assert (got[0][:130] == 0).all() and torch.isinf(got[1][:130]).all()


def test_prefill_without_any_key():
    p = Prefill([20], [0], 2, seed=4)
    got = p.run()
    assert (got[0] == 0).all() and torch.isinf(got[1]).all() and got[2] == 0


@pytest.mark.parametrize("lq,lk", [([100, 300], [40, 700]), ([5], [0]), ([260], [129])])
def test_prefill_full_mask(lq, lk):
    p = Prefill(lq, lk, 3, seed=5)
    p.check(p.run(flags=kda.KDA_LATENT_FULL), full=True)


def test_prefill_merges_with_an_earlier_context_through_lse():
    # causal over the new keys merged with the full mask over the context = causal over both
    p = Prefill([200], [900], 2, seed=6)
    whole = p.run(out_dtype=torch.float32)
    cu = lambda n: i32([0, n])  # noqa: E731
    parts = []
    for a, b, f in ((0, 700, kda.KDA_LATENT_FULL), (700, 900, 0)):
        parts.append(p.run(out_dtype=torch.float32, flags=f, k=p.kv[a:b, :, :128], v=p.kv[a:b, :, 128:],
                           kr=p.kr[a:b], cu_k=cu(b - a)))
    lse = torch.logaddexp(parts[0][1], parts[1][1])
    out = sum(torch.exp(z - lse)[..., None] * o for o, z, _ in parts)
    # weights rounded relative to different maxima: twice the bound of one rounding
    assert (out - whole[0]).norm() <= 2 * 2.0 ** -8 * whole[0].norm()
    assert (lse - whole[1]).abs().max() <= 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("std,scale", [(3.0, SCALE), (1.0, 0.0), (1.5, -SCALE), (0.01, SCALE)])
def test_prefill_moving_maximum(std, scale, dtype):
    p = Prefill([600, 300], [1500, 300], 2, dtype, seed=7, std=std, rising=True)
    p.check(p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
def test_prefill_output_types(out_dtype):
    p = Prefill([130, 77], [130, 300], 3, seed=8)
    p.check(p.run(out_dtype=TYPES[out_dtype]))


def test_prefill_strides():
    p = Prefill([300, 20], [333, 90], 4, seed=9)
    plain = p.run()
    q = p.q.transpose(0, 1).contiguous().transpose(0, 1)
    k, v = p.kv[..., :128].contiguous(), p.kv[..., 128:].transpose(0, 1).contiguous().transpose(0, 1)
    kr = torch.cat([p.kr, p.kr], 1)[:, 64:]
    out = torch.full((4, 320, 136), float("nan"), dtype=p.dt, device="cuda").transpose(0, 1)[..., :128]
    got = p.run(q=q, k=k, v=v, kr=kr, out=out)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


def test_prefill_does_not_see_its_neighbours():
    # rows outside a sequence hold NaN: the tiles at its end read them, the results must not
    p = Prefill([70, 40, 100], [200, 90, 100], 2, seed=10, pad=5)
    p.kv[200:290] = float("nan")
    p.kr[200:290] = float("nan")
    p.q[70:110] = float("nan")
    p.kv[390:] = float("nan")
    p.kr[390:] = float("nan")
    out, lse, _ = p.run()
    p.check((out, lse, 0), skip=(1,))
    assert torch.isnan(out[210:]).all() and torch.isnan(lse[210:]).all()  # past the last sequence: not written


def test_prefill_reports_bad_bounds():
    p = Prefill([60, 50, 40], [60, 50, 40], 2, seed=11)
    out, lse, st = p.run(cu_k=i32([0, 60, 160, 150]))  # sequence 1 past the keys, 2 decreasing
    assert st == kda.KDA_DEV_BAD_SEQLEN
    p.check((out, lse, 0), skip=(1, 2))
    assert torch.isnan(out[60:]).all()
    out, lse, st = p.run(cu_q=i32([0, 60, -3, 150]))
    assert st == kda.KDA_DEV_BAD_SEQLEN
    p.check((out, lse, 0), skip=(1, 2))


def test_prefill_repeats_bit_for_bit_and_on_another_stream():
    p = Prefill([700, 90], [1700, 90], 3, seed=12)
    a = p.run()
    b = p.run(stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prefill_is_captured_and_replayed():
    p = Prefill([300, 1200], [300, 1500], 3, seed=16)
    out = torch.zeros(1500, 3, 128, dtype=p.dt, device="cuda")
    lse = torch.zeros(1500, 3, device="cuda")

    def step():
        kda.kda_latent_prefill(p.q, p.kv[..., :128], p.kr, p.kv[..., 128:], p.cu_q, p.cu_k, out, scale=SCALE, lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # the replay reads the bounds anew
    p.lq, p.lk = [700, 800], [1000, 800]
    p.cu_q.copy_(i32([0, 700, 1500]))
    p.cu_k.copy_(i32([0, 1000, 1800]))
    graph.replay()
    torch.cuda.synchronize()
    p.check((out, lse, 0))


def test_decode_agrees_with_prefill_on_the_same_model():
    """Both forms of one layer: keys and values expanded from the latent vectors, and the query
    and output products absorbed; the last query of each sequence."""
    g = gen(15)
    H, lens, page = 4, [50, 333], 16
    wk, wv = randn(g, H, 128, DL, std=DL ** -0.5).double(), randn(g, H, 128, DL, std=DL ** -0.5).double()
    d = Decode(lens, 1, H, page, seed=15)
    qn = randn(g, 2, H, 128).double()
    ql = torch.einsum("rhd,hdl->rhl", qn, wk)
    out, _, _ = d.run(ql=ql.bfloat16(), out_dtype=torch.float32)
    absorbed = torch.einsum("rhl,hdl->rhd", out.double(), wv)
    toks = torch.cat(d.tokens)
    k = torch.einsum("tl,hdl->thd", toks[:, :DL].double(), wk).bfloat16()
    v = torch.einsum("tl,hdl->thd", toks[:, :DL].double(), wv).bfloat16()
    q = torch.cat([qn.bfloat16(), d.qr], 2)
    o2 = torch.empty(2, H, 128, device="cuda")
    kda.kda_latent_prefill(q, k, toks[:, DL:].contiguous(), v, i32([0, 1, 2]),
                           i32([0, lens[0], sum(lens)]), o2, scale=SCALE)
    # two bf16 roundings of keys / queries on either side move the scores by about 2^-8 of their size
    assert (absorbed - o2.double()).norm() <= 0.03 * o2.double().norm()
