"""Token log probabilities, entropy and top alternatives against their definition in 64 bits.

Bounds: fp32 sums of V terms, taken as partial sums of at most a few hundred terms each, with
exponentials of relative error 2^-21: lse is off by at most 2^-19 plus its own rounding, a log
probability by that plus the rounding of the difference x - max (2^-23 of max|x|), the entropy by
2^-19 (1 + entropy) + 2^-22 max|x - max|.  The ids are exact."""
import pytest
import torch

from helpers import i32

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def run(x, tokens, top, entropy=True):
    R = x.shape[0]
    f = lambda *n: torch.full(n, 7.0, device="cuda")  # noqa: E731
    lp, ent, tl = f(R), f(R), f(R, top)
    ids = torch.full((R, top), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_token_logprobs(x, tokens, lp, entropy=ent if entropy else None, top_ids=ids if top else None,
                           top_logprobs=tl if top else None, dev_status=st)
    return lp, ent, ids, tl, int(st)


def check(x, tokens, top, got):
    lp, ent, ids, tl, _ = got
    for i in range(0, x.shape[0], 512):
        s = slice(i, i + 512)
        y = x[s].double()
        d = y - y.amax(1, keepdim=True)  # before the logarithm: |x| may be too large for 64 bits to hold both
        logp = d - d.exp().sum(1, keepdim=True).log()
        p = logp.exp()
        want_e = -torch.where(p > 0, p * logp, 0.0).sum(1)
        big = torch.where(torch.isinf(y), 0.0, y).abs().amax(1)
        gap = (y.amax(1, keepdim=True) - torch.where(torch.isinf(y), y.amax(1, keepdim=True), y)).amax(1)
        lim = 2.0 ** -19 + 2.0 ** -22 * (big + gap)
        tok = tokens[s].long()
        want = logp.gather(1, tok.clamp(0, x.shape[1] - 1)[:, None])[:, 0]
        use = (tok >= 0) & (tok < x.shape[1])
        fin = use & torch.isfinite(want)
        assert ((lp[s].double() - want).abs()[fin] <= lim[fin]).all()
        assert (lp[s][use & ~fin] == -torch.inf).all()
        assert (lp[s][~use] == 0).all()
        assert ((ent[s].double() - want_e).abs() <= 2.0 ** -19 * (1 + want_e) + 2.0 ** -22 * gap).all()
        if top:
            order = torch.sort(y, dim=1, descending=True, stable=True).indices[:, :top]
            assert torch.equal(ids[s].long(), order)
            w = logp.gather(1, order)
            f = torch.isfinite(w)
            assert ((tl[s].double() - w).abs()[f] <= lim[:, None].expand_as(w)[f]).all()
            assert torch.equal(tl[s][~f], w[~f].float())


def logits(R, V, dtype, seed, std=2.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(R, V, generator=g, device="cuda") * std).to(TYPES[dtype])
    return x, torch.randint(0, V, (R,), generator=g, device="cuda").to(torch.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,V,top", [
    (1, 1, 1), (3, 2, 2), (2, 33, 32), (1, 1000, 5), (5, 1023, 0), (4, 4097, 8), (64, 32000, 20),
    (1, 160000, 20), (7, 200003, 32), (2, 1000003, 3), (300, 50001, 1), (2000, 777, 5), (1, 32, 32),
])
def test_logprobs(R, V, top, dtype):
    x, t = logits(R, V, dtype, R + V)
    check(x, t, top, run(x, t, top))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 400])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "steps", "one column", "signed zeros", "peak"])
def test_orders_and_ties(kind, R, dtype):
    V, top = 20011, 32
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    row = {"equal": torch.zeros(V, device="cuda"), "rising": i / 1000, "falling": -i / 1000,
           "steps": torch.floor(i / 977) % 7, "one column": (i % 1024 == 5).float() * (3 + i / V),
           "signed zeros": torch.where(i % 3 == 0, -0.0, 0.0), "peak": (i == 12345).float() * 80}[kind]
    x = row[None].expand(R, V).contiguous().to(TYPES[dtype])
    t = torch.arange(R, device="cuda", dtype=torch.int32) % V
    check(x, t, top, run(x, t, top))


def test_masked_vocabulary():
    x, t = logits(9, 30011, "bf16", 1)
    x[:, ::2] = -torch.inf
    x[0, 10:] = -torch.inf      # fewer finite logits than alternatives
    x[1, 1:] = -torch.inf       # one token left
    x[1, 0] = 3.0
    x[2] = torch.finfo(torch.bfloat16).min
    x[2, 77] = 0
    t[:3] = i32([5, 0, 77])
    check(x, t, 8, run(x, t, 8))


def test_large_and_small_magnitudes():
    x, t = logits(6, 5003, "f32", 2)
    x[0] *= 1e4
    x[1] *= 1e-6
    x[2] += 3e4
    x[3] = -3.0e38
    x[4] = 3.0e38
    x[5, :] = -1e30
    x[5, 9] = 1e30
    lp, ent, ids, tl, _ = got = run(x, t, 5)
    rows = [0, 1, 2, 3, 4]
    check(x[rows], t[rows], 5, tuple(y[rows] for y in got[:4]) + (0,))
    assert ids[5].tolist() == [9, 0, 1, 2, 3] and ent[5] == 0 and tl[5, 0] == 0


def test_rows_without_a_distribution_give_nan_and_distinct_ids():
    x, t = logits(4, 3001, "f32", 3)
    x[0] = -torch.inf
    x[1, 50] = torch.inf
    x[2, 60] = torch.nan
    good = x[3:].clone()
    lp, ent, ids, tl, st = run(x, t, 4)
    assert torch.isnan(lp[:3]).all() and torch.isnan(ent[:3]).all() and st == 0
    assert ids[0].tolist() == [0, 1, 2, 3]
    assert ids[1, 0] == 50 and 60 not in ids[2].tolist()
    check(good, t[3:], 4, (lp[3:], ent[3:], ids[3:], tl[3:], 0))
    x = torch.full((1, 5), torch.nan, device="cuda")
    assert sorted(run(x, i32([1]), 5)[2][0].tolist()) == [0, 1, 2, 3, 4]


def test_padding_and_bad_tokens():
    x, t = logits(4, 500, "bf16", 4)
    t[1], t[2] = -1, 500
    got = run(x, t, 3)
    assert got[4] == kda.KDA_DEV_BAD_SLOT
    check(x, t, 3, got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows_of_any_alignment(dtype):
    x, t = logits(6, 1500, dtype, 5)
    for a in range(0, 9):
        y = x[:, a:a + 1400 + a]
        check(y, t % 1400, 4, run(y, t % 1400, 4))


def test_entropy_is_optional_and_results_repeat():
    x, t = logits(33, 60007, "bf16", 6)
    a, b = run(x, t, 20), run(x, t, 20, entropy=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
    c = run(x, t, 20)
    assert all(torch.equal(u, v) for u, v in zip(a[:4], c[:4]))


def test_offsets_past_32_bits():
    x = torch.zeros(20, 110000003, dtype=torch.bfloat16, device="cuda")  # 2.2e9 elements
    x[19, 7] = 9.0
    y = x[:, :5003]
    t = torch.full((20,), 7, dtype=torch.int32, device="cuda")
    check(y, t, 2, run(y, t, 2))
