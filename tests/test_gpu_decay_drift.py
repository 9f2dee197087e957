"""Thousands of decoded tokens under one fixed slope: what is off in the decay alike at every token would add up in the
state.  Against the recurrence in 64 bits.

Tolerances are relative 2-norms over a head's state.  A token's product and sum are rounded once each, by 2^-24 of the
state at most and at random in sign (the keys' summands change the last bits): sqrt(2 n) 2^-24 / sqrt(3) after n tokens,
of which twice are allowed.  The decay of a call's K positions is a sum of K logs in fp32, (K - 1) 2^-24 of it off at most, and its
exponential less one 2^-23 of itself, at each call alike: over the state's memory of at most 1 / |g| tokens that is
(K + 1) 2^-24 in all.  A key enters once, with a product of up to K - 1 exponentials that are 2^-23 off each.
"""
import pytest
import torch

import serving_kda_chunk_gb300 as kda
from test_gpu_decay import BF16, D, F32, gen, i32, randn

pytestmark = pytest.mark.gpu
SLOPES = [-1e-4, -2.5e-4, -1e-3, -4e-3]


@pytest.mark.parametrize("source", ["head", "token"])
@pytest.mark.parametrize("K,outputs", [(1, True), (4, False), (8, True), (8, False), (16, True)])
def test_decode_of_thousands_of_tokens_under_a_fixed_slope(K, outputs, source):
    n, H = 4096, len(SLOPES)
    g = gen(21)
    head = torch.tensor(SLOPES, device="cuda")
    token = head.expand(n, H).contiguous()
    q, k, v = (randn(g, n, H, D, dt=BF16, std=s) for s in (1.0, D ** -0.5, 1.0))
    pool = randn(g, 1, H, D, D, std=0.3)
    S, a = pool[0].double(), head.double().exp()[:, None, None]
    out, slot = torch.empty(K, H, D, dtype=BF16, device="cuda") if outputs else None, i32([0])
    for t in range(0, n, K):
        r = slice(t, t + K)
        decay = dict(head_decay=head) if source == "head" else dict(log_decay=token[r])
        kda.kda_decay_decode(q[r] if outputs else None, k[r], v[r], pool, slot, out, K=K, **decay)
    for t in range(n):
        S = S * a + v[t, :, :, None].double() * k[t, :, None, :].double()
    off = (pool[0].double() - S).flatten(1).norm(dim=1) / S.flatten(1).norm(dim=1)
    ulp = 2.0 ** -24
    assert off.max().item() <= 2 * (2 * n / 3) ** 0.5 * ulp + (K + 1) * ulp + 2 * (K - 1) * ulp, off.tolist()


@pytest.mark.parametrize("K", [1, 5])
@pytest.mark.parametrize("g", [-0.6, -0.75, -5.0, -30.0, -103.9, -104.0, -200.0, float("-inf"), 0.0, 3.0])
def test_decode_of_one_decay(K, g):
    """On both sides of where the exponential is taken less one; a forgotten state leaves nothing, one that is kept all."""
    H = 2
    x = gen(22)
    k, v = randn(x, K, H, D, dt=BF16, std=D ** -0.5), randn(x, K, H, D, dt=BF16)
    k[K - 1], v[K - 1] = 0, 0
    pool = randn(x, 1, H, D, D)
    S, rate = pool[0].double(), torch.tensor([min(g, 0.0)], dtype=F32).double().exp().item()
    token = torch.zeros(K, H, device="cuda")
    token[K - 1] = g  # the last of the positions, without a key of its own
    for t in range(K):
        S = S * (rate if t == K - 1 else 1.0) + v[t, :, :, None].double() * k[t, :, None, :].double()
    kda.kda_decay_decode(None, k, v, pool, i32([0]), None, K=K, log_decay=token)
    got = pool[0].double()
    if g <= -104:
        assert (got == 0).all()
        return
    # fp32: exponential 2^-23 of itself, a rounding each for K sums and K products; and where fp32 holds no smaller steps, the
    # decay is 2^-149 off (-103.9: 7.5e-46 counts as 1.4e-45), times the state before it, and the result 2^-149 more
    least = 2.0 ** -149 * (1 + (S / rate).abs().amax((1, 2)))
    assert ((got - S).abs().amax((1, 2)) <= (2 + 2 * K) * 2.0 ** -24 * S.abs().amax((1, 2)) + least).all()


@pytest.mark.parametrize("K", [1, 4, 7, 16])
@pytest.mark.parametrize("g", [0.0, -1e-3, -0.5, -2.0])
def test_infinities_in_a_state_stay_what_they_are(K, g):
    """inf e^g is inf; the other elements of the state are those of a call without them."""
    x = gen(23)
    k, v = randn(x, K, 2, D, dt=BF16, std=D ** -0.5), randn(x, K, 2, D, dt=BF16)
    pool = randn(x, 1, 2, D, D)
    head, inf = torch.full((2,), g, device="cuda"), float("inf")
    want = pool.clone()
    kda.kda_decay_decode(None, k, v, want, i32([0]), None, K=K, head_decay=head)
    pool[0, 0, 3, 5], pool[0, 1, 127, 0] = inf, -inf
    want[0, 0, 3, 5], want[0, 1, 127, 0] = inf, -inf
    kda.kda_decay_decode(None, k, v, pool, i32([0]), None, K=K, head_decay=head)
    assert torch.equal(pool, want)
