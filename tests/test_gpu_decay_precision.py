"""What the decayed calls' fp32 states and their instances for other types and position counts are good for.

A prefill's fp32 state, relative 2-norm over a head.  bf16 keys, decayed in fp32, are split in three parts with nothing
left, fp16 keys in two with 2^-22 of a key or 2^-25 left.  A key's weight: two exponentials (2^-22 each), logs of up to 4 in
fp32 (2^-22 after ln 2, twice) and two roundings of 2^-24: 9.4e-7 at most.  The products' sum: up to 24 tensor-core sums a chunk that
lose 2^-23 each at most: 2.9e-6.  Eight chunks' products and sums: 16 2^-24 = 1e-6.  In all 5e-6.  (Without the third part,
which is spread over 0 to 2^-15 of a key's leading power of two, the state would be 1.2e-5 off.)
"""
import pytest
import torch

from test_gpu_decay import (BF16, D, F16, F32, call_decode, call_prefill, decode_case, i32, prefill_case, rel, tol,
                            want_decode, want_prefill)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("lens", [[1000], [128, 700, 65], [3]], ids=str)
def test_prefill_state_is_good_to_fp32(dt, lens):
    c = prefill_case(lens, 3, 1, dt, "token", seed=31)
    c["token"].mul_(0.1)  # some 0.01 a token: up to 2 a chunk
    N = len(lens)
    init, final = i32(list(range(N))), i32([N + n for n in range(N)])
    want = want_prefill(c, init)
    for ws in (True, None):
        pool, out = c["pool"].clone(), torch.zeros(c["T"], 3, D, dtype=dt, device="cuda")
        assert call_prefill(c, out, pool, init, final, ws=ws) == 0
        for n, (_, s) in enumerate(want):
            assert rel(pool[N + n], s[-1]) <= 5e-6, n


def test_prefill_state_of_small_fp16_keys():
    """A decayed fp16 key is 2^-25 off at most where that is more than 2^-22 of it, as an fp16 key of that size is itself."""
    c = prefill_case([600], 2, 2, F16, "none", seed=32)
    c["k"].mul_(1e-4 * D ** 0.5)
    c["pool"].zero_()
    want = want_prefill(c, None)[0][1][-1]
    pool, out = c["pool"].clone(), torch.zeros(c["T"], 2, D, dtype=F16, device="cuda")
    assert call_prefill(c, out, pool, None, i32([0])) == 0
    assert rel(pool[0], want) <= 2.0 ** -25 / c["k"][:600].double().square().mean().sqrt().item() + 5e-6


def test_decode_goes_on_where_the_prefill_ends():
    """A prompt and 300 tokens behind it, one by one and seven at a time."""
    n, extra = 500, 294
    c = prefill_case([n + extra], 3, 3, BF16, "token", extra=0, seed=33)
    c["token"].mul_(0.1)
    want = want_prefill(c, None)[0][1]
    cut = {**c, "q": c["q"][:n], "k": c["k"][:n], "v": c["v"][:n], "token": c["token"][:n], "cu": i32([0, n]), "T": n, "lens": [n]}
    for K in (1, 7):
        pool, out = c["pool"].clone(), torch.zeros(n, 3, D, dtype=BF16, device="cuda")
        assert call_prefill(cut, out, pool, None, i32([1])) == 0
        for t in range(n, n + extra, K):
            r = slice(t, t + K)
            row = dict(q=None, k=c["k"][r], v=c["v"][r], head=None, token=c["token"][r], K=K, slot=i32([1]))
            assert call_decode(row, pool, None) == 0
        # the prefill's 5e-6, and two roundings of 2^-24 a token
        assert rel(pool[1], want[-1]) <= 5e-6 + 2 * (2 * extra / 3) ** 0.5 * 2.0 ** -24


@pytest.mark.parametrize("K", [7, 16])
@pytest.mark.parametrize("dt,out_dt,st", [(BF16, BF16, BF16), (F16, F16, F16), (F32, F32, F32), (F32, BF16, F16), (F32, F32, BF16)])
def test_many_positions_of_all_types(K, dt, out_dt, st):
    R, H = 4, 3
    c = decode_case(R, K, H, 1, dt, "token", st, seed=34)
    ql, nc = i32([K, K - 2, 1, K]), i32([K, K // 2, 0, 1])
    zero = i32([0] * R)
    pool, out = c["pool"].clone(), torch.full((R * K, H, D), 7.0, dtype=out_dt, device="cuda")
    assert call_decode(c, pool, out, q_len=ql, n_commit=zero) == 0  # verify
    assert torch.equal(pool, c["pool"])
    assert call_decode({**c, "q": None}, pool, None, q_len=ql, n_commit=nc) == 0  # commit
    both, again = c["pool"].clone(), torch.zeros_like(out)
    assert call_decode(c, both, again, q_len=ql, n_commit=nc) == 0  # a step of both
    assert torch.equal(again, out) and torch.equal(both, pool)
    for r in range(R):
        o, s = want_decode(c, r, int(ql[r]))
        at = int(c["slot"][r])
        assert rel(out[r * K:r * K + len(o)].reshape(-1, D), (o * D ** -0.5).reshape(-1, D)) <= tol(out_dt)
        assert (out[r * K + len(o):(r + 1) * K] == 0).all()
        assert rel(pool[at], s[int(nc[r])]) <= tol(st) if int(nc[r]) else torch.equal(pool[at], c["pool"][at])
