"""Decayed prefill: a (sequence, head) pair whose range lies over more SMs than a warp has lanes, so that a block joins
the states of its predecessors in several rounds, and its lanes read states whose flags other lanes waited for."""
import pytest
import torch

from test_gpu_decay import BF16, D, call_prefill, half_step, i32, log_decay, prefill_case, rel

pytestmark = pytest.mark.gpu


def last_state(c, S, L):
    """State after L rows of the call's one sequence, in 64 bits, 1000 rows at a time."""
    g = log_decay(c["head"], c["token"], c["T"], c["H"])[:L]
    rep = c["H"] // c["k"].shape[1]
    for a in range(0, L, 1000):
        G = g[a:a + 1000].cumsum(0)
        k = c["k"][a:min(a + 1000, L)].double().repeat_interleave(rep, 1) * (G[-1] - G).exp()[:, :, None]
        S = S * G[-1].exp()[:, None, None] + torch.einsum("thv,thk->hvk", c["v"][a:min(a + 1000, L)].double(), k)
    return S


@pytest.mark.parametrize("tokens,H", [(30000, 1), (100000, 1), (110000, 2)])  # 40, 131 and 2 x 76 ranges
def test_prefill_joins_more_states_than_a_warp_has_lanes(tokens, H):
    c = prefill_case([tokens], H, 1, BF16, "both", seed=11)
    # states that outlive the whole prompt nearly: every predecessor counts
    c["head"].fill_(-1e-6)
    c["token"].mul_(1e-4)
    init, final = i32([0]), i32([1])
    got = []
    for ws in (True, True, None):
        pool, out = c["pool"].clone(), torch.full((c["T"], H, D), 7.0, dtype=BF16, device="cuda")
        assert call_prefill(c, out, pool, init, final, ws=ws) == 0
        got.append((out, pool))
    (a, p), (b, q), (alone, r) = got
    assert torch.equal(a, b) and torch.equal(p, q)  # the same bits each time
    # without a workspace one block goes through the pair and joins nothing.  Outputs: 1.5 half steps each, as elsewhere;
    # states: up to 860 chunks, each a product and a sum that are 2^-24 off at most, random in sign: 2 sqrt(860) 2^-24
    # = 3.5e-6 on each side, and up to 131 ranges' decays and joins: 2 131 2^-24 / 2 = 7.8e-6.
    assert rel(a[:tokens].transpose(0, 1), alone[:tokens].transpose(0, 1)) <= 2 * 1.5 * half_step(BF16)
    assert rel(p[1], r[1]) <= 1.5e-5
    # (keys split in three parts, products summed in fp32: 5e-6; a range left out would be some 1e-2 of the state)
    assert rel(p[1], last_state(c, c["pool"][0].double(), tokens)) <= 2e-5
    assert (a[tokens:] == 7.0).all()
