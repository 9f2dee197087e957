"""Decayed prefill with a workspace: how many blocks a call has."""
import pytest
import torch

import serving_kda_chunk_gb300 as kda
from test_gpu_decay import BF16, D, call_prefill, check_prefill, half_step, i32, prefill_case, rel, want_prefill
from test_gpu_decay_edges import raw_prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H", [([70] * 16, 4), ([100] * 16, 8), ([20] * 40, 2), ([300, 0, 7] * 4, 3)], ids=str)
def test_many_short_prompts_have_a_block_a_pair(lens, H):
    """Pairs that are not worth cutting go one to a block as long as there are SMs: the last pair's block is the one of that
    number.  (Loads that are stopped in a block that a call has not change nothing: the self-test's contract.)"""
    c = prefill_case(lens, H, 1, BF16, "token", extra=2, seed=12)
    N = len(lens)
    init, final = i32(list(range(N))), i32([N + n for n in range(N)])
    ws = torch.zeros(kda.kda_decay_prefill_workspace_size(c["T"], N, H), dtype=torch.uint8, device="cuda")
    want, last = want_prefill(c, init), N * H - 1
    for block, status in ((last, kda.KDA_DEV_TIMEOUT), (last + 1, 0)):
        pool, out = c["pool"].clone(), torch.full((c["T"], H, D), 7.0, dtype=BF16, device="cuda")
        assert raw_prefill(c, out, pool, init, final, ws, (block, 0)) == status
        if status == 0:
            check_prefill(c, out, pool, want, final, BF16)
            continue
        a, missing = 0, 0
        for n, (o, s) in enumerate(want):
            for h in range(H):
                got = out[a:a + len(o), h]
                if n == N - 1 and h == H - 1:
                    assert (got == 7.0).all() and torch.equal(pool[N + n, h], c["pool"][N + n, h])
                    missing += 1
                elif len(o):
                    assert rel(got[None], o[:, h][None]) <= 1.5 * half_step(BF16)
            a += len(o)
        assert missing == 1


@pytest.mark.parametrize("lens,H", [([1400] + [70] * 15, 4), ([70] * 15 + [1400], 4), ([500, 30] * 8, 5), ([900, 1, 1, 1], 30)],
                         ids=str)
def test_short_prompts_beside_a_longer_one(lens, H):
    """Ranges of a few chunks, some of which cut the longer pairs, answer as one block a pair does."""
    c = prefill_case(lens, H, 1, BF16, "both", seed=13)
    N = len(lens)
    slots = i32(list(range(N)))
    want = want_prefill(c, slots)
    for ws in (True, None):
        pool, out = c["pool"].clone(), torch.full((c["T"], H, D), 7.0, dtype=BF16, device="cuda")
        assert call_prefill(c, out, pool, slots, slots, ws=ws) == 0
        check_prefill(c, out, pool, want, slots, BF16)
        assert (out[sum(lens):] == 7.0).all()
