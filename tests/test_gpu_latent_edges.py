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
