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
