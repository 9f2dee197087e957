"""Latent attention when a wait inside a kernel runs out: the call ends, says so, leaves nothing in
flight and the context usable.  The self-test entry stops one block's loads before a given one; every
other wait of that block then runs out by itself after about a second."""
import ctypes

import pytest
import torch

from helpers import i32
from test_gpu_latent import DL, DR, SCALE, Prefill, W

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
H = 16


def rows(t):
    return ctypes.byref(kda.RowsDesc(t.data_ptr(), t.stride(0), t.stride(1)))


class Batch:
    """Requests over one paged cache; run() with a stop (block, load) through the self-test."""

    def __init__(self, lens, page, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.R, self.page = len(lens), page
        used = [-(-n // page) for n in lens]
        self.cache = torch.randn(sum(used), page, W, generator=g, device="cuda").bfloat16()
        self.table = torch.zeros(self.R, max(used), dtype=torch.int32, device="cuda")
        at = 0
        for r, u in enumerate(used):
            self.table[r, :u] = torch.arange(at, at + u, device="cuda", dtype=torch.int32)
            at += u
        self.lens = i32(lens)
        self.ws = torch.zeros(kda.kda_latent_decode_workspace_size(self.R, 1, H), dtype=torch.uint8, device="cuda")

    def queries(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        q = torch.randn(self.R, H, W, generator=g, device="cuda").bfloat16()
        return q[..., :DL], q[..., DL:]

    def run(self, q, stop=None, fill=7.0, keep=None):
        out = torch.full((self.R, H, DL), fill, device="cuda")
        lse = torch.full((self.R, H), fill, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = [rows(q[0]), rows(q[1]), kda.KDA_BF16, self.R, 1, None, H, DL, DR, SCALE, self.cache.data_ptr(),
                self.cache.shape[0], self.page, self.page * W, self.table.data_ptr(), self.table.shape[1],
                self.lens.data_ptr(), rows(out), kda.KDA_F32, lse.data_ptr(), self.ws.data_ptr(), self.ws.nbytes,
                st.data_ptr(), torch.cuda.current_stream().cuda_stream]
        L = kda.lib()
        rc = L.kda_latent_decode(*args) if stop is None else L.kda_selftest_latent_decode_give_up(*args, *stop)
        assert rc == 0
        torch.cuda.synchronize()
        return out, lse, int(st)


# few requests over all blocks, and more requests than blocks; pages of one box a tile and of several
BATCHES = [([60000, 50000, 30000], 64), ([90000, 70000], 16), ([300 + 7 * r for r in range(200)], 32)]


@pytest.mark.parametrize("lens,page", BATCHES)
# before a block's first load, at a tile's start, between the loads of a tile, in the last of a ring's turns
@pytest.mark.parametrize("load", [0, 4, 9, 11, 13, 31])
def test_decode_gives_up_and_the_context_stays_usable(lens, page, load):
    b = Batch(lens, page, seed=page)
    q = b.queries(1)
    want = b.run(q)
    assert want[2] == 0
    out, lse, st = b.run(q, stop=(70, load))
    assert st == kda.KDA_DEV_TIMEOUT
    # the requests without a part in that block (it has two, seldom three) are as ever
    same = (out == want[0]).flatten(1).all(1) & (lse == want[1]).all(1)
    assert (~same).sum() <= 3
    again = b.run(q)
    assert again[2] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_decode_self_test_beyond_the_call_changes_nothing():
    b = Batch([3000, 70], 64, seed=5)
    q = b.queries(2)
    want = b.run(q)
    for stop in ((500, 0), (0, 1 << 20)):
        got = b.run(q, stop=stop)
        assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("lens,page", BATCHES)
@pytest.mark.parametrize("block", [0, 70, 71, 151])
@pytest.mark.parametrize("load", [0, 6, 31])
def test_decode_that_gave_up_joins_nothing_of_an_earlier_call(lens, page, block, load):
    b = Batch(lens, page, seed=page + 1)
    want = b.run(b.queries(2))
    earlier = b.run(b.queries(1))  # leaves its parts in the workspace
    out, lse, st = b.run(b.queries(2), stop=(block, load))
    assert st == kda.KDA_DEV_TIMEOUT
    same = (out == want[0]).flatten(1).all(1) & (lse == want[1]).all(1)
    assert not same.all()
    lost = out[~same]
    assert (torch.isnan(lost) | (lost == 7.0)).all()  # not joined at all, or joined to NaN
    z = lse[~same]
    assert (torch.isnan(z) | (z == 7.0) | (z == want[1][~same])).all()
    assert not torch.equal(earlier[0], want[0])


def run_prefill(p, q, stop=None, fill=7.0):
    Tq, n = q.shape[:2]
    out = torch.full((Tq, n, 128), fill, device="cuda")
    lse = torch.full((Tq, n), fill, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [rows(q), rows(p.kv[..., :128]), p.kr.data_ptr(), 64, rows(p.kv[..., 128:]), kda.KDA_BF16, p.cu_q.data_ptr(),
            p.cu_k.data_ptr(), len(p.lq), Tq, p.kv.shape[0], n, 128, 64, 128, SCALE, 0, rows(out), kda.KDA_F32,
            lse.data_ptr(), st.data_ptr(), torch.cuda.current_stream().cuda_stream]
    L = kda.lib()
    rc = L.kda_latent_prefill(*args) if stop is None else L.kda_selftest_latent_prefill_give_up(*args, *stop)
    assert rc == 0
    torch.cuda.synchronize()
    return out, lse, int(st)


# one block of rows a pair, and several one after another (32 heads); tile 27 of the first pair is the
# sequence's last, cut short; tile 30 lies in the pair's second block
@pytest.mark.parametrize("heads,block,tile", [
    (8, 0, 0), (8, 1, 0), (8, 0, 5), (8, 1, 6), (8, 70, 4), (8, 0, 27), (8, 1, 27), (8, 0, 26), (32, 0, 2), (32, 1, 30),
    (32, 0, 31), (32, 70, 3),
])
def test_prefill_gives_up_and_leaves_no_half_result(heads, block, tile):
    p = Prefill([3000, 700], [3500, 700], heads, seed=heads)
    want = run_prefill(p, p.q)
    assert want[2] == 0
    out, lse, st = run_prefill(p, p.q, stop=(block, tile))
    assert st == kda.KDA_DEV_TIMEOUT
    same = (out == want[0]).all(2) & (lse == want[1])
    assert not same.all() and same.any()
    lost, z = out[~same], lse[~same]
    assert (torch.isnan(lost) | (lost == 7.0)).all() and (torch.isnan(z) | (z == 7.0)).all()
    again = run_prefill(p, p.q)
    assert again[2] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    never = run_prefill(p, p.q, stop=(block, 1 << 20))
    assert never[2] == 0 and torch.equal(never[0], want[0])
