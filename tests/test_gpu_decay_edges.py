"""Decayed attention and the norms at the edges of what their calls allow: waits that run out, launches that the
runtime refuses, offsets past 32 bits, in-place slots of sequences that many SMs share, calls on other streams."""
import ctypes

import pytest
import torch

import serving_kda_chunk_gb300 as kda
from test_gpu_decay import (BF16, D, F32, call_prefill, check_prefill, decode_case, gen, half_step, i32, log_decay,
                            prefill_case, randn, recur, rel, tol, want_decode, want_prefill)

pytestmark = pytest.mark.gpu


def rows(t):
    return ctypes.byref(kda.RowsDesc(t.data_ptr(), t.stride(0), t.stride(1)))


def raw_prefill(c, out, pool, init, final, ws, stop=None):
    st = i32([0])
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    args = [rows(c["q"]), rows(c["k"]), rows(c["v"]), kda.KDA_BF16, p(c["head"]), p(c["token"]), p(c["cu"]), len(c["lens"]),
            c["T"], c["H"], c["k"].shape[1], D, D, D ** -0.5, 0, p(pool), pool.shape[0], p(init), p(final), None, 0, None,
            rows(out), kda.KDA_BF16, p(ws), 0 if ws is None else ws.nbytes, p(st), torch.cuda.current_stream().cuda_stream]
    L = kda.lib()
    rc = L.kda_decay_prefill(*args) if stop is None else L.kda_selftest_decay_prefill_give_up(*args, *stop)
    assert rc == 0
    torch.cuda.synchronize()
    return int(st)


# a first load, one in the middle of a pair that other blocks wait for, and one of a pair that nobody waits for
@pytest.mark.parametrize("cut,stop", [(True, (0, 0)), (True, (1, 3)), (True, (3, 9)), (False, (2, 1))])
def test_prefill_whose_loads_stop(cut, stop):
    c = prefill_case([5000, 200], 2, 2, BF16, "both", extra=0)
    init, final = i32([0, 1]), i32([2, 3])
    ws = torch.zeros(kda.kda_decay_prefill_workspace_size(c["T"], 2, 2), dtype=torch.uint8, device="cuda") if cut else None
    want = want_prefill(c, init)
    pool, out = c["pool"].clone(), torch.full((c["T"], 2, D), 7.0, dtype=BF16, device="cuda")
    assert raw_prefill(c, out, pool, init, final, ws, stop) == kda.KDA_DEV_TIMEOUT
    # what was written is right, the rest as it was
    a = 0
    for n, (o, s) in enumerate(want):
        for h in range(2):
            got = out[a:a + len(o), h]
            done = (got != 7.0).any(1)
            assert rel(got[done][None], o[done][:, h][None]) <= 1.5 * half_step(BF16) if done.any() else True
            state = pool[int(final[n]), h]
            assert torch.equal(state, c["pool"][int(final[n]), h]) or rel(state[None], s[-1][h][None]) <= 3.1e-5
        a += len(o)
    assert (out == 7.0).all(2).any()
    # the same workspace, right away
    pool, out = c["pool"].clone(), torch.zeros(c["T"], 2, D, dtype=BF16, device="cuda")
    assert raw_prefill(c, out, pool, init, final, ws) == 0
    check_prefill(c, out, pool, want, final, BF16)


def test_prefill_self_test_beyond_the_call():
    c = prefill_case([300], 2, 2, BF16, "head", extra=0)
    pool, out = c["pool"].clone(), torch.zeros(c["T"], 2, D, dtype=BF16, device="cuda")
    assert raw_prefill(c, out, pool, i32([0]), i32([1]), None, (9, 0)) == 0
    check_prefill(c, out, pool, want_prefill(c, i32([0])), i32([1]), BF16)


@pytest.mark.parametrize("shape", [([9000], 2), ([6000, 40, 3000], 3), ([2500], 16)], ids=str)
def test_prefill_in_place_over_many_blocks(shape):
    """Initial and final slot the same where a pair is gone through twice and its last block may be done first."""
    lens, H = shape
    c = prefill_case(lens, H, 1, BF16, "none", seed=4)
    slots = i32(list(range(len(lens))))
    want = want_prefill(c, slots)
    ref = None
    for _ in range(4):
        pool, out = c["pool"].clone(), torch.zeros(c["T"], H, D, dtype=BF16, device="cuda")
        assert call_prefill(c, out, pool, slots, slots) == 0
        check_prefill(c, out, pool, want, slots, BF16)
        assert ref is None or torch.equal(ref, pool)
        ref = pool


@pytest.mark.parametrize("n", [33, 600, 1500])
def test_prefill_of_many_sequences(n):
    """More sequences than a warp, and than a block, has threads; empty ones among them."""
    lens = [(7 * i * i + i) % 200 if i % 5 else 0 for i in range(n)]
    c = prefill_case(lens, 2, 1, BF16, "token", seed=5)
    want = want_prefill({**c, "lens": lens[:40]}, None)
    pool, out = c["pool"].clone(), torch.zeros(c["T"], 2, D, dtype=BF16, device="cuda")
    final = i32([n + i for i in range(n)])
    assert call_prefill(c, out, pool, None, final) == 0
    check_prefill({**c, "lens": lens[:40]}, out, pool, want, final, BF16)
    alone, other = torch.zeros_like(out), c["pool"].clone()
    assert call_prefill(c, alone, other, None, final, ws=None) == 0
    assert torch.equal(alone, out) and torch.equal(other, pool)


@pytest.mark.parametrize("seed", range(10))
def test_prefill_cut_anywhere(seed):
    """Pairs cut between blocks, wherever that falls, against one block a pair: states in place, empty and refused
    sequences among them.  Outputs are within 1.5 half steps each (as elsewhere); states add up to 40 chunks and the
    ranges' states in fp32, each addition 2^-24 off."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda n: int(torch.randint(0, n, (1,), generator=g))  # noqa: E731
    n, H = (1, 2, 3, 7, 33, 50)[pick(6)], (1, 2, 3, 5, 16)[pick(5)]
    most = min(5000, 120000 // (n * H))
    lens = [(0, 128, 129, pick(most) + 1, pick(most) + 1)[pick(5)] for _ in range(n)] + [1000]
    n += 1
    c = prefill_case(lens, H, H, BF16, "both", extra=0)
    pool = torch.randn(n, H, D, D, generator=gen(seed), device="cuda")
    slots = list(range(n))
    if seed % 2 and n > 2:
        slots[n // 2] = n + 5  # there is none
    slot = i32(slots)
    got = []
    for size in (kda.kda_decay_prefill_workspace_size(c["T"], n, H), 0):
        p, out = pool.clone(), torch.full((c["T"], H, D), 7.0, dtype=BF16, device="cuda")
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
        st = raw_prefill(c, out, p, slot, slot, ws)
        assert st == (kda.KDA_DEV_BAD_SLOT if max(slots) >= n else 0)
        got.append((out, p))
    (a, p), (b, q) = got
    at = 0
    for length, s in zip(lens, slots):
        if s >= n:
            assert (a[at:at + length] == 7.0).all()
        elif length:
            assert rel(a[at:at + length].transpose(0, 1), b[at:at + length].transpose(0, 1)) <= 2 * 1.5 * half_step(BF16)
        at += length
    assert rel(p, q) <= 1e-5


def test_offsets_past_32_bits():
    """Rows that lie 2^23 elements apart, a pool of more than 2^32 bytes."""
    g, n, step = gen(6), 300, 1 << 23
    wide = torch.empty(n * step, dtype=BF16, device="cuda")
    q, k, v, out = (torch.as_strided(wide, (n, 2, D), (step, 1024, 1), 256 * i) for i in range(4))
    for t in (q, k, v):
        t.copy_(randn(g, n, 2, D, dt=BF16, std=0.3))
    ld = -torch.rand(n, 2, generator=g, device="cuda")
    P = 70000
    pool = torch.empty(P, 2, D, D, dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    pool[P - 3:].zero_()
    kda.kda_decay_prefill(q, k, v, i32([0, n]), out, log_decay=ld, state_pool=pool, final_slot=i32([P - 1]))
    gd = log_decay(None, ld, n, 2)
    o, s = recur(torch.zeros(2, D, D, dtype=torch.float64, device="cuda"), q, k, v, gd)
    assert rel(out.transpose(0, 1), o.transpose(0, 1)) <= 1.5 * half_step(BF16)
    assert rel(pool[P - 1], s[-1]) <= half_step(BF16) + 3.1e-5
    for K in (1, 3):
        pool[P - 2].copy_(pool[P - 1])
        r = slice(n - K, n)
        want, last = recur(pool[P - 2].double(), q[r], k[r], v[r], gd[r])
        kda.kda_decay_decode(q[r], k[r], v[r], pool, i32([P - 2]), out[r], K=K, log_decay=ld[r].contiguous())
        assert rel(out[r].reshape(-1, D), want.reshape(-1, D)) <= tol(BF16)
        assert rel(pool[P - 2], last[-1]) <= tol(BF16)
    x = torch.as_strided(wide, (n, 1, 264), (step, 264, 1), 4096)
    x.copy_(randn(g, n, 1, 264, dt=BF16))
    y = torch.as_strided(wide, (n, 1, 264), (step, 264, 1), 8192)
    kda.kda_gated_norm(x, y)
    f = (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    assert rel(y.flatten(1), (x.double() * f).flatten(1)) <= half_step(BF16)
    kda.kda_residual_norm(x[:, 0], x[:, 0], out=y[:, 0])
    h = 2 * x.double()
    assert rel(y.flatten(1), (h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).flatten(1)) <= half_step(BF16)


def test_calls_on_a_stream_of_their_own():
    """Work on another stream than the current one, ordered by it alone."""
    c = prefill_case([400, 90], 2, 2, BF16, "token", seed=8)
    want = want_prefill(c, None)
    s = torch.cuda.Stream()
    pool, out = torch.zeros(4, 2, D, D, device="cuda"), torch.zeros(c["T"], 2, D, dtype=BF16, device="cuda")
    normed = torch.empty_like(out)
    s.wait_stream(torch.cuda.current_stream())
    kda.kda_decay_prefill(c["q"], c["k"], c["v"], c["cu"], out, log_decay=c["token"], state_pool=pool, final_slot=i32([0, 3]),
                          scale=D ** -0.5, stream=s)
    kda.kda_gated_norm(out, normed, stream=s)
    s.synchronize()
    check_prefill(c, out, pool, want, i32([0, 3]), BF16)
    f = (out.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    live = out[:490]
    assert rel(normed[:490].flatten(0, 1), (live.double() * f[:490]).flatten(0, 1)) <= half_step(BF16)


def test_decode_without_decay_of_a_state_with_infinities():
    """What is not finite stays where it is: other value channels, heads and requests do not see it."""
    for K in (1, 4):
        c = decode_case(3, K, 2, 2, BF16, "token")
        pool = c["pool"].clone()
        at = int(c["slot"][1])
        pool[at, 1, 5, 7] = float("inf")
        c["pool"] = pool.clone()
        out = torch.zeros(3 * K, 2, D, device="cuda")
        kda.kda_decay_decode(c["q"], c["k"], c["v"], pool, c["slot"], out, K=K, log_decay=c["token"], scale=D ** -0.5)
        bad = ~torch.isfinite(out)
        assert bad[K:2 * K, 1, 5].all() and int(bad.sum()) == K
        for r in (0, 2):
            o, s = want_decode(c, r, K)
            assert rel(out[r * K:(r + 1) * K].reshape(-1, D), (o * D ** -0.5).reshape(-1, D)) <= 1e-5
            assert rel(pool[int(c["slot"][r])], s[-1]) <= 1e-5


def test_prefill_values_that_are_not_finite():
    """They reach the rows behind them; chunks before theirs, and other sequences and heads, keep their results."""
    c = prefill_case([400, 300], 2, 2, BF16, "token", extra=0)
    a, b = (torch.zeros(700, 2, D, dtype=BF16, device="cuda") for _ in range(2))
    pa, pb = c["pool"].clone(), c["pool"].clone()
    call_prefill(c, a, pa, None, i32([0, 1]))
    c["v"][200, 1, 3] = float("nan")
    call_prefill(c, b, pb, None, i32([0, 1]))
    assert torch.equal(a[:128], b[:128]) and torch.equal(a[400:], b[400:]) and torch.equal(a[:, 0], b[:, 0])
    assert torch.isnan(b[200:400, 1, 3]).all() and torch.isnan(pb[0, 1, 3]).all()
    assert torch.equal(pa[1], pb[1]) and torch.equal(pa[0, 0], pb[0, 0])


@pytest.mark.parametrize("name", ["prefill", "cut", "step", "steps", "gated", "residual", "stream"])
def test_a_refused_launch_leaves_no_error(name):
    rt = ctypes.CDLL("libcudart.so.13")
    z = lambda *n, dt=BF16: torch.zeros(*n, dtype=dt, device="cuda")  # noqa: E731
    q, pool, hd, cu = z(1100, 2, D), z(6, 2, D, D, dt=F32), z(2, dt=F32), i32([0, 1100])
    ws = z(kda.kda_decay_prefill_workspace_size(1100, 1, 2), dt=torch.uint8)
    out, wide = torch.empty_like(q), z(1100, 1024)
    calls = {
        "prefill": lambda s: kda.kda_decay_prefill(q, q, q, cu, out, head_decay=hd, stream=s),
        "cut": lambda s: kda.kda_decay_prefill(q, q, q, cu, out, head_decay=hd, workspace=ws, stream=s),
        "step": lambda s: kda.kda_decay_decode(q[:3], q[:3], q[:3], pool, i32([0, 1, 2]), out[:3], head_decay=hd, stream=s),
        "steps": lambda s: kda.kda_decay_decode(q[:6], q[:6], q[:6], pool, i32([0, 1, 2]), out[:6], K=2, head_decay=hd, stream=s),
        "gated": lambda s: kda.kda_gated_norm(q, out, stream=s),
        "residual": lambda s: kda.kda_residual_norm(q[:, 0], q[:, 1], out=out[:, 0], stream=s),
        "stream": lambda s: kda.kda_residual_norm(wide, wide, out=torch.empty_like(wide), stream=s),
    }
    call, s = calls[name], torch.cuda.Stream()
    call(s)
    torch.cuda.synchronize()
    h = ctypes.c_void_p(s.cuda_stream)
    assert rt.cudaStreamBeginCapture(h, 2) == 0  # relaxed
    assert rt.cudaStreamSynchronize(h) != 0      # not allowed while capturing: the capture is invalid now
    rt.cudaGetLastError()
    try:
        with pytest.raises(kda.KdaError):
            call(s)
        left = rt.cudaGetLastError()
    finally:
        graph = ctypes.c_void_p()
        rt.cudaStreamEndCapture(h, ctypes.byref(graph))
        rt.cudaGetLastError()
    assert left == 0
    call(s)
    torch.cuda.synchronize()


def test_indexes_of_another_shape_are_refused():
    z = lambda *n, dt=BF16: torch.zeros(*n, dtype=dt, device="cuda")  # noqa: E731
    x, pool, hd = z(4, 2, D), z(3, 2, D, D, dt=F32), z(2, dt=F32)
    for slot in (z(4, 2, dt=torch.int32), z(4, 1, dt=torch.int32)):
        with pytest.raises(ValueError, match="slot must have shape"):
            kda.kda_decay_decode(x, x, x, pool, slot, torch.empty_like(x), head_decay=hd)
    with pytest.raises(ValueError, match="cu_seqlens must have shape"):
        kda.kda_decay_prefill(x, x, x, z(2, 2, dt=torch.int32), torch.empty_like(x), head_decay=hd)
