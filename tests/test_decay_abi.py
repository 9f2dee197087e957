"""Host-side refusals of the decayed-attention and norm calls, without a GPU."""
import ctypes

import pytest

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: checks fail first
OK, INVALID, UNSUPPORTED = 0, 1, 2
BF16, F32, F16 = 0, 1, 2
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__

    __graft_entry__.build()
    import serving_kda_chunk_gb300 as kda

    return kda


def rows(kda, base=FAKE, rs=512, hs=128):
    return ctypes.byref(kda.RowsDesc(base, rs, hs))


def test_prefill_refusals(kda):
    L = kda.lib()
    ok = rows(kda)

    def call(q=ok, k=ok, v=ok, dt=BF16, hd=FAKE, ld=None, cu=FAKE, N=2, T=10, H=4, Hk=2, dk=128, dv=128, scale=1.0,
             flags=0, pool=FAKE, P=8, init=FAKE, final=FAKE, track=None, M=0, snap=None, out=ok, odt=BF16, ws=None, wb=0):
        return L.kda_decay_prefill(q, k, v, dt, hd, ld, cu, N, T, H, Hk, dk, dv, scale, flags, pool, P, init, final,
                                   track, M, snap, out, odt, ws, wb, None, None)

    assert call(N=0, q=None, k=None, v=None, out=None, cu=None, hd=None, pool=None, init=None, final=None) == OK
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(hd=None), dict(cu=None), dict(N=-1),
                dict(T=-1), dict(H=0), dict(Hk=0), dict(Hk=3), dict(P=-1), dict(M=-1), dict(M=1), dict(M=1, track=FAKE),
                dict(pool=None), dict(pool=FAKE + 8), dict(cu=FAKE + 4), dict(init=FAKE + 4), dict(final=FAKE + 2),
                dict(hd=FAKE + 2), dict(ld=FAKE + 1), dict(q=rows(kda, None)), dict(k=rows(kda, FAKE + 8)),
                dict(v=rows(kda, rs=516)), dict(out=rows(kda, hs=4)), dict(scale=NAN), dict(scale=INF),
                dict(ws=FAKE + 4, wb=1 << 30), dict(q=rows(kda, rs=-512)), dict(k=rows(kda, rs=0))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=F32), dict(dt=7), dict(odt=7), dict(dk=64), dict(dv=256), dict(flags=1), dict(flags=32),
                dict(flags=24), dict(T=1 << 30), dict(N=1 << 26, H=2)):
        assert call(**bad) == UNSUPPORTED, bad


def test_prefill_workspace_size(kda):
    f = kda.kda_decay_prefill_workspace_size
    for T, N, H in [(0, 0, 1), (1, 1, 1), (210, 3, 2), (131072, 1, 16), (41460, 8, 32), ((1 << 30) - 1, 4096, 128)]:
        assert 0 <= f(T, N, H) < 1 << 33 and f(T, N, H) % 16 == 0


def test_decode_refusals(kda):
    L = kda.lib()
    ok = rows(kda)

    def call(q=ok, k=ok, v=ok, dt=BF16, hd=FAKE, ld=None, R=4, K=2, ql=None, nc=None, H=4, Hk=2, dk=128, dv=128,
             scale=1.0, flags=0, pool=FAKE, P=8, slot=FAKE, dst=None, out=ok, odt=BF16):
        return L.kda_decay_decode(q, k, v, dt, hd, ld, R, K, ql, nc, H, Hk, dk, dv, scale, flags, pool, P, slot, dst,
                                  out, odt, None, None)

    none = dict(q=None, k=None, v=None, out=None, pool=None, slot=None, hd=None)
    assert call(R=0, **none) == OK and call(K=0, **none) == OK
    for bad in (dict(k=None), dict(v=None), dict(q=None), dict(hd=None), dict(pool=None), dict(slot=None), dict(R=-1),
                dict(K=-1), dict(H=0), dict(Hk=0), dict(Hk=3), dict(P=-1), dict(pool=FAKE + 8), dict(slot=FAKE + 4),
                dict(dst=FAKE + 4), dict(ql=FAKE + 4), dict(nc=FAKE + 8), dict(hd=FAKE + 1), dict(ld=FAKE + 2),
                dict(k=rows(kda, FAKE + 2)), dict(q=rows(kda, rs=100)), dict(out=rows(kda, hs=9)), dict(scale=-INF),
                dict(scale=NAN)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=17), dict(dt=5), dict(odt=-1), dict(dk=64), dict(dv=64), dict(flags=4), dict(flags=24),
                dict(R=1 << 28, H=4)):
        assert call(**bad) == UNSUPPORTED, bad


def test_gated_norm_refusals(kda):
    L = kda.lib()
    ok = rows(kda)

    def call(x=ok, gate=None, w=None, dt=BF16, R=4, H=2, d=100, eps=1e-6, off=0.0, act=1, flags=0, out=ok, odt=BF16):
        return L.kda_gated_norm(x, gate, w, dt, R, H, d, eps, off, act, flags, out, odt, None)

    assert call(R=0, x=None, out=None) == OK
    for bad in (dict(x=None), dict(out=None), dict(x=rows(kda, None)), dict(gate=rows(kda, None)), dict(R=-1), dict(H=0),
                dict(d=0), dict(eps=-1e-6), dict(eps=NAN), dict(off=INF), dict(x=rows(kda, FAKE + 1)),
                dict(gate=rows(kda, FAKE + 1)), dict(w=FAKE + 1), dict(out=rows(kda, FAKE + 2), odt=F32)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=3), dict(odt=9), dict(d=16385), dict(act=3), dict(act=-1), dict(flags=1)):
        assert call(**bad) == UNSUPPORTED, bad


def test_residual_norm_refusals(kda):
    L = kda.lib()

    def call(x=FAKE, r=FAKE, rdt=BF16, post=None, gate=None, act=0, w=None, dt=BF16, R=4, d=100, rsc=1.0, bsc=1.0,
             eps=1e-6, off=0.0, hidden=FAKE, out=FAKE, odt=BF16):
        return L.kda_residual_norm(x, d, r, d, rdt, post, gate, 0, act, w, dt, R, d, rsc, bsc, eps, off, hidden, d, out,
                                   d, odt, None)

    assert call(R=0, x=None, r=None, hidden=None, out=None) == OK
    for bad in (dict(x=None), dict(r=None), dict(hidden=None, out=None), dict(R=-1), dict(d=0), dict(eps=-1.0),
                dict(eps=INF), dict(rsc=NAN), dict(bsc=INF), dict(off=NAN), dict(x=FAKE + 1), dict(hidden=FAKE + 1),
                dict(r=FAKE + 2, rdt=F32), dict(post=FAKE + 1), dict(gate=FAKE + 1), dict(w=FAKE + 1),
                dict(out=FAKE + 2, odt=F32)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=3, rdt=3), dict(odt=3), dict(rdt=F16), dict(dt=F32, rdt=BF16), dict(d=16385), dict(act=4)):
        assert call(**bad) == UNSUPPORTED, bad


def test_binding_refuses_shapes_and_types(kda):
    torch = pytest.importorskip("torch")
    z, h, i = torch.zeros, torch.bfloat16, torch.int32
    q, v, cu, hd = z(6, 2, 128, dtype=h), z(6, 4, 128, dtype=h), z(2, dtype=i), z(4)
    pool, slot = z(3, 4, 128, 128), z(6, dtype=i)
    for kw, what in ((dict(q=q[:5]), "q must have"), (dict(out=q), "out must have"), (dict(head_decay=None), "is needed"),
                     (dict(head_decay=hd[:3]), "head_decay"), (dict(head_decay=hd.double()), "head_decay"),
                     (dict(head_decay=None, log_decay=z(6, 3)), "log_decay"), (dict(k=q.half()), "one dtype"), (dict(), "CUDA")):
        a = {**dict(q=q, k=q, v=v, cu_seqlens=cu, out=v, head_decay=hd), **kw}
        with pytest.raises(ValueError, match=what):
            kda.kda_decay_prefill(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("cu_seqlens"), a.pop("out"), **a)
        if "cu_seqlens" not in kw:
            a = {**dict(q=q, k=q, v=v, out=v, head_decay=hd), **kw}
            with pytest.raises(ValueError, match=what):
                kda.kda_decay_decode(a.pop("q"), a.pop("k"), a.pop("v"), pool, slot, a.pop("out"), **a)
    with pytest.raises(ValueError, match="needs q"):
        kda.kda_decay_decode(None, q, v, pool, slot, v, head_decay=hd)
    with pytest.raises(ValueError, match="shape of x"):
        kda.kda_gated_norm(v, q)
    with pytest.raises(ValueError, match="one dtype"):
        kda.kda_gated_norm(v, v, weight=z(128))
    x = z(3, 64, dtype=h)
    with pytest.raises(ValueError, match="hidden or out"):
        kda.kda_residual_norm(x, x)
    with pytest.raises(ValueError, match="residual's dtype"):
        kda.kda_residual_norm(x, x.float(), hidden=x)
    with pytest.raises(ValueError, match="gate must have"):
        kda.kda_residual_norm(x, x, out=x, gate=z(2, 64, dtype=h))


def test_prefill_self_test_refusals(kda):
    ok = rows(kda)

    def call(block=0, load=0, hd=FAKE):
        return kda.lib().kda_selftest_decay_prefill_give_up(ok, ok, ok, BF16, hd, None, FAKE, 2, 10, 4, 2, 128, 128, 1.0, 0,
                                                            FAKE, 8, FAKE, FAKE, None, 0, None, ok, BF16, None, 0, None,
                                                            None, block, load)

    assert call(block=-1) == INVALID and call(load=-1) == INVALID and call(hd=None) == INVALID
