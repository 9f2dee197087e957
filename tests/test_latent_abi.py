"""Host-side refusals of the latent attention and log-probability calls, without a GPU."""
import ctypes

import pytest

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: checks fail first
INVALID, UNSUPPORTED = 1, 2
BF16, F32, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__

    __graft_entry__.build()
    import serving_kda_chunk_gb300 as kda

    return kda


def rows(kda, base=FAKE, rs=512, hs=512):
    return ctypes.byref(kda.RowsDesc(base, rs, hs))


def test_recurrent_calls_refuse_fp16_activations(kda):
    st = kda.lib().kda_recurrent_decode(FAKE, FAKE, FAKE, FAKE, FAKE, F16, 4, 2, 128, 128, 1.0, 0, FAKE, 8,
                                        FAKE, FAKE, 0, None, None)
    assert st == UNSUPPORTED


def test_append_refusals(kda):
    def call(kv=FAKE, stride=576, weight=None, dt=BF16, T=4, dl=512, dr=64, slot=FAKE, cache=FAKE, P=8, page=16,
             ps=16 * 576):
        return kda.lib().kda_latent_append(kv, stride, weight, 1e-6, dt, T, dl, dr, slot, cache, P, page, ps,
                                           None, None)

    assert call(T=0, kv=None, slot=None, cache=None) == 0
    for bad in (dict(kv=None), dict(slot=None), dict(cache=None), dict(kv=FAKE + 2), dict(cache=FAKE + 8),
                dict(weight=FAKE + 4), dict(stride=570), dict(stride=580), dict(T=-1), dict(page=0),
                dict(ps=16 * 576 - 8), dict(ps=16 * 576 + 4), dict(P=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=F32), dict(dt=7), dict(dl=256), dict(dr=32), dict(page=12, ps=12 * 576)):
        assert call(**bad) == UNSUPPORTED, bad


def test_decode_refusals(kda):
    L = kda.lib()
    need = L.kda_latent_decode_workspace_size(4, 2, 8)
    ok = rows(kda)

    def call(ql=ok, qr=ok, dt=BF16, R=4, K=2, qlen=None, H=8, dl=512, dr=64, cache=FAKE, P=8, page=16, ps=16 * 576,
             table=FAKE, mp=4, sl=FAKE, out=ok, odt=BF16, lse=None, ws=FAKE, wb=need):
        return L.kda_latent_decode(ql, qr, dt, R, K, qlen, H, dl, dr, 1.0, cache, P, page, ps, table, mp, sl, out,
                                   odt, lse, ws, wb, None, None)

    assert call(R=0, ql=None, cache=None, table=None, sl=None, out=None, ws=None, wb=0) == 0
    assert call(K=0, ql=None, cache=None, table=None, sl=None, out=None, ws=None, wb=0) == 0
    for bad in (dict(ql=None), dict(qr=None), dict(out=None), dict(ql=rows(kda, None)), dict(ql=rows(kda, FAKE + 8)),
                dict(qr=rows(kda, rs=516)), dict(out=rows(kda, hs=4)), dict(cache=None), dict(table=None),
                dict(sl=None), dict(ws=None), dict(wb=need - 1), dict(ws=FAKE + 4), dict(table=FAKE + 4),
                dict(qlen=FAKE + 4), dict(lse=FAKE + 8), dict(R=-1), dict(K=-1), dict(H=0), dict(page=0),
                dict(mp=-1), dict(ps=576)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=F32), dict(dt=9), dict(odt=9), dict(K=17), dict(dl=576), dict(dr=0), dict(page=4, ps=4 * 576),
                dict(R=1 << 20, K=16, H=128), dict(mp=1 << 28)):
        assert call(**bad) == UNSUPPORTED, bad


def test_decode_workspace_size(kda):
    f = kda.kda_latent_decode_workspace_size
    assert f(0, 1, 16) >= 0
    for R, K, H in [(1, 1, 1), (256, 1, 32), (64, 7, 32), (4096, 16, 128)]:
        assert 0 < f(R, K, H) < 1 << 31 and f(R, K, H) % 16 == 0


def test_prefill_refusals(kda):
    ok = rows(kda)

    def call(q=ok, k=ok, kr=FAKE, krs=64, v=ok, dt=BF16, cq=FAKE, ck=FAKE, N=2, Tq=10, Tk=10, H=4, dn=128, dr=64,
             dv=128, flags=0, out=ok, odt=BF16, lse=None):
        return kda.lib().kda_latent_prefill(q, k, kr, krs, v, dt, cq, ck, N, Tq, Tk, H, dn, dr, dv, 1.0, flags, out,
                                            odt, lse, None, None)

    assert call(N=0, q=None, k=None, v=None, kr=None, cq=None, ck=None, out=None) == 0
    assert call(Tq=0, q=None, k=None, v=None, kr=None, cq=None, ck=None, out=None) == 0
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(kr=None), dict(cq=None),
                dict(ck=None), dict(q=rows(kda, FAKE + 2)), dict(k=rows(kda, rs=100)), dict(v=rows(kda, hs=9)),
                dict(krs=60), dict(krs=56), dict(kr=FAKE + 8), dict(lse=FAKE + 4), dict(N=-1), dict(Tq=-1),
                dict(Tk=-1), dict(H=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=F32), dict(odt=5), dict(dn=64), dict(dr=0), dict(dv=256), dict(flags=1), dict(flags=128)):
        assert call(**bad) == UNSUPPORTED, bad


def test_logprob_refusals(kda):
    def call(x=FAKE, rs=1000, dt=BF16, R=4, V=1000, tok=FAKE, lp=FAKE, ent=None, top=0, ids=None, tl=None):
        return kda.lib().kda_token_logprobs(x, rs, dt, R, V, tok, lp, ent, top, ids, tl, None, None)

    assert call(R=0, x=None, tok=None, lp=None) == 0
    for bad in (dict(x=None), dict(x=FAKE + 1), dict(rs=999), dict(tok=None), dict(lp=None), dict(tok=FAKE + 4),
                dict(top=2), dict(top=2, ids=FAKE), dict(top=2, ids=FAKE, tl=FAKE + 4), dict(V=0), dict(R=-1),
                dict(top=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=3), dict(top=33, ids=FAKE, tl=FAKE), dict(V=5, top=6, ids=FAKE, tl=FAKE)):
        assert call(**bad) == UNSUPPORTED, bad


def test_binding_refuses_shapes_and_types(kda):
    torch = pytest.importorskip("torch")
    z = torch.zeros
    h = torch.bfloat16
    cache, slot = z(2, 8, 576, dtype=h), z(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="one dtype"):
        kda.kda_latent_append(z(3, 576), cache, slot)
    with pytest.raises(ValueError, match="slot"):
        kda.kda_latent_append(z(3, 576, dtype=h), cache, slot[:2])
    q, qr, out, ws = z(4, 2, 512, dtype=h), z(4, 2, 64, dtype=h), z(4, 2, 512, dtype=h), z(16, dtype=torch.uint8)
    table, sl = z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="4 rows, not 2 requests x K = 1"):
        kda.kda_latent_decode(q, qr, cache, table, sl, out, ws, K=1)
    with pytest.raises(ValueError, match="q_rope"):
        kda.kda_latent_decode(q, qr[:3], cache, table, sl, out, ws, K=2)
    with pytest.raises(ValueError, match="one dtype"):
        kda.kda_latent_decode(q.half(), qr, cache, table, sl, out, ws, K=2)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_latent_decode(q, qr, cache, table, sl, out, ws, K=2)
    with pytest.raises(ValueError, match="contiguous pages"):
        kda.kda_latent_decode(q, qr, cache.transpose(0, 1), table, sl, out, ws, K=2)
    k, kr, cu = z(5, 2, 128, dtype=h), z(5, 64, dtype=h), z(2, dtype=torch.int32)
    o = z(4, 2, 128, dtype=h)
    with pytest.raises(ValueError, match="q must have shape"):
        kda.kda_latent_prefill(q, k, kr, k, cu, cu, o)
    with pytest.raises(ValueError, match="v must have shape"):
        kda.kda_latent_prefill(z(4, 2, 192, dtype=h), k, kr, k[:4], cu, cu, o)
    with pytest.raises(ValueError, match="together"):
        kda.kda_token_logprobs(z(2, 9), sl, z(2), top_ids=table)
    with pytest.raises(ValueError, match="contiguous rows"):
        kda.kda_token_logprobs(z(9, 2).T, sl, z(2))
