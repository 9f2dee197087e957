"""The norms around a block against their formulas in 64 bits.

Outputs are rounded once: eps / 2 of the value.  On top come fp32 sums of d squares (a tree: log2 d roundings, below
2e-6), the reciprocal root and the exponential (a few 2^-23): 4e-6 of the value, and the residual sum's cancellation,
counted against its summands."""
import pytest
import torch

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def half_step(dt):
    return torch.finfo(dt).eps / 2 if dt != F32 else 0.0


def close(got, want, dt, size=None):
    """|got - want| within the roundings; size: the summands' magnitude where it is not |want|."""
    size = want.abs() if size is None else size
    tiny = torch.finfo(dt).tiny * torch.finfo(dt).eps  # a subnormal's whole step
    bad = (got.double() - want).abs() > half_step(dt) * want.abs() * 1.001 + 4e-6 * size + tiny
    assert not bad.any() and not torch.isnan(got).any(), int(bad.sum())


def gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dt=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def act(z, kind):
    z = z.double()
    return z if kind == 0 else torch.sigmoid(z) * (z if kind == 2 else 1)


def norm(x, w, off):
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    return y if w is None else y * (w.double() + off)


DIMS = [1, 7, 8, 63, 64, 80, 128, 129, 256, 257, 1000, 1024, 1028, 2048, 4096, 4100, 8192, 16384, 16383]


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (F16, F32), (F32, F32), (F32, BF16)])
def test_gated(d, dt, out_dt):
    g = gen(d)
    for R, H, kind, first, off in ((1, 1, 1, False, 0.0), (5, 3, 2, False, 1.0), (3, 2, 1, True, 0.0), (2, 1, None, False, 0.0)):
        x, w = randn(g, R, H, d, dt=dt, std=0.5), randn(g, d, dt=dt)
        z = None if kind is None else randn(g, R, H, d, dt=dt, std=2.0)
        out = torch.full((R, H, d), 7.0, dtype=out_dt, device="cuda")
        kda.kda_gated_norm(x, out, gate=z, weight=w, weight_offset=off, act=kind if kind is not None else 1,
                           flags=kda.KDA_NORM_AFTER_GATE if first else 0)
        a = 1.0 if z is None else act(z, kind)
        close(out, norm(x.double() * a, w, off) if first else norm(x.double(), w, off) * a, out_dt,
              ((norm(x.double() * a, None, 0) if first else norm(x.double(), None, 0) * a) * (w.double().abs() + off)).abs())


@pytest.mark.parametrize("rows", [1023, 1024, 70000])
@pytest.mark.parametrize("d", [40, 128, 136, 1024])
def test_gated_many_rows(rows, d):
    if rows * d > 1 << 24:
        rows = 1500
    g = gen(rows + d)
    x, z = randn(g, rows, 1, d, dt=BF16), randn(g, rows, 1, d, dt=BF16)
    guard = torch.full((rows + 2, 1, d), 7.0, dtype=BF16, device="cuda")
    kda.kda_gated_norm(x, guard[1:-1], gate=z)
    close(guard[1:-1], norm(x.double(), None, 0) * act(z, 1), BF16)
    assert (guard[0] == 7.0).all() and (guard[-1] == 7.0).all()


@pytest.mark.parametrize("d", [128, 96, 50])
def test_gated_strided_in_place_and_without_weight(d):
    g = gen(1)
    wide = randn(g, 6, 4, 2, d + 3, dt=BF16)  # x and gate side by side in rows of an odd length
    x, z = wide[:, :, 0, :d], wide[:, :, 1, 1:d + 1]
    want = norm(x.double(), None, 0) * act(z, kda.KDA_ACT_NONE)
    out = torch.zeros(4, 6, d, dtype=F32, device="cuda").transpose(0, 1)
    kda.kda_gated_norm(x, out, gate=z, act=kda.KDA_ACT_NONE)
    close(out, want, F32)
    same = randn(g, 6, 4, d, dt=BF16)
    want = norm(same.double(), None, 0)
    kda.kda_gated_norm(same, same)
    close(same, want, BF16)


def test_gated_values_at_the_edges():
    """Rows of zeros, huge and tiny values, gates whose exponential overflows."""
    x = torch.zeros(6, 1, 128, device="cuda")
    x[1], x[2], x[3, 0, 5] = 1e18, 1e-20, 3.0
    x[4], x[5] = 1.0, 1.0
    z = torch.ones(6, 1, 128, device="cuda")
    z[4], z[5] = -200.0, 200.0
    for kind in (1, 2):
        out = torch.empty_like(x)
        kda.kda_gated_norm(x, out, gate=z, act=kind)
        close(out, norm(x.double(), None, 0) * act(z, kind), F32)


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("dt,rdt,out_dt", [(BF16, BF16, BF16), (BF16, F32, F16), (F16, F16, F16), (F32, F32, F32)])
def test_residual(d, dt, rdt, out_dt):
    g = gen(d)
    for R, post, gate, a, b, off, kind in ((1, True, None, 1.0, 1.0, 0.0, 0), (5, False, 1, 0.7, 0.25, 0.0, 0),
                                           (4, True, 4, 1.0, -0.5, 1.0, 1), (3, False, None, 1.0, 1.0, 0.0, 0)):
        x, r = randn(g, R, d, dt=dt, std=0.5), randn(g, R, d, dt=rdt, std=2.0)
        pw, w = (randn(g, d, dt=dt) if post else None), randn(g, d, dt=dt)
        z = None if gate is None else randn(g, gate, d, dt=dt)
        hidden, out = torch.full((R, d), 7.0, dtype=rdt, device="cuda"), torch.full((R, d), 7.0, dtype=out_dt, device="cuda")
        kda.kda_residual_norm(x, r, hidden=hidden, out=out, post_weight=pw, gate=z, act=kind, weight=w, residual_scale=a,
                              branch_scale=b, weight_offset=off)
        br = b * (norm(x.double(), pw, off) if post else x.double()) * (1.0 if z is None else act(z, kind))
        h = a * r.double() + br
        size = (a * r.double()).abs() + br.abs() + (abs(b) * x.double().abs() if post else 0)
        close(hidden, h, rdt, size)
        f = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
        # the sum's error against its summands, and that of all of them through the norm
        close(out, norm(h, w, off), out_dt, (size + h.abs()) * f * (w.double().abs() + off) * 2)


def test_residual_in_place_one_output_and_strides():
    g = gen(2)
    for d in (256, 100):
        wide = randn(g, 9, 3 * d + 1, dt=BF16)
        x, r = wide[:, :d], wide[:, d:2 * d]
        h = r.double() + x.double()
        only = torch.empty(9, d, dtype=BF16, device="cuda")
        kda.kda_residual_norm(x, r, out=only)  # the last norm: no residual goes on
        size = x.double().abs() + r.double().abs()
        close(only, norm(h, None, 0), BF16, 2 * size * (h.square().mean(-1, keepdim=True) + EPS).rsqrt())
        kda.kda_residual_norm(x, r, hidden=r)  # in place, without the next norm
        close(r, h, BF16, size)


@pytest.mark.parametrize("rows,d", [(1023, 512), (1024, 512), (3000, 4096), (2000, 1000), (5000, 64)])
def test_residual_many_rows(rows, d):
    g = gen(rows)
    x, r, w = randn(g, rows, d, dt=BF16), randn(g, rows, d, dt=BF16), randn(g, d, dt=BF16)
    guard = torch.full((rows + 2, d), 7.0, dtype=BF16, device="cuda")
    hidden = torch.empty(rows, d, dtype=BF16, device="cuda")
    kda.kda_residual_norm(x, r, hidden=hidden, out=guard[1:-1], post_weight=w, weight=w)
    br = norm(x.double(), w, 0)
    h = r.double() + br
    close(hidden, h, BF16, r.double().abs() + 2 * br.abs())
    f = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    close(guard[1:-1], norm(h, w, 0), BF16, 4 * (r.double().abs() + br.abs()) * f * w.double().abs())
    assert (guard[0] == 7.0).all() and (guard[-1] == 7.0).all()


def test_no_rows():
    e = torch.empty(0, 2, 128, dtype=BF16, device="cuda")
    kda.kda_gated_norm(e, e)
    kda.kda_residual_norm(e[:, 0], e[:, 0], out=e[:, 1])


def test_a_layer_of_decayed_attention():
    """residual norm -> projections -> decayed attention -> gated norm -> projection -> residual norm, a prompt of two
    sequences and then tokens one by one: the same hidden states as the longer prompt's, all bf16."""
    g, H, Dm, n, extra = gen(5), 4, 256, (70, 150), 3
    wq, wo = randn(g, Dm, 4 * H * 128, std=Dm ** -0.5, dt=BF16), randn(g, H * 128, Dm, std=(H * 128) ** -0.5, dt=BF16)
    wg, wn, wh = randn(g, Dm, H, std=Dm ** -0.5), 1 + randn(g, Dm, dt=BF16, std=0.1), 1 + randn(g, 128, dt=BF16, std=0.1)
    xs = [randn(g, L + extra, Dm, dt=BF16) for L in n]

    def layer(block, residual, attend):
        T = block.shape[0]
        hidden, y = torch.empty_like(residual), torch.empty_like(residual)
        kda.kda_residual_norm(block, residual, hidden=hidden, out=y, weight=wn, branch_scale=0.5)
        q, k, v, z = (y @ wq).view(T, 4, H, 128).unbind(1)
        o = torch.empty(T, H, 128, dtype=BF16, device="cuda")
        attend(q, k, v, -torch.nn.functional.softplus(y.float() @ wg), o)
        kda.kda_gated_norm(o, o, gate=z, weight=wh, act=kda.KDA_ACT_SILU)
        last = torch.empty_like(residual)
        kda.kda_residual_norm(o.view(T, -1) @ wo, hidden, hidden=hidden, out=last, post_weight=wn, weight=wn)
        return hidden, last

    def prefill(parts, pool, final):
        x = torch.cat(parts)
        L = [p.shape[0] for p in parts]
        cu = torch.tensor([0, L[0], L[0] + L[1]], dtype=torch.int32, device="cuda")
        ws = torch.empty(kda.kda_decay_prefill_workspace_size(len(x), 2, H), dtype=torch.uint8, device="cuda")
        return layer(x, x.flip(1).contiguous(), lambda q, k, v, d, o: kda.kda_decay_prefill(
            q, k, v, cu, o, log_decay=d, state_pool=pool, final_slot=final, scale=128 ** -1.0, workspace=ws))

    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    pool, other = torch.zeros(3, H, 128, 128, device="cuda"), torch.zeros(3, H, 128, 128, device="cuda")
    want = prefill(xs, other, slots)
    prefill([x[:L] for x, L in zip(xs, n)], pool, slots)
    for t in range(extra):
        x = torch.stack([x[L + t] for x, L in zip(xs, n)])
        got = layer(x, x.flip(1).contiguous(), lambda q, k, v, d, o: kda.kda_decay_decode(
            q, k, v, pool, slots, o, log_decay=d, scale=128 ** -1.0))
        at = [n[0] + t, n[0] + extra + n[1] + t]
        for a, b in zip(got, want):
            # some ten bf16 roundings a side, products of other row counts among them: sqrt(20) 2^-9 < 0.01
            assert (a.float() - b[at].float()).norm() <= 0.015 * b[at].float().norm(), t
    assert (pool[slots.long()] - other[slots.long()]).norm() <= 0.015 * other.norm()


@pytest.mark.parametrize("rows,d", [(1024, 1024), (1030, 1280), (1025, 2048), (1100, 2056), (1500, 4096), (16384, 4096),
                                    (300, 5120), (256, 8192), (1024, 8200), (1030, 16384)])
@pytest.mark.parametrize("dt,rdt,out_dt", [(BF16, BF16, BF16), (BF16, F32, BF16), (F16, F16, F32), (F32, F32, F32)])
def test_residual_many_long_rows(rows, d, dt, rdt, out_dt):
    """Rows through the ring in shared memory, with and without the norm after the block, gates a row, in place."""
    g = gen(rows + d)
    for post, gate, kind in ((True, None, 0), (False, 1, 0), (False, rows, 1), (True, rows, 2)):
        x, r = randn(g, rows, d, dt=dt, std=0.5), randn(g, rows, d, dt=rdt, std=2.0)
        pw, w = (randn(g, d, dt=dt) if post else None), randn(g, d, dt=dt)
        z = None if gate is None else randn(g, gate, d, dt=dt)
        br = -0.5 * (norm(x.double(), pw, 0) if post else x.double()) * (1.0 if z is None else act(z, kind))
        h = r.double() + br
        out = torch.empty(rows, d, dtype=out_dt, device="cuda")
        size = r.double().abs() + br.abs()
        kda.kda_residual_norm(x, r, hidden=r, out=out, post_weight=pw, gate=z, act=kind, weight=w, branch_scale=-0.5)
        close(r, h, rdt, size)
        f = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
        close(out, norm(h, w, 0), out_dt, (size + h.abs()) * f * w.double().abs() * 2)
    only = torch.empty_like(out)
    kda.kda_residual_norm(x, r, out=only)
    h = r.double() + x.double()
    f = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    close(only, h * f, out_dt, 2 * (r.double().abs() + x.double().abs()) * f)
