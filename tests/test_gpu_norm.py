"""rsq_gated_norm and rsq_residual_norm on the GPU against their formulas in 64 bits.

Tolerances.  Every output is one rounding of a binary32 value whose factors
(a sum of `group` squares, the reciprocal root, two fast exponentials) are good
to (sqrt(group) + 16) 2^-24 relative.  du = r (dn - n mean(dn n)) is a difference of
two such terms, so its error is that share of r (|dn| + |n| mean(|dn n|)) -- not of
du, which is far below it where n nearly determines dn (a group of one: n = +-1 and
du is eps's share alone).  dw and dscale are binary32 sums over rows:
(sqrt(rows) + sqrt(group) + 16) 2^-24 of the root sum of squares of their terms.
"""
import pytest
import torch

import ssm_decode_02_b200 as rsq
from scan_reference import U16, U32, gated64, norm64, silu

pytestmark = pytest.mark.gpu
EPS = 1e-5


def rand(g, rows, width, dtype, std=1.0):
    return (torch.randn((rows, width), generator=g) * std).to(dtype)


def terms_of(u, dn, group):
    """r (|dn| + |n| mean(|dn n|)): the terms whose difference is the gradient of u."""
    u, dn = u.detach().unflatten(-1, (-1, group)), dn.detach().unflatten(-1, (-1, group))
    r = 1 / (u.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    n = u * r
    return (r * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True))).flatten(-2)


def slope_terms(z):
    """sigmoid (1 + |z| (1 - sigmoid)): the slope of the gate is the difference of these
    terms for z < 0 (it crosses zero near z = -1.28)."""
    sig = torch.sigmoid(z.detach())
    return sig * (1 + z.detach().abs() * (1 - sig))


def within(got, ref, terms, group):
    half = U16 if got.dtype == torch.bfloat16 else U32
    return torch.all((got.double().cpu() - ref).abs() <= half * ref.abs() + terms * (group ** 0.5 + 16) * U32 + 1e-37)


CASES = [  # rows, width, group, strided
    (1, 1, 1, False), (3, 16, 16, False), (5, 128, 16, True), (37, 2048, 128, False), (2, 188, 47, False), (7, 999, 333, True),
    (4, 2560, 2560, True), (600, 264, 264, False), (2, 5120, 5120, False), (3, 8200, 8200, False), (2, 16384, 16384, False),
    (2, 16383, 16383, False), (1300, 48, 8, False),
]


def strided(t, on):
    if not on:
        return t.cuda()
    wide = torch.full((t.shape[0], t.shape[1] + 24), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


@pytest.mark.parametrize("rows,width,group,apart", CASES)
@pytest.mark.parametrize("xd,zd", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                   (torch.bfloat16, torch.float32), (torch.float32, torch.float32)])
@pytest.mark.parametrize("order", [rsq.RSQ_NORM_GATE, rsq.RSQ_GATE_NORM, None])
def test_gated_norm(rows, width, group, apart, xd, zd, order):
    g = torch.Generator().manual_seed(rows * width)
    x, w = rand(g, rows, width, xd, 1.5), 1 + 0.2 * torch.randn(width, generator=g)
    z = None if order is None else rand(g, rows, width, zd)
    yd = torch.float32 if rows % 2 else torch.bfloat16
    dy = rand(g, rows, width, yd)
    leaves = [t.double().requires_grad_() for t in (x, z, w) if t is not None]
    xx, zz, ww = leaves if z is not None else (leaves[0], None, leaves[1])
    want = gated64(xx, zz, ww, group, EPS, order == rsq.RSQ_GATE_NORM)
    grads = torch.autograd.grad(want, leaves, dy.double())
    xc, zc, wc = strided(x, apart), None if z is None else strided(z, apart), w.cuda()
    cfg = rsq.norm_config(xc, zc, yd, group=group, order=order or 0, eps=EPS)
    y = torch.empty((rows, width), dtype=yd, device="cuda")
    rsq.rsq_gated_norm(cfg, xc, zc, wc, y)
    half = U16 if yd == torch.bfloat16 else U32
    tol = half * want.abs() + want.abs().max() * (group ** 0.5 + 16) * U32
    assert torch.all((y.double().cpu() - want).abs() <= tol)
    dx = torch.empty((rows, width), dtype=xd, device="cuda")
    dz = None if z is None else torch.empty((rows, width), dtype=zd, device="cuda")
    dw = torch.empty_like(wc)
    ws = torch.full((rsq.rsq_norm_workspace(cfg),), 255, dtype=torch.uint8, device="cuda")
    rsq.rsq_gated_norm_backward(cfg, xc, zc, wc, dy.cuda(), dx, dz, dw, ws)
    if order == rsq.RSQ_GATE_NORM:
        t = terms_of(xx * silu(zz), dy.double() * ww, group)
        tx, tz = t * silu(zz).detach().abs(), t * xx.detach().abs() * slope_terms(zz)
    else:
        tx = terms_of(xx, dy.double() * ww * (1 if z is None else silu(zz)), group)
        tz = None if z is None else (dy.double() * norm64(xx, ww, group, EPS)).detach().abs() * slope_terms(zz)
    assert within(dx, grads[0], tx, group)
    assert z is None or within(dz, grads[1], tz, group)
    n = norm64(xx * (zz / (1 + torch.exp(-zz))) if order == rsq.RSQ_GATE_NORM else xx, torch.ones_like(ww), group, EPS)
    terms = dy.double() * n * (zz / (1 + torch.exp(-zz)) if order == rsq.RSQ_NORM_GATE else 1)
    tol = terms.pow(2).sum(0).sqrt() * (rows ** 0.5 + group ** 0.5 + 16) * U32
    assert torch.all((dw.double().cpu() - grads[-1]).abs() <= tol)


@pytest.mark.parametrize("rows,width,group,apart", [c for c in CASES if c[1] == c[2]])
@pytest.mark.parametrize("xd,hd", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("scaled", [False, True])
def test_residual_norm(rows, width, group, apart, xd, hd, scaled):
    g = torch.Generator().manual_seed(rows + width)
    x, res, w = rand(g, rows, width, xd), rand(g, rows, width, hd, 2.0), 1 + 0.2 * torch.randn(width, generator=g)
    scale = 0.7 + 0.1 * torch.randn(width, generator=g) if scaled else None
    sc = 1.0 if scale is None else scale.double()
    xc, rc, wc = strided(x, apart), strided(res, apart), w.cuda()
    cfg = rsq.norm_config(xc, rc, torch.bfloat16, eps=EPS)
    h = torch.empty((rows, width), dtype=hd, device="cuda")
    y = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
    cs = None if scale is None else scale.cuda()
    rsq.rsq_residual_norm(cfg, xc, rc, cs, wc, h, y)
    want_h = res.double() + x.double() * sc
    half = U16 if hd == torch.bfloat16 else U32
    hc = h.double().cpu()
    assert torch.all((hc - want_h).abs() <= half * want_h.abs() * (1 + 2 * U16) + 4 * U32 * (res.double().abs() + x.double().abs()))
    want = norm64(hc, w.double(), width, EPS)   # of the stream as stored
    assert torch.all((y.double().cpu() - want).abs() <= U16 * want.abs() + want.abs().max() * (width ** 0.5 + 16) * U32)
    if not apart:   # in place, and without a residual
        r2 = rc.clone()
        y2 = torch.empty_like(y)
        rsq.rsq_residual_norm(cfg, xc, r2, cs, wc, r2, y2)
        assert torch.equal(r2, h) and torch.equal(y2, y)
        rsq.rsq_residual_norm(cfg, xc, None, cs, wc, r2, y2)
        assert torch.all((r2.double().cpu() - x.double() * sc).abs() <= (half + U32) * (x.double() * sc).abs())
    dy, dh = rand(g, rows, width, torch.bfloat16), rand(g, rows, width, hd)
    hl, wl = hc.clone().requires_grad_(), w.double().requires_grad_()
    gh, gw = torch.autograd.grad(norm64(hl, wl, width, EPS), [hl, wl], dy.double())
    dx, dres, dw = torch.empty_like(xc.contiguous()), torch.empty_like(h), torch.empty_like(wc)
    ds = None if scale is None else torch.empty_like(wc)
    ws = torch.full((rsq.rsq_norm_workspace(cfg),), 255, dtype=torch.uint8, device="cuda")
    rsq.rsq_residual_norm_backward(cfg, xc if scaled else None, h, cs, wc, dy.cuda(), dh.cuda(), dx, dres, ds, dw, ws)
    total = gh + dh.double()
    t = terms_of(hc, dy.double() * w.double(), width) + dh.double().abs()
    assert within(dres, total, t, width) and within(dx, total * sc, t * sc, width)
    n = norm64(hc, torch.ones(width, dtype=torch.float64), width, EPS)
    grow = (rows ** 0.5 + width ** 0.5 + 16) * U32
    assert torch.all((dw.double().cpu() - gw).abs() <= (dy.double() * n).pow(2).sum(0).sqrt() * grow)
    if scaled:
        terms = t * x.double()
        assert torch.all((ds.double().cpu() - (total * x.double()).sum(0)).abs() <= terms.pow(2).sum(0).sqrt() * grow)
    again = dh.cuda()                       # dresidual in the place of dh
    rsq.rsq_residual_norm_backward(cfg, xc, h, cs, wc, dy.cuda(), again, None, again, None, None)
    assert torch.equal(again, dres)


def test_no_rows_and_extreme_gates():
    w = torch.ones(64, device="cuda")
    x = torch.empty((0, 64), device="cuda")
    cfg = rsq.norm_config(x, None, torch.float32)
    rsq.rsq_gated_norm(cfg, x, None, w, torch.empty_like(x))
    dw = torch.full_like(w, 5.0)
    rsq.rsq_gated_norm_backward(cfg, x, None, w, x, None, None, dw, torch.empty(rsq.rsq_norm_workspace(cfg), dtype=torch.uint8, device="cuda"))
    assert (dw == 0).all()
    x = torch.ones((2, 64), device="cuda")
    z = torch.full_like(x, -200.0)          # e^200 overflows: the gate is 0
    z[1] = 200.0
    cfg = rsq.norm_config(x, z, torch.float32)
    y = torch.empty_like(x)
    rsq.rsq_gated_norm(cfg, x, z, w, y)
    assert (y[0] == 0).all() and (y[1] - 200.0).abs().max() < 0.01
    dx, dz = torch.empty_like(x), torch.empty_like(x)
    rsq.rsq_gated_norm_backward(cfg, x, z, w, torch.ones_like(x), dx, dz, None)
    assert torch.isfinite(dx).all() and (dz[0].abs() < 1e-30).all()


def test_rows_are_independent_of_a_nan_and_graph_replay():
    g = torch.Generator().manual_seed(3)
    x, z, w = rand(g, 70, 128, torch.bfloat16).cuda(), rand(g, 70, 128, torch.bfloat16).cuda(), torch.ones(128).cuda()
    cfg = rsq.norm_config(x, z, torch.bfloat16, group=32, order=rsq.RSQ_GATE_NORM)
    y, ws = torch.empty_like(x), torch.empty(rsq.rsq_norm_workspace(cfg), dtype=torch.uint8, device="cuda")
    dx, dz, dw, dy = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), rand(g, 70, 128, torch.bfloat16).cuda()

    def both():
        rsq.rsq_gated_norm(cfg, x, z, w, y)
        rsq.rsq_gated_norm_backward(cfg, x, z, w, dy, dx, dz, dw, ws)
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    x.copy_(rand(g, 70, 128, torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    a = [t.clone() for t in (y, dx, dz, dw)]
    both()
    for s, t in zip(a, (y, dx, dz, dw)):
        assert torch.equal(s, t)
    x[7, 40] = float("nan")
    rsq.rsq_gated_norm(cfg, x, z, w, y)
    bad = torch.isnan(y.float())
    assert bad[7, 32:64].all() and bad.sum() == 32
    assert torch.equal(y[~bad], a[0][~bad])
