"""The norms on arrays that start anywhere: rows that are no whole vectors are worked on element
by element, and every array may be a piece of a longer one."""
import pytest
import torch

import ssm_decode_02_b200 as rsq

pytestmark = pytest.mark.gpu


def piece(t, off):
    """The values of t, off elements behind an aligned address; NaN around them."""
    if t is None:
        return None
    long = torch.full((t.numel() + 2 * off + 3,), float("nan"), dtype=t.dtype, device="cuda")
    p = long[off:off + t.numel()].view(t.shape)
    p.copy_(t)
    return p


@pytest.mark.parametrize("rows,width,group", [(7, 333, 111), (3, 99, 99), (130, 47, 47), (2, 8201, 8201)])
@pytest.mark.parametrize("off", [1, 3])
@pytest.mark.parametrize("xd,sd", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_unaligned_arrays(rows, width, group, off, xd, sd):
    """The same as on aligned ones, bit for bit."""
    g = torch.Generator().manual_seed(rows + width)
    r = lambda d: torch.randn((rows, width), generator=g).to(d).cuda()  # noqa: E731
    x, z, dy, res, dh = r(xd), r(sd), r(torch.bfloat16), r(sd), r(sd)
    w, scale = torch.randn(width, generator=g).cuda(), torch.randn(width, generator=g).cuda()

    def all_of(put):
        a = [put(t) for t in (x, z, dy, res, dh, w, scale)]
        X, Z, DY, R, DH, W, S = a
        new = lambda t: put(torch.full_like(t, 5.0))  # noqa: E731
        cfg = rsq.norm_config(X, Z, torch.bfloat16, group=group, order=rsq.RSQ_GATE_NORM)
        ws = torch.empty(rsq.rsq_norm_workspace(cfg), dtype=torch.uint8, device="cuda")
        y, dx, dz, dw = new(dy), new(x), new(z), new(w)
        rsq.rsq_gated_norm(cfg, X, Z, W, y)
        rsq.rsq_gated_norm_backward(cfg, X, Z, W, DY, dx, dz, dw, ws)
        out = [y, dx, dz, dw]
        if group == width:
            h, y2, dx2, dr, ds, dw2 = new(res), new(dy), new(x), new(res), new(w), new(w)
            rsq.rsq_residual_norm(cfg, X, R, S, W, h, y2)
            rsq.rsq_residual_norm_backward(cfg, X, h, S, W, DY, DH, dx2, dr, ds, dw2, ws)
            out += [h, y2, dx2, dr, ds, dw2]
        return out

    for a, b in zip(all_of(lambda t: t.clone()), all_of(lambda t: piece(t, off))):
        assert b.data_ptr() % 16 and torch.isfinite(a.float()).all() and torch.equal(a, b)
