"""The scan's and the norms' entry points on the host: struct layouts, and refusals
of bad arguments before any CUDA call (no GPU needed: device pointers are made up
and never followed)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import ssm_decode_02_b200 as rsq

P = 1 << 20  # a well-aligned address that no call here may follow
INVAL, UNSUPPORTED = rsq.RSQ_E_INVAL, rsq.RSQ_E_UNSUPPORTED


def test_structs_match_the_c_header_layout(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = {n: getattr(rsq, n) for n in ("rsq_scan_config", "rsq_scan_inputs", "rsq_scan_grads", "rsq_norm_config")}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "rsq.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f[0], name, f[0]) for f in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-I", inc, str(src), "-o", str(exe)], check=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f in cls._fields_:
            assert int(got["%s.%s" % (name, f[0])]) == getattr(cls, f[0]).offset, (name, f[0])


def _status(call, *a, **k):
    with pytest.raises(rsq.RsqError) as e:
        call(*a, **k)
    assert rsq.lib.rsq_last_error().decode()
    return e.value.status


BASE = dict(sequences=2, tokens=256, heads=4, dk=64, dv=64)


@pytest.mark.parametrize("change,status", [
    (dict(family=rsq.RSQ_GDN), UNSUPPORTED), (dict(family=rsq.RSQ_GLA), UNSUPPORTED), (dict(family=rsq.RSQ_KDA), UNSUPPORTED),
    (dict(family=9), INVAL), (dict(in_dtype=rsq.RSQ_F32), UNSUPPORTED), (dict(in_dtype=5), INVAL),
    (dict(sequences=0), INVAL), (dict(sequences=65537, tokens=0), INVAL), (dict(heads=0), INVAL), (dict(heads=513), INVAL),
    (dict(dk=96), UNSUPPORTED), (dict(dv=8), UNSUPPORTED), (dict(dk=512), UNSUPPORTED), (dict(ngroups=3), INVAL),
    (dict(ngroups=0), INVAL), (dict(tokens=-1), INVAL), (dict(tokens=2 ** 31), INVAL), (dict(tokens=255), INVAL),
])
def test_scan_refuses_configs(change, status):
    assert _status(rsq.Scan, **(BASE | change)) == status


def _inputs(**kw):
    f = dict(x=P, Bm=P, Cm=P, dt=P, A=P, D=P, decay=None, x_stride=0, b_stride=0, c_stride=0)
    return rsq.rsq_scan_inputs(**(f | kw))


def test_scan_refuses_arguments():
    s, r = rsq.Scan(**BASE), rsq.Scan(**BASE, ragged=True)
    need, back = s.workspace_bytes, s.backward_workspace_bytes
    assert need > 0 and back > need

    def fwd(scan=s, cu=None, out=P, ws=P, n=need, state_in=None, state_out=None, **kw):
        return rsq.lib.rsq_scan(ctypes.byref(scan.cfg), ctypes.byref(_inputs(**kw)), cu, state_in, state_out, out, ws, n, None)

    bad = [dict(x=None), dict(Bm=None), dict(Cm=None), dict(dt=None), dict(A=None), dict(out=None), dict(x=P + 2), dict(Bm=P + 8),
           dict(dt=P + 2), dict(state_in=P + 4), dict(state_out=P + 8), dict(out=P + 2), dict(ws=None), dict(ws=P + 8),
           dict(n=need - 1), dict(x_stride=255), dict(x_stride=260), dict(b_stride=8), dict(c_stride=-64), dict(cu=P),
           dict(scan=r), dict(scan=r, cu=P + 2, n=1 << 40)]
    for kw in bad:
        assert fwd(**kw) == INVAL, kw
    assert rsq.lib.rsq_scan(None, None, None, None, None, None, None, 0, None) == INVAL
    assert rsq.lib.rsq_scan(ctypes.byref(s.cfg), None, None, None, None, P, P, need, None) == INVAL

    def bwd(dout=P, ws=P, n=back, grads=None, **kw):
        g = rsq.rsq_scan_grads(**(dict(dx=P) | (grads or {})))
        return rsq.lib.rsq_scan_backward(ctypes.byref(s.cfg), ctypes.byref(_inputs(**kw)), None, None, dout, None, ctypes.byref(g),
                                         ws, n, None)
    for kw in [dict(dout=None), dict(dout=P + 2), dict(ws=None), dict(n=back - 1), dict(grads=dict(dx=P + 2)),
               dict(grads=dict(ddt=P + 1)), dict(grads=dict(dstate_in=P + 4)), dict(decay=P, grads=dict(dA=P))]:
        assert bwd(**kw) == INVAL, kw
    assert rsq.lib.rsq_scan_backward(ctypes.byref(s.cfg), ctypes.byref(_inputs()), None, None, P, None, None, P, back, None) == INVAL
    assert rsq.lib.rsq_scan_workspace(ctypes.byref(s.cfg), 2, ctypes.byref(ctypes.c_size_t())) == INVAL
    assert rsq.lib.rsq_scan_workspace(ctypes.byref(s.cfg), 0, None) == INVAL
    assert rsq.lib.rsq_scan_check(None, None) == INVAL and rsq.lib.rsq_scan_check(P + 4, None) == INVAL


def test_single_tokens_need_no_workspace():
    assert rsq.Scan(7, 7, 4, 64, 64).workspace_bytes == 0


def _norm(**kw):
    f = dict(rows=4, width=64, group=32, order=0, x_dtype=1, side_dtype=1, y_dtype=1, eps=1e-5, x_stride=0, side_stride=0)
    return rsq.rsq_norm_config(**(f | kw))


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVAL), (dict(width=0), INVAL), (dict(width=16385), UNSUPPORTED), (dict(group=48), INVAL), (dict(group=-1), INVAL),
    (dict(order=2), INVAL), (dict(x_dtype=3), INVAL), (dict(side_dtype=-1), INVAL), (dict(y_dtype=2), INVAL), (dict(eps=0.0), INVAL),
    (dict(eps=float("nan")), INVAL), (dict(x_stride=63), INVAL), (dict(side_stride=-64), INVAL),
])
def test_norms_refuse_configs(change, status):
    cfg = _norm(**change)
    assert _status(rsq.rsq_norm_workspace, cfg) == status
    assert _status(rsq.rsq_gated_norm, cfg, P, P, P, P, stream=0) == status
    assert _status(rsq.rsq_gated_norm_backward, cfg, P, P, P, P, P, P, None, stream=0) == status
    cfg.group = 0 if "group" not in change else cfg.group
    assert _status(rsq.rsq_residual_norm, cfg, P, P, None, P, P, P, stream=0) == (INVAL if "group" in change else status)


def test_norms_refuse_arguments():
    cfg, one = _norm(), _norm(group=0)
    for a in [(None, P, P, P), (P, P, None, P), (P, P, P, None), (P + 2, P, P, P), (P, P + 8, P, P), (P, P, P + 4, P), (P, P, P, P + 2)]:
        assert _status(rsq.rsq_gated_norm, cfg, *a, stream=0) == INVAL, a
    for a in [(None, P, P, P, P, P, None), (P, None, P, P, P, P, None), (P, P, P, None, P, P, None), (P, P, P, P, P + 2, P, None),
              (P, P, P, P, P, P, P), (P, P, P, P, P, P, P + 4)]:   # a dw needs a workspace
        assert _status(rsq.rsq_gated_norm_backward, cfg, *a, stream=0) == INVAL, a
    ws = torch.empty(0, dtype=torch.uint8)
    with pytest.raises(ValueError):
        rsq.rsq_gated_norm_backward(cfg, P, P, P, P, P, P, P, ws, stream=0)   # a host workspace
    assert _status(rsq.rsq_residual_norm, cfg, P, P, None, P, P, P, stream=0) == INVAL   # groups
    for a in [(None, P, None, P, P, P), (P, P, P + 4, P, P, P), (P, P, None, None, P, P), (P, P, None, P, None, P), (P, P, None, P, P, None)]:
        assert _status(rsq.rsq_residual_norm, one, *a, stream=0) == INVAL, a
    assert _status(rsq.rsq_residual_norm, _norm(group=0, side_stride=72), P, P, None, P, P, P, stream=0) == INVAL  # h is packed
    assert _status(rsq.rsq_residual_norm_backward, one, None, P, P, P, P, P, P, P, P, P, stream=0) == INVAL  # dscale needs x


def test_binding_refuses_tensors():
    t = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        rsq.scan_inputs(t.view(4, 1, 64), None, None)            # on the host
    with pytest.raises(ValueError):
        rsq.scan_inputs(torch.zeros(4, 2, 128)[:, :, :64], None, None)   # a token's row has gaps
    with pytest.raises(ValueError):
        rsq.norm_config(t, t[:, :32], torch.bfloat16)
    with pytest.raises(ValueError):
        rsq.norm_config(t.half(), None, torch.bfloat16)
    with pytest.raises(ValueError):
        rsq.rsq_gated_norm(_norm(), t, None, t, t, stream=0)


class _On:
    """What the binding reads of a CUDA tensor; its address is never followed."""

    def __init__(self, *shape, dtype=torch.float32, device=0):
        self.t, self.device = torch.empty(shape, dtype=dtype, device="meta"), device
        self.is_cuda, self.shape, self.dtype = True, self.t.shape, dtype

    def __getattr__(self, name):
        return getattr(self.t, name)

    def data_ptr(self):
        return P

    def get_device(self):
        return self.device


def test_binding_refuses_sizes_and_types(monkeypatch):
    monkeypatch.setattr(rsq, "_current_device", lambda: 0)
    monkeypatch.setattr(rsq, "lib", None)                        # no call goes through
    bf = torch.bfloat16
    T, H, N, D = 256, 4, 64, 64
    scan = rsq.Scan.__new__(rsq.Scan)
    scan.cfg = rsq.rsq_scan_config(rsq.RSQ_MAMBA2, rsq.RSQ_BF16, 2, H, N, D, 1, 0, T)
    good = dict(x=_On(T, H, D, dtype=bf), Bm=_On(T, 1, N, dtype=bf), Cm=_On(T, 1, N, dtype=bf), dt=_On(T, H), A=_On(H), D=_On(H))
    out, state = _On(T, H, D, dtype=bf), _On(2, H, N, D)
    for name, t in [("x", _On(T, H, D)), ("Bm", _On(T, 1, N)), ("dt", _On(T, H, dtype=bf)), ("A", _On(H, dtype=bf))]:
        with pytest.raises(ValueError, match=name):
            rsq.scan_inputs(**(good | {name: t}))
    for name, t in [("x", _On(T - 1, H, D, dtype=bf)), ("Cm", _On(T, 2, N, dtype=bf)), ("dt", _On(T, 1)), ("D", _On(H - 1))]:
        with pytest.raises(ValueError, match=name):
            scan.forward(rsq.scan_inputs(**(good | {name: t})), out)
    ins = rsq.scan_inputs(**good)
    for kw in [dict(out=_On(T, H, D)), dict(state_in=_On(1, H, N, D)), dict(state_out=_On(2, H, N, D, dtype=bf)),
               dict(cu_seqlens=_On(2, dtype=torch.int32)), dict(cu_seqlens=_On(3, dtype=torch.int64))]:
        with pytest.raises(ValueError):
            scan.forward(ins, **(dict(out=out) | kw))
    for kw in [dict(dx=_On(T, H, D)), dict(dBm=_On(1, N, dtype=bf)), dict(ddt=_On(H)),
               dict(dA=_On(1)), dict(dstate_in=_On(1, H, N, D))]:
        with pytest.raises(ValueError):
            scan.backward(ins, out, rsq.scan_grads(**kw))
    with pytest.raises(ValueError, match="cuda:1"):
        scan.forward(rsq.scan_inputs(**(good | {"x": _On(T, H, D, dtype=bf, device=1)})), out)
    assert ins.tensors[0] is good["x"] and state.is_cuda

    x, z, w = _On(4, 64, dtype=bf), _On(4, 64, dtype=bf), _On(64)
    cfg = rsq.rsq_norm_config(4, 64, 0, 0, rsq.RSQ_BF16, rsq.RSQ_BF16, rsq.RSQ_BF16, 1e-5, 0, 0)
    for a in [(_On(4, 64), z, w, x), (x, _On(3, 64, dtype=bf), w, x), (x, z, _On(63), x), (x, z, w, _On(4, 64)),
              (x, z, w, _On(4, 64, dtype=bf, device=1))]:
        with pytest.raises(ValueError):
            rsq.rsq_gated_norm(cfg, *a)
    for a in [(x, z, None, w, z, _On(4, 64)), (x, z, _On(1), w, z, x), (x, z, None, w, _On(4, 64), x)]:
        with pytest.raises(ValueError):
            rsq.rsq_residual_norm(cfg, *a)
    with pytest.raises(ValueError):
        rsq.rsq_gated_norm_backward(cfg, x, z, w, x, _On(4, 64), z, None)
    with pytest.raises(ValueError):
        rsq.rsq_residual_norm_backward(cfg, x, z, None, w, x, z, x, _On(4, 63, dtype=bf), None, None)
