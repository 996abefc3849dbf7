"""What the Python binding of the scan and the norms refuses before a kernel sees it
(no GPU: tensors are stand-ins whose address is never followed, and no call goes
through)."""
import pytest
import torch

import ssm_decode_02_b200 as rsq

P = 1 << 20
BF = torch.bfloat16
T, H, N, D, G = 256, 4, 64, 64, 1


class Fake:
    """A CUDA tensor of given shape and strides without memory."""

    def __init__(self, t, device=0):
        self.t, self.at, self.is_cuda = t, device, True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, i):
        return Fake(self.t[i], self.at)

    def view(self, *shape):
        return Fake(self.t.view(*shape), self.at)

    def expand(self, *shape):
        return Fake(self.t.expand(*shape), self.at)

    def data_ptr(self):
        return P

    def get_device(self):
        return self.at


def on(*shape, dtype=torch.float32, device=0):
    return Fake(torch.empty(shape, dtype=dtype, device="meta"), device)


class Calls:
    """In the place of the library: records the names of the functions called, all of which succeed."""

    def __init__(self):
        self.names = []

    def __getattr__(self, name):
        def call(*a):
            self.names.append(name)
            return rsq.RSQ_OK
        return call


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(rsq, "_current_device", lambda: 0)
    monkeypatch.setattr(rsq, "_stream", lambda s: 0)
    monkeypatch.setattr(rsq, "lib", c)
    return c


def scan_of(**kw):
    s = rsq.Scan.__new__(rsq.Scan)
    s.cfg = rsq.rsq_scan_config(**(dict(family=rsq.RSQ_MAMBA2, in_dtype=rsq.RSQ_BF16, sequences=2, heads=H, dk=N, dv=D, ngroups=G,
                                        ragged=0, tokens=T) | kw))
    return s


def tokens(**kw):
    return dict(x=on(T, H, D, dtype=BF), Bm=on(T, G, N, dtype=BF), Cm=on(T, G, N, dtype=BF), dt=on(T, H), A=on(H), D=on(H)) | kw


def slices(*widths, rows=T):
    """Column ranges of one wide array."""
    wide = on(rows, sum(widths) + 8, dtype=BF)
    at = [sum(widths[:i]) for i in range(len(widths))]
    return [wide[:, a:a + w] for a, w in zip(at, widths)]


# ------------------------------------------------------------------------------- rows of a tensor
@pytest.mark.parametrize("name,t", [("x", on(1, H, D, dtype=BF).expand(T, H, D)), ("Bm", on(1, G, N, dtype=BF).expand(T, G, N)),
                                    ("Cm", on(1, G, N, dtype=BF).expand(T, G, N)),
                                    ("Cm", Fake(torch.empty(T * N, dtype=BF, device="meta").as_strided((T, G, N), (8, N, 1))))])
def test_scan_refuses_rows_that_share_memory(calls, name, t):
    """A broadcast tensor has one row stored; a stride of 0 means packed rows to the kernels."""
    with pytest.raises(ValueError, match=name):
        rsq.scan_inputs(**tokens(**{name: t}))


def test_scan_takes_rows_that_lie_apart(calls):
    x, Bm, Cm = slices(H * D, N, N)
    ins = rsq.scan_inputs(**tokens(x=x.view(T, H, D), Bm=Bm.view(T, 1, N), Cm=Cm.view(T, 1, N)))
    assert ins.x_stride == ins.b_stride == ins.c_stride == H * D + 2 * N + 8
    scan_of().forward(ins, on(T, H, D, dtype=BF))
    one = tokens(x=on(1, H, D, dtype=BF).expand(1, H, D), Bm=on(1, G, N, dtype=BF), Cm=on(1, G, N, dtype=BF), dt=on(1, H))
    scan_of(sequences=1, tokens=1).forward(rsq.scan_inputs(**one), on(1, H, D, dtype=BF))
    assert calls.names == ["rsq_scan", "rsq_scan"]


def test_norm_config_refuses_rows_that_share_memory(calls):
    x = on(T, N, dtype=BF)
    for a, b in [(on(1, N, dtype=BF).expand(T, N), x), (x, on(1, N, dtype=BF).expand(T, N)), (on(N, dtype=BF).expand(T, N), None),
                 (x, Fake(torch.empty(4 * T + N, dtype=BF, device="meta").as_strided((T, N), (4, 1))))]:
        with pytest.raises(ValueError, match="row"):
            rsq.norm_config(a, b, BF)
    assert rsq.norm_config(on(N, dtype=BF).expand(1, N), None, BF).x_stride == 0


def norm_cfg(rows=T, width=N, x_stride=0, side_stride=0, x=rsq.RSQ_BF16, side=rsq.RSQ_BF16, y=rsq.RSQ_BF16):
    return rsq.rsq_norm_config(rows, width, 0, 0, x, side, y, 1e-5, x_stride, side_stride)


def norm_calls(cfg, x, side):
    """Every norm call that reads x and side (z, or the residual) by the configuration's strides."""
    w, y = on(N), on(T, N, dtype=BF)
    h = y if side is None else on(T, N, dtype=side.dtype)
    return [lambda: rsq.rsq_gated_norm(cfg, x, side, w, y), lambda: rsq.rsq_gated_norm_backward(cfg, x, side, w, y, None, None, None),
            lambda: rsq.rsq_residual_norm(cfg, x, side, None, w, h, y)]


def test_norms_refuse_rows_that_lie_other_than_configured(calls):
    """A configuration is made once and used with other tensors: a packed tensor read at a slice's
    stride is left behind its end."""
    packed, (a, b) = on(T, N, dtype=BF), slices(N, N)
    apart = int(a.stride(0))
    wrong = [(norm_cfg(x_stride=apart), packed, packed), (norm_cfg(side_stride=apart), packed, packed), (norm_cfg(), a, packed),
             (norm_cfg(), packed, b), (norm_cfg(x_stride=apart, side_stride=apart), a, packed),
             (norm_cfg(x_stride=apart), on(T - 1, apart, dtype=BF)[:, :N], packed),
             (norm_cfg(x_stride=apart), on(T, apart, dtype=BF)[:, :N - 8], None),
             (norm_cfg(), on(1, N, dtype=BF).expand(T, N), packed), (norm_cfg(), packed, on(1, N, dtype=BF).expand(T, N)),
             (norm_cfg(x_stride=apart), on(T, 2, apart // 2, dtype=BF)[:, :, :N // 2], None),
             (norm_cfg(rows=1), on(1, 2, apart // 2, dtype=BF)[:, :, :N // 2], None)]
    for cfg, x, side in wrong:
        for call in norm_calls(cfg, x, side):
            with pytest.raises(ValueError):
                call()
    cfg = norm_cfg(x_stride=apart, side=rsq.RSQ_F32)
    with pytest.raises(ValueError):
        rsq.rsq_residual_norm_backward(cfg, packed, on(T, N), None, on(N), packed, None, None, None, None, None)
    assert not calls.names


def test_norms_take_rows_as_configured(calls):
    packed, (a, b) = on(T, N, dtype=BF), slices(N, N)
    apart = int(a.stride(0))
    right = [(norm_cfg(), packed, packed), (norm_cfg(x_stride=N, side_stride=N), packed, packed), (norm_cfg(x_stride=apart), a, packed),
             (norm_cfg(x_stride=apart, side_stride=apart), a, b), (norm_cfg(), packed.view(T * N), packed.view(T // 2, 2 * N)),
             (norm_cfg(rows=1), a[:1], b[:1]), (norm_cfg(x_stride=apart), a.view(T, 2, N // 2), None), (norm_cfg(rows=T - 3), packed, packed),
             (norm_cfg(rows=1, x_stride=apart), packed.view(T * N), packed), (norm_cfg(rows=0, x_stride=apart), a[:0], None)]
    for cfg, x, side in right:
        for call in norm_calls(cfg, x, side):
            call()
    # the backward pass has h as the forward pass wrote it, whatever the residual's stride was
    rsq.rsq_residual_norm_backward(norm_cfg(side_stride=apart), packed, packed, None, on(N), packed, None, None, None, None, None)
    assert len(calls.names) == 3 * len(right) + 1


# ------------------------------------------------------------------------------------------ types
HALF, INT = torch.float16, torch.int32


def test_scan_refuses_types_of_the_same_size(calls):
    """float16 bits are no bfloat16, int32 bits no float32."""
    for name, t in [("x", on(T, H, D, dtype=HALF)), ("Bm", on(T, G, N, dtype=HALF)), ("Cm", on(T, G, N, dtype=torch.int16)),
                    ("dt", on(T, H, dtype=INT)), ("A", on(H, dtype=INT)), ("D", on(H, dtype=INT)), ("decay", on(T, H, dtype=INT))]:
        with pytest.raises(ValueError, match=name):
            rsq.scan_inputs(**tokens(**{name: t}))
    ins, out, state, s = rsq.scan_inputs(**tokens()), on(T, H, D, dtype=BF), on(2, H, N, D), scan_of()
    for kw in [dict(out=on(T, H, D, dtype=HALF)), dict(state_in=on(2, H, N, D, dtype=INT)), dict(state_out=on(2, H, N, D, dtype=INT)),
               dict(cu_seqlens=on(3)), dict(cu_seqlens=on(3, dtype=torch.uint32))]:
        with pytest.raises(ValueError):
            s.forward(ins, **(dict(out=out) | kw))
    rows = dict(dx=(T, H, D), dBm=(T, G, N), dCm=(T, G, N))
    single = dict(ddt=(T, H), dlog_decay=(T, H), dA=(H,), dD=(H,), dstate_in=(2, H, N, D))
    for name, shape in (rows | single).items():
        with pytest.raises(ValueError):
            s.backward(ins, out, rsq.scan_grads(**{name: on(*shape, dtype=HALF if name in rows else INT)}))
    with pytest.raises(ValueError):
        s.backward(ins, on(T, H, D, dtype=HALF), rsq.scan_grads())
    with pytest.raises(ValueError):
        s.backward(ins, out, rsq.scan_grads(), dstate_out=on(2, H, N, D, dtype=INT))
    assert not calls.names
    s.forward(ins, out, state_in=state, state_out=state)
    s.backward(ins, out, rsq.scan_grads(**{k: on(*v, dtype=BF) for k, v in rows.items()}, **{k: on(*v) for k, v in single.items()}),
               state_in=state, dstate_out=state)
    scan_of(ragged=1).forward(ins, out, cu_seqlens=on(3, dtype=INT))
    assert calls.names == ["rsq_scan", "rsq_scan_backward", "rsq_scan"]


def test_norms_refuse_types_of_the_same_size(calls):
    cfg, x, w, half = norm_cfg(), on(T, N, dtype=BF), on(N), on(T, N, dtype=HALF)
    wide = norm_cfg(x=rsq.RSQ_F32, side=rsq.RSQ_F32, y=rsq.RSQ_F32)
    f, i, wi = on(T, N), on(T, N, dtype=INT), on(N, dtype=INT)
    for c, good, bad in ((cfg, x, half), (wide, f, i)):
        for a in [(bad, good, w, good), (good, bad, w, good), (good, good, w, bad), (good, good, wi, good), (good, None, w, bad)]:
            with pytest.raises(ValueError):
                rsq.rsq_gated_norm(c, *a)
        for k in range(7):
            a = [good, good, w, good, good, good, w]          # x, z, w, dy, dx, dz, dw
            a[k] = wi if k in (2, 6) else bad
            with pytest.raises(ValueError):
                rsq.rsq_gated_norm_backward(c, *a)
        for k in range(6):
            a = [good, good, w, w, good, good]                # x, residual, scale, w, h, y
            a[k] = wi if k in (2, 3) else bad
            with pytest.raises(ValueError):
                rsq.rsq_residual_norm(c, *a)
        for k in range(10):
            a = [good, good, w, w, good, good, good, good, w, w]   # x, h, scale, w, dy, dh, dx, dresidual, dscale, dw
            a[k] = wi if k in (2, 3, 8, 9) else bad
            with pytest.raises(ValueError):
                rsq.rsq_residual_norm_backward(c, *a)
    assert not calls.names
    bad = norm_cfg()
    bad.x_dtype = 7                                           # the library's to refuse
    rsq.rsq_gated_norm(bad, x, x, w, x)
    assert calls.names == ["rsq_gated_norm"]


# ---------------------------------------------------------------------------- devices and addresses
def elsewhere(t):
    return Fake(t.t, 1)


def test_scan_refuses_any_tensor_of_another_device(calls):
    s, out, state, cu = scan_of(ragged=1), on(T, H, D, dtype=BF), on(2, H, N, D), on(3, dtype=torch.int32)
    for name in ("x", "Bm", "Cm", "dt", "A", "D", "decay"):
        a = tokens(decay=on(T, H))
        with pytest.raises(ValueError, match="cuda:1"):
            s.forward(rsq.scan_inputs(**(a | {name: elsewhere(a[name])})), out, cu_seqlens=cu)
    ins = rsq.scan_inputs(**tokens())
    ws = on(8, dtype=torch.uint8)
    good = dict(out=out, state_in=state, state_out=state, cu_seqlens=cu, workspace=ws)
    for name in good:
        with pytest.raises(ValueError, match="cuda:1"):
            s.forward(ins, **(good | {name: elsewhere(good[name])}))
    grads = dict(dx=out, dBm=on(T, G, N, dtype=BF), dCm=on(T, G, N, dtype=BF), ddt=on(T, H), dlog_decay=on(T, H), dA=on(H), dD=on(H),
                 dstate_in=state)
    good = dict(dout=out, grads=rsq.scan_grads(**grads), state_in=state, dstate_out=state, cu_seqlens=cu, workspace=ws)
    for name in good:
        if name != "grads":
            with pytest.raises(ValueError, match="cuda:1"):
                s.backward(ins, **(good | {name: elsewhere(good[name])}))
    for name in grads:
        with pytest.raises(ValueError, match="cuda:1"):
            s.backward(ins, **(good | {"grads": rsq.scan_grads(**(grads | {name: elsewhere(grads[name])}))}))
    assert not calls.names
    s.forward(ins, out, state_in=state, state_out=state, cu_seqlens=cu, workspace=ws)
    s.backward(ins, **good)
    assert calls.names == ["rsq_scan", "rsq_scan_backward"]


def norm_arguments():
    """Each norm call with the tensors of an ordinary one, by name, in order."""
    r, w, ws = on(T, N, dtype=BF), on(N), on(8, dtype=torch.uint8)
    return [(rsq.rsq_gated_norm, dict(x=r, z=r, w=w, y=r)),
            (rsq.rsq_gated_norm_backward, dict(x=r, z=r, w=w, dy=r, dx=r, dz=r, dw=w, workspace=ws)),
            (rsq.rsq_residual_norm, dict(x=r, residual=r, scale=w, w=w, h=r, y=r)),
            (rsq.rsq_residual_norm_backward, dict(x=r, h=r, scale=w, w=w, dy=r, dh=r, dx=r, dresidual=r, dscale=w, dw=w, workspace=ws))]


def test_norms_refuse_any_tensor_of_another_device(calls):
    cfg = norm_cfg()
    for call, a in norm_arguments():
        for name in a:
            with pytest.raises(ValueError, match="cuda:1"):
                call(cfg, **(a | {name: elsewhere(a[name])}))
    assert not calls.names


def test_an_address_among_tensors_lifts_no_other_check(calls):
    """An argument may be an address; the others are tensors all the same."""
    cfg = norm_cfg()
    for call, a in norm_arguments():
        for name in a:
            call(cfg, **(a | ({name: P} if name != "workspace" else {})))
            for other, t in a.items():
                if other in (name, "workspace"):
                    continue
                few = on(*[d - 1 for d in t.shape], dtype=t.dtype)
                for bad in (few, on(*t.shape, dtype=torch.float16), elsewhere(t)):
                    with pytest.raises(ValueError):
                        call(cfg, **(a | {name: P if name != "workspace" else None, other: bad}))
    assert len(calls.names) == sum(len(a) for _, a in norm_arguments())


def test_host_tensors_and_what_is_no_tensor_are_refused(calls):
    cfg = norm_cfg()
    for call, a in norm_arguments():
        for name, t in a.items():
            with pytest.raises(ValueError):
                call(cfg, **(a | {name: torch.empty(t.shape, dtype=t.dtype)}))
    assert not calls.names


def test_the_functions_check_as_the_class_does(calls):
    cfg, ins, out, state = scan_of().cfg, rsq.scan_inputs(**tokens()), on(T, H, D, dtype=BF), on(2, H, N, D)
    for kw in [dict(out=on(T - 1, H, D, dtype=BF)), dict(state_in=on(1, H, N, D)), dict(state_out=on(1, H, N, D)),
               dict(inputs=rsq.scan_inputs(**tokens(dt=on(T, 1)))), dict(cu_seqlens=on(2, dtype=torch.int32))]:
        with pytest.raises(ValueError):
            rsq.rsq_scan(cfg, **(dict(inputs=ins, out=out) | kw))
    for kw in [dict(dout=on(T - 1, H, D, dtype=BF)), dict(grads=rsq.scan_grads(dA=on(1))), dict(dstate_out=on(1, H, N, D)),
               dict(inputs=rsq.scan_inputs(**tokens(Bm=on(1, G, N, dtype=BF))))]:
        with pytest.raises(ValueError):
            rsq.rsq_scan_backward(cfg, **(dict(inputs=ins, dout=out, grads=rsq.scan_grads()) | kw))
    assert not calls.names
    rsq.rsq_scan(cfg, ins, out, state_in=state)
    rsq.rsq_scan(cfg, rsq.rsq_scan_inputs(P, P, P, P, P, None, None, 0, 0, 0), P)     # addresses alone
    rsq.rsq_scan_backward(cfg, ins, out, rsq.rsq_scan_grads(dx=P), state_in=state)
    assert calls.names == ["rsq_scan", "rsq_scan", "rsq_scan_backward"]


def test_addresses_need_no_torch():
    """A program that has addresses alone, and a stream, loads no torch and starts none of its CUDA."""
    import subprocess
    import sys
    code = """
import ctypes, sys
import ssm_decode_02_b200 as rsq
assert "torch" not in sys.modules
rsq.lib = type("Calls", (), {"__getattr__": lambda s, n: (lambda *a: rsq.RSQ_OK)})()
P = 1 << 20
cfg = rsq.rsq_norm_config(4, 64, 0, 0, 1, 1, 1, 1e-5, 0, 0)
def all_calls():
    rsq.rsq_gated_norm(cfg, P, P, P, P, stream=0)
    rsq.rsq_gated_norm_backward(cfg, P, P, P, P, P, P, None, stream=0)
    rsq.rsq_residual_norm(cfg, P, P, P, P, P, P, stream=0)
    rsq.rsq_residual_norm_backward(cfg, P, P, P, P, P, P, P, P, None, None, stream=0)
    scan = rsq.rsq_scan_config(rsq.RSQ_MAMBA2, rsq.RSQ_BF16, 1, 1, 64, 64, 1, 0, 4)
    ins = rsq.scan_inputs(P, P, P, P, P)
    rsq.rsq_scan(scan, ins, P, state_in=P, state_out=P, stream=0)
    rsq.rsq_scan_backward(scan, ins, P, rsq.scan_grads(dx=P), state_in=P, stream=0)
all_calls()
assert "torch" not in sys.modules
import torch
all_calls()
assert not torch.cuda.is_initialized()
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=rsq.os.path.dirname(rsq.os.path.dirname(rsq.__file__)))
    assert r.returncode == 0, r.stderr[-2000:]
