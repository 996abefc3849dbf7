"""The scan and the norms as a layer uses them together with the decode step, and the
calls around the ordinary ones: poisoned margins, two calls at once, graphs side by
side, offsets beyond 31 bits, the failure mark.
"""
import json
import subprocess
import sys

import numpy as np
import pytest
import torch

import ssm_decode_02_b200 as rsq
from scan_reference import U16, U32, gated64, norm64, rel, scan64
from test_gpu_redzones import MARGIN
from test_gpu_scan import cuda, dbl, inputs, make, poison, shape

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,P", [(128, 64), (32, 32)])
def test_prompt_then_decode_with_norms(N, P):
    """residual norm, scan of a ragged batch, gated norm, the state into a full-precision
    context, decode steps with their gated norm: against one recurrence in 64 bits."""
    H, steps, bounds = 4, 3, [0, 70, 70, 271]
    n, T = len(bounds) - 1, 271
    # the sequences with their later tokens, as one long reference run
    long_bounds = [0]
    for a, b in zip(bounds, bounds[1:]):
        long_bounds.append(long_bounds[-1] + (b - a) + steps)
    d, _ = make(n, long_bounds[-1], H, N, P, 1, bounds=long_bounds, seed=21, state=False)
    at = torch.cat([torch.arange(lo, hi - steps) for lo, hi in zip(long_bounds, long_bounds[1:])])
    later = [torch.tensor([hi - steps + k for hi in long_bounds[1:]]) for k in range(steps)]
    z = torch.randn(long_bounds[-1], H * P).bfloat16()
    w = 1 + 0.1 * torch.randn(H * P)
    want, _ = scan64(**dbl(d), bounds=long_bounds)
    want_y = gated64(want.flatten(1), z.double(), w.double(), H * P, 1e-5, True)

    branch, res = torch.randn(T, 64).bfloat16().cuda(), torch.randn(T, 64).cuda()
    h, y0, w0 = torch.empty_like(res), torch.empty_like(branch), torch.ones(64).cuda()
    rsq.rsq_residual_norm(rsq.norm_config(branch, res, torch.bfloat16), branch, res, None, w0, h, y0)
    ref = norm64((branch.double() + res.double()).cpu(), torch.ones(64).double(), 64, 1e-5)
    assert rel(y0, ref) <= U16

    pick = lambda i: {k: v[i].cuda() if k in ("x", "Bm", "Cm", "dt") else (None if v is None else v.cuda())  # noqa: E731
                      for k, v in d.items()}
    c = pick(at)
    scan = rsq.Scan(n, T, H, N, P, ragged=True)
    out, state = torch.empty_like(c["x"]), torch.empty((n, H, N, P), device="cuda")
    ws = poison(scan.alloc_workspace())
    scan.forward(inputs(c), out, state_out=state, workspace=ws, cu_seqlens=torch.tensor(bounds, dtype=torch.int32, device="cuda"))
    rsq.rsq_scan_check(ws)
    wc, y = w.cuda(), torch.empty((T, H * P), dtype=torch.bfloat16, device="cuda")
    zc = z[at].cuda()
    cfg = rsq.norm_config(out.flatten(1), zc, torch.bfloat16, order=rsq.RSQ_GATE_NORM)
    rsq.rsq_gated_norm(cfg, out.flatten(1), zc, wc, y)
    # the scan's output has three roundings, the norm's one more: each below U16 / 2 in the mean
    assert rel(y, want_y[at]) <= 1.5 * U16

    ctx = rsq.Context(rsq.RSQ_MAMBA2, n, H, N, P, head_bits=np.full(H, 32, np.int8), ngroups=1)
    st = ctx.alloc_state()
    ctx.quantize(state, st)
    for k in range(steps):
        t = pick(later[k])
        o = torch.empty((n, H, P), device="cuda")
        ctx.decode_step(st, st, rsq.mamba2_inputs(t["x"], t["Bm"], t["Cm"], t["dt"], t["A"], t["D"]), o, k)
        big = want[later[k]].abs().max()
        assert (o.double().cpu() - want[later[k]]).abs().max() <= (T + N) * 2.0 ** -23 * big * 8   # |terms| reach a few times |o|
        yk, zk = torch.empty((n, H * P), dtype=torch.bfloat16, device="cuda"), z[later[k]].cuda()
        rsq.rsq_gated_norm(rsq.norm_config(o.flatten(1), zk, torch.bfloat16, order=rsq.RSQ_GATE_NORM), o.flatten(1), zk, wc, yk)
        assert rel(yk, want_y[later[k]]) <= U16
        # the scan's own single-token form, from the same state
        if k == 0:
            one = rsq.Scan(n, n, H, N, P)
            o1, s1 = torch.empty_like(t["x"]), torch.empty_like(state)
            one.forward(inputs(t), o1, state_in=state, state_out=s1)
            assert rel(o1, o.cpu()) <= U16
            S = torch.empty_like(state)
            ctx.dequantize(st, S)
            assert (s1 - S).abs().max() <= 4 * U32 * S.abs().max()
    ctx.close()


class Margins:
    """Tensors inside larger buffers whose margins must not change (outputs) or hold NaN (inputs)."""

    def __init__(self):
        self.kept = []

    def put(self, t, poison=0xFF):
        if t is None:
            return None
        raw = t.contiguous().view(-1).view(torch.uint8)
        big = torch.full((raw.numel() + 2 * MARGIN,), poison, dtype=torch.uint8, device="cuda")
        big[MARGIN:MARGIN + raw.numel()] = raw
        self.kept.append((big, big.clone()))
        return big[MARGIN:MARGIN + raw.numel()].view(t.dtype).view(t.shape)

    def check(self, outputs):
        torch.cuda.synchronize()
        for (big, before), out in zip(self.kept, outputs):
            assert torch.equal(big[:MARGIN], before[:MARGIN]) and torch.equal(big[-MARGIN:], before[-MARGIN:])
            if not out:
                assert torch.equal(big, before), "an input changed"


@pytest.mark.parametrize("N,P,G", [(128, 64, 1), (64, 128, 2), (16, 16, 2), (256, 64, 1)])
@pytest.mark.parametrize("ragged", [False, True])
def test_nothing_outside_the_buffers_is_read_or_written(N, P, G, ragged):
    H, bounds = 4, [0, 130, 130, 301, 400]
    n, T = 4, 400
    d, bounds = make(n, T, H, N, P, G, bounds=bounds if ragged else None, seed=31)
    s = shape(d, n, ragged=ragged)
    m = Margins()
    c = {k: m.put(None if v is None else v.cuda()) for k, v in d.items()}
    cu = m.put(torch.tensor(bounds, dtype=torch.int32, device="cuda")) if ragged else None
    dout, dstate = m.put(torch.randn(d["x"].shape).bfloat16().cuda()), m.put(torch.randn(n, H, N, P).cuda())
    ins = len(m.kept)
    outs = {"out": torch.empty_like(d["x"]), "state": torch.empty(n, H, N, P), "dx": torch.empty_like(d["x"]),
            "dBm": torch.empty_like(d["Bm"]), "dCm": torch.empty_like(d["Cm"]), "ddt": torch.empty(T, H), "dlog_decay": torch.empty(T, H),
            "dA": torch.empty(H), "dD": torch.empty(H), "dstate_in": torch.empty(n, H, N, P)}
    o = {k: m.put(v.cuda(), 0xA5) for k, v in outs.items()}
    ws, bws = (m.put(torch.full((k,), 255, dtype=torch.uint8, device="cuda"), 0xA5) for k in (s.workspace_bytes, s.backward_workspace_bytes))
    s.forward(inputs(c), o["out"], state_in=c["state_in"], state_out=o["state"], cu_seqlens=cu, workspace=ws)
    s.backward(inputs(c), dout, rsq.scan_grads(**{k: v for k, v in o.items() if k.startswith("d")}), state_in=c["state_in"],
               dstate_out=dstate, cu_seqlens=cu, workspace=bws)
    m.check([False] * ins + [True] * (len(m.kept) - ins))
    for k, v in o.items():
        assert torch.isfinite(v.float()).all(), k


@pytest.mark.parametrize("rows,width,group", [(5, 128, 32), (3, 99, 33), (2, 5120, 5120)])
def test_norms_stay_inside_their_buffers(rows, width, group):
    m = Margins()
    x, z, dy = (m.put(torch.randn(rows, width).bfloat16().cuda()) for _ in range(3))
    w = m.put(torch.randn(width).cuda())
    outs = [m.put(torch.empty(rows, width).bfloat16().cuda(), 0xA5) for _ in range(3)] + [m.put(torch.empty(width).cuda(), 0xA5)]
    cfg = rsq.norm_config(x, z, torch.bfloat16, group=group)
    ws = m.put(torch.empty(rsq.rsq_norm_workspace(cfg), dtype=torch.uint8, device="cuda"), 0xA5)
    rsq.rsq_gated_norm(cfg, x, z, w, outs[0])
    rsq.rsq_gated_norm_backward(cfg, x, z, w, dy, outs[1], outs[2], outs[3], ws)
    m.check([False] * 4 + [True] * 5)
    assert all(torch.isfinite(o.float()).all() for o in outs)


def test_two_calls_at_once_and_two_graphs():
    """Two streams, and two captured graphs replayed together, each call with its own workspace."""
    runs = []
    for seed in (41, 42):
        d, bounds = make(2, 1400, 4, 64, 64, 1, seed=seed)
        c = cuda(d)
        s = shape(d, 2)
        dout = torch.randn(d["x"].shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        o = {"out": torch.empty_like(c["x"]), "state": torch.empty_like(c["state_in"]), "dx": torch.empty_like(c["x"]),
             "ddt": torch.empty_like(c["dt"]), "dBm": torch.empty_like(c["Bm"])}
        ws, bws = s.alloc_workspace(), s.alloc_workspace(True)

        def call(c=c, s=s, dout=dout, o=o, ws=ws, bws=bws):
            s.forward(inputs(c), o["out"], state_in=c["state_in"], state_out=o["state"], workspace=ws)
            s.backward(inputs(c), dout, rsq.scan_grads(dx=o["dx"], ddt=o["ddt"], dBm=o["dBm"]), state_in=c["state_in"], workspace=bws)
        call()
        torch.cuda.synchronize()
        runs.append((call, o, {k: v.clone() for k, v in o.items()}))
    streams = [torch.cuda.Stream() for _ in runs]
    graphs = []
    for (call, o, _), st in zip(runs, streams):
        with torch.cuda.stream(st):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                call()
            graphs.append(g)
    for way in ("streams", "graphs"):
        for _, o, _ in runs:
            for v in o.values():
                v.fill_(float("nan"))
        torch.cuda.synchronize()
        for (call, _, _), st, g in zip(runs, streams, graphs):
            with torch.cuda.stream(st):
                for _ in range(3):
                    call() if way == "streams" else g.replay()
        torch.cuda.synchronize()
        for _, o, want in runs:
            for k in o:
                assert torch.equal(o[k], want[k]), (way, k)


def test_offsets_beyond_31_bits():
    """More than 2^31 elements of x.  A decay of zero restarts the state near the end, so that
    the last tokens have to equal a call on them alone."""
    H, P, N, T, tail = 256, 128, 64, 65664, 200
    assert T * H * P > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((T, H, P), dtype=torch.bfloat16, device="cuda")
    x[-tail:] = torch.randn((tail, H, P), generator=g, device="cuda").bfloat16()
    x[:300] = 1.0
    Bm, Cm = (torch.randn((T, 1, N), generator=g, device="cuda").bfloat16() for _ in range(2))
    decay = torch.full((T, H), 0.99, device="cuda")
    decay[-tail] = 0.0

    def run(lo):
        s = rsq.Scan(1, T - lo, H, N, P)
        out = torch.empty((T - lo, H, P), dtype=torch.bfloat16, device="cuda")
        state = torch.empty((1, H, N, P), device="cuda")
        ins = rsq.scan_inputs(x[lo:], Bm[lo:], Cm[lo:], decay=decay[lo:])
        s.forward(ins, out, state_out=state, workspace=s.alloc_workspace())
        dx, dC = torch.empty_like(out), torch.empty_like(Cm[lo:])
        dl = torch.empty((T - lo, H), device="cuda")
        s.backward(ins, x[lo:], rsq.scan_grads(dx=dx, dCm=dC, dlog_decay=dl), workspace=s.alloc_workspace(True))
        return out[-tail:].clone(), state, dx[-tail:].clone(), dC[-tail:].clone(), dl[-tail:].clone()

    whole, part = run(0), run(T - tail)
    # other chunk borders, so other roundings: three of U16 in either, binary32 sums of tail + N terms
    for k, tol in zip(range(5), (2 * U16, 300 * 2.0 ** -23, 2 * U16, 2 * U16, 300 * 2.0 ** -23)):
        assert rel(whole[k], part[k].cpu()) <= tol, k


def test_failure_mark_is_reported():
    d, _ = make(1, 130, 2, 64, 64, 1, seed=3)
    c, s = cuda(d), shape(d, 1)
    ws = poison(s.alloc_workspace())
    s.forward(inputs(c), torch.empty_like(c["x"]), workspace=ws)
    rsq.rsq_scan_check(ws)
    ws[:4] = torch.tensor([2, 0, 0, 0], dtype=torch.uint8, device="cuda")   # as a wait that ran out leaves it
    with pytest.raises(rsq.RsqError) as e:
        rsq.rsq_scan_check(ws)
    assert e.value.status == rsq.RSQ_E_CUDA
    s.forward(inputs(c), torch.empty_like(c["x"]), workspace=ws)             # the next call clears it
    rsq.rsq_scan_check(ws)


@pytest.mark.parametrize("tokens", [64, 512])
def test_prompt_mode_of_the_bench(tokens):
    r = subprocess.run([sys.executable, "bench.py", "--workload", "mamba2_b128_h80_p64_n128_int8_sr", "--prompt", str(tokens), "--steps", "10",
                        "--warmup", "3"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["metric"] == "prompt_tokens_per_s" and line["value"] > 0 and line["flags"] == 0
