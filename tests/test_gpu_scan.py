"""rsq_scan and rsq_scan_backward on the GPU against the recurrence in 64 bits.

Tolerances.  A bf16 output is the sum of two products, each with one operand
rounded to bf16 (the scores, the state), and is rounded itself: element by
element at most U16 (S + |y|) with S the sum of the absolute terms, plus binary32
sums, n terms at n 2^-24 S (U16 = 2^-8, half a step).  Over all elements the
roundings are independent: the 2-norm of the error is below U16 of the 2-norm
(three roundings of rms 2^-8 / sqrt(3) at a power of two, less above it).
A binary32 output has 24-bit operands and sums of n terms in binary32: n 2^-23 S
(2^-23: the matrix units truncate), n = tokens of the longest sequence + dk; the
gradients of the gates add rounded sums of both signs, and are held to n 2^-23 of
their largest element.
"""
import numpy as np
import pytest
import torch

import ssm_decode_02_b200 as rsq
from scan_reference import U16, magnitude, rel, scan64

pytestmark = pytest.mark.gpu


def make(n, tokens, H, N, P, G, *, bounds=None, decay=False, D=True, state=True, seed=0, strong=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    bounds = [tokens // n * i for i in range(n + 1)] if bounds is None else list(bounds)
    d = {"x": r(tokens, H, P).bfloat16(), "Bm": r(tokens, G, N).bfloat16(), "Cm": r(tokens, G, N).bfloat16()}
    if decay:
        a = torch.sigmoid(r(tokens, H) * (6 if strong else 1) + (0 if strong else 2.5))
        if strong:
            a = torch.where(torch.rand(tokens, H, generator=g) < 0.1, torch.zeros_like(a), a)
        d |= {"dt": None, "A": None, "decay": a}
    else:
        d |= {"dt": torch.nn.functional.softplus(r(tokens, H) - (0 if strong else 2)),
              "A": -torch.exp((8 if strong else 2.8) * torch.rand(H, generator=g)), "decay": None}
    d["D"] = 1 + 0.1 * r(H) if D else None
    d["state_in"] = r(n, H, N, P) if state else None
    return d, bounds


def dbl(d, grad=False):
    return {k: None if v is None else v.double().requires_grad_(grad) for k, v in d.items()}


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def inputs(c):
    return rsq.scan_inputs(c["x"], c["Bm"], c["Cm"], c["dt"], c["A"], c["D"], c["decay"])


def shape(d, n, **kw):
    T, H, P = d["x"].shape
    return rsq.Scan(n, T, H, d["Bm"].shape[2], P, ngroups=d["Bm"].shape[1], **kw)


def poison(t):
    """A workspace of NaN: nothing in it may be read before it is written."""
    return None if t is None else t.fill_(255)


def forward(d, bounds, ragged, n):
    c = cuda(d)
    s = shape(d, n, ragged=ragged)
    T, H, P = d["x"].shape
    out = torch.full((T, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    state = torch.empty((n, H, d["Bm"].shape[2], P), device="cuda")
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda") if ragged else None
    s.forward(inputs(c), out, state_in=c["state_in"], state_out=state, cu_seqlens=cu, workspace=poison(s.alloc_workspace()))
    torch.cuda.synchronize()
    return out.cpu(), state.cpu()


def check_forward(d, bounds, out, state):
    want, final = scan64(**dbl(d), bounds=bounds)
    big, fbig = magnitude(**dbl(d), bounds=bounds)
    n = max(b - a for a, b in zip(bounds, bounds[1:])) + d["Bm"].shape[2]
    inside = torch.zeros(d["x"].shape[0], dtype=torch.bool)
    inside[bounds[0]:bounds[-1]] = True
    assert torch.all(out[~inside] == 7.0), "rows of no sequence were written"
    o, w, b = out[inside].double(), want[inside], big[inside]
    assert torch.all((o - w).abs() <= U16 * (b + w.abs()) + n * 2.0 ** -23 * b + 1e-30)
    assert rel(o, w) <= U16
    assert torch.all((state.double() - final).abs() <= n * 2.0 ** -23 * fbig + 1e-30)


EQUAL = [  # n, tokens, H, N, P, G
    (1, 1, 2, 16, 16, 1), (3, 3, 4, 128, 64, 1), (2, 4, 3, 256, 256, 3), (2, 8, 2, 64, 32, 2), (2, 10, 2, 32, 16, 1),
    (1, 127, 2, 128, 64, 1), (2, 256, 4, 64, 128, 2), (1, 129, 3, 16, 256, 3), (1, 300, 2, 256, 64, 1),
    (3, 3 * 65, 2, 32, 16, 2), (1, 513, 5, 128, 64, 1), (1, 200, 2, 128, 32, 1),
    (1, 300, 2, 64, 256, 1), (2, 280, 2, 256, 256, 2), (1, 260, 2, 256, 128, 1), (1, 384, 4, 128, 128, 4), (5, 5 * 20, 2, 64, 64, 2),
]


@pytest.mark.parametrize("n,tokens,H,N,P,G", EQUAL)
@pytest.mark.parametrize("decay", [False, True])
def test_forward_equal_lengths(n, tokens, H, N, P, G, decay):
    d, bounds = make(n, tokens, H, N, P, G, decay=decay, D=not decay, state=tokens % 2 == 1, seed=tokens)
    check_forward(d, bounds, *forward(d, bounds, False, n))


RAGGED = [([0, 1], 1), ([0, 12, 25, 25, 26, 300], 300), ([0, 0, 5, 5, 140, 269], 269), ([3, 3, 131, 259, 300], 310), ([0, 130, 131, 131], 140)]


@pytest.mark.parametrize("bounds,tokens", RAGGED)
@pytest.mark.parametrize("H,N,P,G", [(3, 64, 64, 1), (2, 128, 128, 2), (2, 16, 16, 1)])
def test_forward_ragged(bounds, tokens, H, N, P, G):
    n = len(bounds) - 1
    d, bounds = make(n, tokens, H, N, P, G, bounds=bounds, seed=tokens)
    check_forward(d, bounds, *forward(d, bounds, True, n))


MOSTLY_SHORT = [[13] * 10 + [0],                                   # as many long ones as the tokens allow
                [200] + [1] * 70 + [12, 13, 0, 140] + [1] * 30 + [129],
                [1, 0, 3, 12] * 12 + [300], [12] * 40]


@pytest.mark.parametrize("lengths", MOSTLY_SHORT)
@pytest.mark.parametrize("H,N,P", [(2, 128, 64), (3, 32, 32)])
def test_forward_mostly_short(lengths, H, N, P):
    bounds = [0]
    for k in lengths:
        bounds.append(bounds[-1] + k)
    d, bounds = make(len(lengths), bounds[-1], H, N, P, 1, bounds=bounds, seed=len(lengths))
    check_forward(d, bounds, *forward(d, bounds, True, len(lengths)))


@pytest.mark.parametrize("decay", [False, True])
def test_forward_strong_decays_and_restarts(decay):
    """Decays of zero (a restart) and far below the smallest float, next to slow ones."""
    d, bounds = make(1, 300, 4, 64, 64, 1, decay=decay, strong=True, seed=5)
    check_forward(d, bounds, *forward(d, bounds, False, 1))


def test_forward_long_sequence_in_segments():
    d, bounds = make(1, 128 * 40 + 17, 2, 16, 16, 1, seed=8)
    assert rsq.Scan(1, 128 * 40, 2, 16, 16).workspace_bytes > 0
    check_forward(d, bounds, *forward(d, bounds, False, 1))


@pytest.mark.parametrize("H,N,P", [(1, 16, 16), (2, 64, 64), (1, 128, 128)])
def test_segments_of_a_ragged_batch(H, N, P):
    bounds = [0, 0, 2100, 2101, 5000] if N == 16 else [0, 0, 4500, 4501, 4700]
    total = bounds[-1] + 3
    d, bounds = make(4, total, H, N, P, 1, bounds=bounds, seed=9)
    check_forward(d, bounds, *forward(d, bounds, True, 4))


def test_growing_states():
    """Decays above one: a state that grows."""
    d, bounds = make(1, 300, 2, 64, 64, 1, decay=True, seed=15)
    d["decay"] = 1 + 0.04 * (d["decay"] - 0.5)
    check_forward(d, bounds, *forward(d, bounds, False, 1))


def test_prompt_in_pieces_equals_the_prompt():
    """The state of a prefix carries on: one call, or two with the state between (in place)."""
    d, _ = make(1, 300, 2, 64, 64, 1, seed=3)
    whole, final = forward(d, [0, 300], False, 1)
    c = cuda(d)
    state = c["state_in"].clone()
    outs = []
    for lo, hi in ((0, 171), (171, 172), (172, 300)):
        s = rsq.Scan(1, hi - lo, 2, 64, 64)
        piece = {k: (v[lo:hi].contiguous() if k in ("x", "Bm", "Cm", "dt") else v) for k, v in c.items()}
        out = torch.empty((hi - lo, 2, 64), dtype=torch.bfloat16, device="cuda")
        s.forward(inputs(piece), out, state_in=state, state_out=state, workspace=poison(s.alloc_workspace()))
        outs.append(out)
    check_forward(d, [0, 300], torch.cat(outs).cpu(), state.cpu())
    assert rel(torch.cat(outs).cpu(), whole) <= 2 * U16 and rel(state.cpu(), final) <= 300 * 2.0 ** -23


def test_token_rows_may_lie_apart():
    """x, B and C as slices of one projection's output."""
    d, bounds = make(2, 260, 2, 32, 64, 1, seed=4)
    T = 260
    proj = torch.full((T, 2 * 64 + 32 + 32 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    x, Bm, Cm = proj[:, :128].view(T, 2, 64), proj[:, 128:160].view(T, 1, 32), proj[:, 160:192].view(T, 1, 32)
    x.copy_(d["x"]), Bm.copy_(d["Bm"]), Cm.copy_(d["Cm"])
    c = cuda(d)
    s = shape(d, 2)
    out, state = torch.empty((T, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 2, 32, 64), device="cuda")
    s.forward(rsq.scan_inputs(x, Bm, Cm, c["dt"], c["A"], c["D"]), out, state_in=c["state_in"], state_out=state,
              workspace=poison(s.alloc_workspace()))
    check_forward(d, bounds, out.cpu(), state.cpu())


@pytest.mark.parametrize("N", [16, 64])
def test_no_tokens_keeps_the_state(N):
    c = torch.randn(2, 2, N, 64, device="cuda")
    for ragged in (False, True):
        s = rsq.Scan(2, 0, 2, N, 64, ragged=ragged)
        state = torch.empty_like(c)
        ones = torch.ones(4, device="cuda")
        cu = torch.zeros(3, dtype=torch.int32, device="cuda") if ragged else None
        none = rsq.scan_inputs(None, None, None, ones, ones)
        s.forward(none, None, state_in=c, state_out=state, cu_seqlens=cu, workspace=poison(s.alloc_workspace()))
        assert torch.equal(state, c)
        dA, dS = torch.full((2,), 5.0, device="cuda"), torch.empty_like(c)
        ws = poison(s.alloc_workspace(True))
        s.backward(none, None, rsq.scan_grads(dA=dA, dstate_in=dS), dstate_out=c, cu_seqlens=cu, workspace=ws)
        rsq.rsq_scan_check(ws)
        assert torch.equal(dS, c) and (dA == 0).all()


def test_nan_stays_in_its_sequence_and_behind_bad_bounds_nothing_moves():
    d, bounds = make(3, 390, 2, 32, 32, 1, bounds=[0, 130, 260, 390], seed=6, state=False)
    d["x"][140] = float("nan")
    out, state = forward(d, bounds, True, 3)
    assert torch.isfinite(out[:130].float()).all() and torch.isfinite(out[260:].float()).all()
    assert torch.isfinite(state[[0, 2]]).all() and torch.isnan(out[260 - 1].float()).all()
    # bounds outside of the rows are clamped
    d["x"][140] = 0.5
    want, _ = forward(d, [0, 130, 260, 390], True, 3)
    got, _ = forward(d, [-7, 130, 260, 4000], True, 3)
    assert torch.equal(got, want)


# --------------------------------------------------------------------------------------- backward
def backward(d, bounds, ragged, n, dout, dstate):
    c = cuda(d)
    s = shape(d, n, ragged=ragged)
    new = lambda t, v: torch.full_like(t, v)  # noqa: E731
    g = {"dx": new(c["x"], 7), "dBm": new(c["Bm"], 7), "dCm": new(c["Cm"], 7), "dstate_in": torch.empty(
        (n, *c["x"].shape[1:2], c["Bm"].shape[2], c["x"].shape[2]), device="cuda")}
    gates = torch.full(c["x"].shape[:2], 7.0, device="cuda")
    g["dlog_decay"] = gates
    if c["decay"] is None:
        g |= {"ddt": gates.clone(), "dA": torch.empty_like(c["A"])}
    if c["D"] is not None:
        g["dD"] = torch.empty_like(c["D"])
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda") if ragged else None
    s.backward(inputs(c), dout.cuda(), rsq.scan_grads(**g), state_in=c["state_in"],
               dstate_out=None if dstate is None else dstate.cuda(), cu_seqlens=cu,
               workspace=poison(s.alloc_workspace(backward=True)))
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in g.items()}


def reference_grads(d, bounds, dout, dstate):
    """Autograd through the recurrence in 64 bits; the decay's logarithm by its own leaf."""
    v = dbl(d, grad=True)
    T, H, _ = d["x"].shape
    scale = torch.zeros(T, H, dtype=torch.float64, requires_grad=True)   # log of a factor on a_t
    a = (v["decay"] if v["decay"] is not None else torch.exp(v["dt"] * v["A"])) * torch.exp(scale)
    n, N, P = len(bounds) - 1, d["Bm"].shape[2], d["x"].shape[2]
    start = v["state_in"] if v["state_in"] is not None else torch.zeros(n, H, N, P, dtype=torch.float64, requires_grad=True)
    out, final = scan64(v["x"], v["Bm"], v["Cm"], v["dt"], None, v["D"], a, start, bounds)
    loss = (out * dout.double()).sum() + (0 if dstate is None else (final * dstate.double()).sum())
    names = {"dx": v["x"], "dBm": v["Bm"], "dCm": v["Cm"], "dstate_in": start, "dlog_decay": scale}
    if v["decay"] is None:
        names |= {"ddt": v["dt"], "dA": v["A"]}
    if v["D"] is not None:
        names["dD"] = v["D"]
    return dict(zip(names, torch.autograd.grad(loss, list(names.values()), allow_unused=True)))


def check_backward(d, bounds, got, want):
    n = max(b - a for a, b in zip(bounds, bounds[1:])) + d["Bm"].shape[2]
    inside = torch.zeros(d["x"].shape[0], dtype=torch.bool)
    inside[bounds[0]:bounds[-1]] = True
    for k, w in want.items():
        o = got[k].double()
        w = torch.zeros_like(o) if w is None else w
        if k in ("dx", "dBm", "dCm", "ddt", "dlog_decay"):
            assert torch.all(o[~inside] == 7.0), k
            o, w = o[inside], w[inside]
        if k in ("dx", "dBm", "dCm"):
            assert rel(o, w) <= U16, (k, rel(o, w))
            # three roundings, each half a step of a partial sum; partial sums reach a few times the largest result
            assert (o - w).abs().max() <= 8 * U16 * w.abs().max(), k
        else:
            assert (o - w).abs().max() <= n * 2.0 ** -23 * w.abs().max(), (k, (o - w).abs().max() / w.abs().max())


BACK = [(1, 1, 2, 16, 16, 1), (2, 256, 4, 64, 64, 2), (1, 129, 3, 128, 64, 1), (1, 140, 2, 256, 128, 2), (2, 60, 3, 32, 256, 1),
        (1, 400, 2, 16, 32, 2), (3, 3 * 131, 2, 128, 128, 1), (1, 200, 2, 64, 256, 1), (1, 256, 2, 256, 256, 2), (1, 256, 4, 128, 128, 4),
        (2, 2 * 70, 6, 64, 64, 2)]


@pytest.mark.parametrize("n,tokens,H,N,P,G", BACK)
@pytest.mark.parametrize("decay", [False, True])
def test_backward_equal_lengths(n, tokens, H, N, P, G, decay):
    d, bounds = make(n, tokens, H, N, P, G, decay=decay, D=not decay, state=tokens % 2 == 0, seed=tokens)
    g = torch.Generator().manual_seed(1)
    dout = torch.randn(d["x"].shape, generator=g).bfloat16()
    dstate = torch.randn((n, H, N, P), generator=g) if tokens % 3 else None
    check_backward(d, bounds, backward(d, bounds, False, n, dout, dstate), reference_grads(d, bounds, dout, dstate))


@pytest.mark.parametrize("bounds,tokens", RAGGED)
def test_backward_ragged(bounds, tokens):
    n = len(bounds) - 1
    d, bounds = make(n, tokens, 3, 64, 32, 1, bounds=bounds, seed=tokens)
    g = torch.Generator().manual_seed(2)
    dout, dstate = torch.randn(d["x"].shape, generator=g).bfloat16(), torch.randn((n, 3, 64, 32), generator=g)
    check_backward(d, bounds, backward(d, bounds, True, n, dout, dstate), reference_grads(d, bounds, dout, dstate))


@pytest.mark.parametrize("decay", [False, True])
def test_backward_strong_decays_and_restarts(decay):
    d, bounds = make(1, 200, 3, 32, 32, 1, decay=decay, strong=True, seed=5)
    g = torch.Generator().manual_seed(3)
    dout, dstate = torch.randn(d["x"].shape, generator=g).bfloat16(), torch.randn((1, 3, 32, 32), generator=g)
    got = backward(d, bounds, False, 1, dout, dstate)
    check_backward(d, bounds, got, reference_grads(d, bounds, dout, dstate))
    if decay:
        assert (got["dlog_decay"][d["decay"] == 0] == 0).all()


@pytest.mark.parametrize("T,H,N,P", [(128 * 33 + 5, 1, 16, 16), (128 * 18 + 70, 2, 64, 64)])
def test_backward_long_sequence_in_segments(T, H, N, P):
    d, bounds = make(1, T, H, N, P, 1, seed=8)
    g = torch.Generator().manual_seed(4)
    dout, dstate = torch.randn(d["x"].shape, generator=g).bfloat16(), torch.randn((1, H, N, P), generator=g)
    check_backward(d, bounds, backward(d, bounds, False, 1, dout, dstate), reference_grads(d, bounds, dout, dstate))


def test_gradient_against_differences():
    """The loss along a direction of all inputs, by central differences of the 64-bit recurrence."""
    d, bounds = make(2, 260, 2, 32, 32, 1, seed=11)
    g = torch.Generator().manual_seed(5)
    dout, dstate = torch.randn(d["x"].shape, generator=g).bfloat16(), torch.randn((2, 2, 32, 32), generator=g)
    got = backward(d, bounds, False, 2, dout, dstate)
    names = {"x": "dx", "Bm": "dBm", "Cm": "dCm", "dt": "ddt", "A": "dA", "D": "dD", "state_in": "dstate_in"}
    base = dbl(d)
    h = 1e-5
    for k, gk in names.items():
        way = torch.randn(base[k].shape, generator=g, dtype=torch.float64)
        # along the gradient itself too, so that the derivative is not small beside the norms
        way = way + got[gk].double() / got[gk].double().norm() * way.norm()

        def loss(sign):
            out, final = scan64(**(base | {k: base[k] + sign * h * way}), bounds=bounds)
            return (out * dout.double()).sum() + (final * dstate.double()).sum()
        slope = ((loss(1) - loss(-1)) / (2 * h)).item()
        mine = (got[gk].double() * way).sum().item()
        assert abs(slope - mine) <= 2 * U16 * abs(slope), (k, slope, mine)


def test_backward_is_repeatable_and_takes_partial_requests():
    d, bounds = make(2, 260, 4, 64, 64, 2, seed=12)
    dout = torch.randn(d["x"].shape).bfloat16()
    a, b = (backward(d, bounds, False, 2, dout, None) for _ in range(2))
    for k in a:
        assert torch.equal(a[k], b[k]), k
    c = cuda(d)
    s = shape(d, 2)
    dx = torch.empty_like(c["x"])
    s.backward(inputs(c), dout.cuda(), rsq.scan_grads(dx=dx), state_in=c["state_in"], workspace=s.alloc_workspace(True))
    assert torch.equal(dx.cpu(), a["dx"])


def test_graph_replay_and_side_stream():
    """Captured with its own workspace and replayed on other inputs; and on a stream of its own."""
    d, bounds = make(2, 600, 2, 64, 64, 1, seed=13)
    e, _ = make(2, 600, 2, 64, 64, 1, seed=14)
    c = cuda(d)
    s = shape(d, 2)
    out, state = torch.empty_like(c["x"]), torch.empty_like(c["state_in"])
    ws, bws = s.alloc_workspace(), s.alloc_workspace(True)
    dout = torch.randn(d["x"].shape).bfloat16().cuda()
    dx, ddt = torch.empty_like(c["x"]), torch.empty_like(c["dt"])

    def both():
        s.forward(inputs(c), out, state_in=c["state_in"], state_out=state, workspace=ws)
        s.backward(inputs(c), dout, rsq.scan_grads(dx=dx, ddt=ddt), state_in=c["state_in"], workspace=bws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    check_forward(d, bounds, out.cpu(), state.cpu())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k, v in cuda(e).items():
        if v is not None:
            c[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(e, bounds, out.cpu(), state.cpu())
    got = {"dx": dx.cpu(), "ddt": ddt.cpu()}
    want = reference_grads(e, bounds, dout.cpu(), None)
    check_backward(e, bounds, got, {k: want[k] for k in got})
