"""Paths of the scan that its other tests do not take: ragged batches in segments, token
rows that lie apart on the tensor-map path, strong decays in the tcgen05 gradient, states in
place.  References and tolerances are those of test_gpu_scan.py."""
import pytest
import torch

import ssm_decode_02_b200 as rsq
from scan_reference import scan64
from test_gpu_scan import check_backward, check_forward, cuda, dbl, inputs, make, poison, reference_grads, shape

pytestmark = pytest.mark.gpu


def run(d, bounds, *, ragged, apart=False, in_place=False, dout=None, dstate=None):
    """(out, state_out, gradients): forward and, with dout, backward.  Rows of no sequence hold NaN.
    apart: x, B and C are slices of one array whose other columns hold NaN."""
    c, n = cuda(d), len(bounds) - 1
    T, H, P = d["x"].shape
    G, N = d["Bm"].shape[1:]
    if apart:
        wide = torch.full((T, H * P + 2 * G * N + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        at = [0, H * P + 8, H * P + G * N + 8, H * P + 2 * G * N + 8]
        for k, lo, hi in (("x", at[0], H * P), ("Bm", at[1], at[2]), ("Cm", at[2], at[3])):
            wide[:, lo:hi] = c[k].flatten(1)
            c[k] = wide[:, lo:hi].view(c[k].shape)
            assert not c[k].is_contiguous()
    for k in ("x", "Bm", "Cm", "dt", "decay"):
        if c[k] is not None:
            c[k][:bounds[0]] = float("nan")
            c[k][bounds[-1]:] = float("nan")
    s = shape(d, n, ragged=ragged)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda") if ragged else None
    out = torch.full((T, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    start = c["state_in"]
    state = start.clone() if in_place else torch.empty((n, H, N, P), device="cuda")
    ws = poison(s.alloc_workspace())
    s.forward(inputs(c), out, state_in=state if in_place else start, state_out=state, cu_seqlens=cu, workspace=ws)
    rsq.rsq_scan_check(ws)
    if dout is None:
        return out.cpu(), state.cpu(), None
    full = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")  # noqa: E731
    g = {"dx": full(d["x"]), "dBm": full(d["Bm"]), "dCm": full(d["Cm"]), "dlog_decay": torch.full((T, H), 7.0, device="cuda"),
         "dstate_in": dstate.cuda() if in_place else torch.empty((n, H, N, P), device="cuda")}
    if d["dt"] is not None:
        g["ddt"] = full(d["dt"])
    if d["decay"] is None:
        g["dA"] = full(d["A"])
    if d["D"] is not None:
        g["dD"] = full(d["D"])
    doutc = dout.cuda()
    doutc[:bounds[0]] = float("nan")
    doutc[bounds[-1]:] = float("nan")
    bws = poison(s.alloc_workspace(backward=True))
    s.backward(inputs(c), doutc, rsq.scan_grads(**g), state_in=start, dstate_out=g["dstate_in"] if in_place else dstate.cuda(),
               cu_seqlens=cu, workspace=bws)
    rsq.rsq_scan_check(bws)
    return out.cpu(), state.cpu(), {k: v.cpu() for k, v in g.items()}


def gradients_of(d, n, seed):
    g = torch.Generator().manual_seed(seed)
    T, H, P = d["x"].shape
    return torch.randn(d["x"].shape, generator=g).bfloat16(), torch.randn((n, H, d["Bm"].shape[2], P), generator=g)


def check_all(d, bounds, got, dout, dstate):
    out, state, grads = got
    check_forward(d, bounds, out, state)
    check_backward(d, bounds, grads, reference_grads(d, bounds, dout, dstate))


# ------------------------------------------------------------------------------------- segments
def bytes_without_segments(n, T, H, N, P, backward):
    """The workspace of a ragged call whose sequences are not cut into segments."""
    slots = T // 128 + n
    cells, state = slots * H, N * 64 * -(-P // 64)
    sizes = [4, slots * 8, cells * 128 * 8, cells * 128 * 4]
    sizes += [cells * state * 4, cells * state * 4, 2 * cells * 4] if backward else [cells * state * 2]
    return sum(-(-k // 256) * 256 for k in sizes)


SEGMENTED = [3, 5603, 5603, 5604, 5613, 9690]    # long, empty, one token, nine tokens, long
ROWS = 9700


def test_the_size_without_segments_is_known():
    s = rsq.Scan(40, ROWS, 2, 64, 64, ragged=True)     # too many sequences for segments
    assert s.workspace_bytes == bytes_without_segments(40, ROWS, 2, 64, 64, False)
    assert s.backward_workspace_bytes == bytes_without_segments(40, ROWS, 2, 64, 64, True)


@pytest.mark.parametrize("H,N,P", [(1, 16, 16), (2, 64, 64), (1, 64, 256), (1, 256, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_ragged_batch_in_segments(H, N, P, in_place):
    n = len(SEGMENTED) - 1
    s = rsq.Scan(n, ROWS, H, N, P, ragged=True)
    assert s.workspace_bytes > bytes_without_segments(n, ROWS, H, N, P, False)
    assert s.backward_workspace_bytes > bytes_without_segments(n, ROWS, H, N, P, True)
    d, bounds = make(n, ROWS, H, N, P, 1, bounds=SEGMENTED, seed=51)
    dout, dstate = gradients_of(d, n, 52)
    check_all(d, bounds, run(d, bounds, ragged=True, in_place=in_place, dout=dout, dstate=dstate), dout, dstate)


# --------------------------------------------------------------------------------- rows that lie apart
@pytest.mark.parametrize("H,N,P,G", [(2, 64, 64, 1), (4, 128, 64, 2), (2, 128, 128, 2), (2, 256, 64, 1), (1, 64, 256, 1)])
@pytest.mark.parametrize("bounds", [[0, 300, 600], [5, 261, 261, 274, 590]])
def test_rows_apart_on_tensor_maps(H, N, P, G, bounds):
    """x, B and C as slices of one projection, as a Mamba-2 layer has them: whole chunks come as
    tensor-map boxes, the last rows of a sequence by themselves."""
    n, ragged = len(bounds) - 1, bounds[0] > 0
    d, bounds = make(n, 600, H, N, P, G, bounds=bounds, seed=61)
    dout, dstate = gradients_of(d, n, 62)
    check_all(d, bounds, run(d, bounds, ragged=ragged, apart=True, dout=dout, dstate=dstate), dout, dstate)


# --------------------------------------------------------------------------------------- strong decays
@pytest.mark.parametrize("H,N,P,G", [(4, 64, 64, 1), (4, 128, 64, 2), (3, 128, 128, 3), (2, 256, 64, 1), (2, 64, 256, 1)])
@pytest.mark.parametrize("decay", [False, True])
def test_strong_decays_and_restarts_on_tensor_cores(H, N, P, G, decay):
    """Decays of zero and far below the smallest float within a block of 32 tokens, where the kernels
    take a power for each pair in the place of two factors."""
    d, bounds = make(2, 2 * 270, H, N, P, G, decay=decay, strong=True, seed=71)
    dout, dstate = gradients_of(d, 2, 72)
    got = run(d, bounds, ragged=False, dout=dout, dstate=dstate)
    check_all(d, bounds, got, dout, dstate)
    if decay:
        assert (d["decay"] == 0).any() and (got[2]["dlog_decay"][d["decay"] == 0] == 0).all()


# ------------------------------------------------------------------------------- inputs and requests
@pytest.mark.parametrize("n,tokens,H,N,P", [(3, 9, 2, 64, 64), (1, 270, 3, 32, 32), (2, 600, 2, 64, 64), (2, 300, 2, 256, 128)])
def test_dt_beside_a_given_decay(n, tokens, H, N, P):
    """dt weights the tokens and the decay is given: ddt has no way through exp(dt A)."""
    d, bounds = make(n, tokens, H, N, P, 1, decay=True, seed=91)
    d["dt"] = torch.nn.functional.softplus(torch.randn(tokens, H, generator=torch.Generator().manual_seed(92)) - 1)
    dout, dstate = gradients_of(d, n, 93)
    out, state, got = run(d, bounds, ragged=False, dout=dout, dstate=dstate)
    check_forward(d, bounds, out, state)
    want = reference_grads(d, bounds, dout, dstate)
    v = dbl(d)
    v["dt"].requires_grad_()
    o, f = scan64(**v, bounds=bounds)
    want["ddt"], = torch.autograd.grad((o * dout.double()).sum() + (f * dstate.double()).sum(), [v["dt"]])
    check_backward(d, bounds, got, want)


@pytest.mark.parametrize("H,N,P", [(3, 32, 32), (2, 64, 64), (2, 256, 64)])
def test_each_gradient_by_itself(H, N, P):
    """What is asked for does not depend on what else is."""
    d, bounds = make(2, 2 * 150, H, N, P, 1, seed=95)
    dout, dstate = gradients_of(d, 2, 96)
    all_of = run(d, bounds, ragged=False, dout=dout, dstate=dstate)[2]
    c, s = cuda(d), shape(d, 2)
    for name, want in all_of.items():
        t = torch.full(want.shape, 7.0, dtype=want.dtype, device="cuda")
        s.backward(inputs(c), dout.cuda(), rsq.scan_grads(**{name: t}), state_in=c["state_in"], dstate_out=dstate.cuda(),
                   workspace=poison(s.alloc_workspace(backward=True)))
        assert torch.equal(t.cpu(), want), name


def test_segments_of_a_ragged_batch_in_a_graph():
    """Captured once, replayed on other inputs and other bounds."""
    n, H, N, P = len(SEGMENTED) - 1, 2, 64, 64
    d, bounds = make(n, ROWS, H, N, P, 1, bounds=SEGMENTED, seed=97)
    e, other = make(n, ROWS, H, N, P, 1, bounds=[0, 12, 4700, 4700, 4701, 9700], seed=98)
    c, s = cuda(d), rsq.Scan(n, ROWS, H, N, P, ragged=True)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    out, state, ws = torch.full_like(c["x"], 7.0), c["state_in"].clone(), poison(s.alloc_workspace())

    def call():
        s.forward(inputs(c), out, state_in=state, state_out=state, cu_seqlens=cu, workspace=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k, v in cuda(e).items():
        if v is not None:
            c[k].copy_(v)
    cu.copy_(torch.tensor(other, dtype=torch.int32))
    state.copy_(c["state_in"])
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    rsq.rsq_scan_check(ws)
    check_forward(e, other, out.cpu(), state.cpu())


@pytest.mark.parametrize("N,P", [(32, 32), (64, 64), (256, 64)])
def test_no_gradient_of_a_restart_beside_a_nan(N, P):
    """A decay of zero has no gradient, whatever stands on the other side of it.  A token's x is in the
    gradients of the decays behind it, so those of 41 to 49 are no numbers."""
    d, bounds = make(1, 300, 2, N, P, 1, decay=True, seed=99)
    d["decay"][50] = 0.0
    d["x"][40] = float("nan")
    dout, dstate = gradients_of(d, 1, 100)
    dlog = run(d, bounds, ragged=False, dout=dout, dstate=dstate)[2]["dlog_decay"]
    assert (dlog[50] == 0).all() and torch.isnan(dlog[41:50]).any()


# ------------------------------------------------------------------------------------------ failure mark
@pytest.mark.parametrize("tokens", [0, 2, 24])
def test_a_call_of_single_tokens_clears_the_mark_of_a_workspace_that_it_is_given(tokens):
    """rsq_scan_check speaks of the last call with the workspace; one that needs none is a call too."""
    d, bounds = make(2, tokens, 2, 64, 64, 1, seed=81)
    s, c = shape(d, 2), cuda(d)
    assert s.alloc_workspace() is None
    ws = torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")   # as an earlier call, or nobody, left it
    out, state = torch.empty_like(c["x"]), torch.empty_like(c["state_in"])
    s.forward(inputs(c), out, state_in=c["state_in"], state_out=state, workspace=ws)
    rsq.rsq_scan_check(ws)
    check_forward(d, bounds, out.cpu(), state.cpu()) if tokens else None
    assert torch.equal(ws[4:], torch.full_like(ws[4:], 255))
