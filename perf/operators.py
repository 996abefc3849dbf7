"""Cases of the scan and norm operators: their inputs, plain forms, 64-bit definitions and floors.

Operators: the scan of a scalar-decay layer over whole sequences (prompt and training forward, and one
token per sequence), its backward pass, the gated norm behind the mixer and the residual norm before the
block, both with their gradients.  ``own`` chooses between the framework's kernels and the plain forms.
"""
import math
import random

import numpy as np
import torch

own = False

CHUNK = 64  # chunk of the plain scan


# ---------------------------------------------------------------------------------------------- cases
def _scan(name, op, seqs, tokens, heads, dk, dv, groups, *, ragged=0, decay=False, state=False):
    """ragged: 0 for equal lengths, else the seed of a cut of `tokens` into `seqs` lengths.  decay: the
    decay is given (RetNet style, no dt, no D) instead of dt, A and D.  state: with an initial state."""
    return {"name": name, "op": op, "seqs": seqs, "tokens": tokens, "heads": heads, "dk": dk, "dv": dv,
            "groups": groups, "ragged": ragged, "decay": decay, "state": state}


def _norm(name, op, rows, width, group, *, first=False, x="bf16", side="bf16", scale=False):
    """first: the gate multiplies before the norm.  side: type of the gate, or of the residual stream."""
    return {"name": name, "op": op, "rows": rows, "width": width, "group": group, "first": first, "x": x,
            "side": side, "scale": scale}


def listed():
    return [
        # serving: one token for each of 128 requests on full-precision states (the Mamba-2 decode shape)
        _scan("scan_step_b128", "scan", 128, 128, 80, 128, 64, 1, state=True),
        # prefill of a batch of equal prompts
        _scan("scan_prefill", "scan", 8, 16384, 80, 128, 64, 1),
        # chunked prefill of a ragged batch that continues stored states; retention decays, a key per head
        _scan("scan_ragged", "scan", 29, 7001, 16, 128, 128, 16, ragged=5, decay=True, state=True),
        # one long document: few heads, so the sequence itself has to be split
        _scan("scan_long", "scan", 1, 32768, 16, 128, 128, 16, decay=True),
        # a training step of the layer
        _scan("scan_backward_train", "scan_backward", 4, 8192, 80, 128, 64, 1),
        # fine-tuning on packed documents of uneven length, from given initial states
        _scan("scan_backward_ragged", "scan_backward", 17, 3001, 16, 64, 64, 4, ragged=9, decay=True, state=True),
        # norm behind a Mamba-2 mixer over a prompt, gate before the norm
        _norm("gated_norm_prefill", "gated_norm", 16384, 5120, 5120, first=True),
        # norm behind the decode step's fp32 output, per head, gate after the norm
        _norm("gated_norm_step", "gated_norm", 1024, 2048, 128, x="f32"),
        _norm("gated_norm_backward", "gated_norm_backward", 8192, 5120, 5120, first=True),
        # residual stream of a prompt, and of a handful of requests, where latency counts
        _norm("residual_norm_prefill", "residual_norm", 16384, 2560, 2560, side="f32"),
        _norm("residual_norm_step", "residual_norm", 4, 2560, 2560, side="f32", scale=True),
        _norm("residual_norm_backward", "residual_norm_backward", 8192, 2560, 2560, side="f32", scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "scan_backward", "scan_backward", "gated_norm", "gated_norm_backward",
                     "residual_norm", "residual_norm_backward"])
    if op.startswith("scan"):
        most = 600e6 if op == "scan" else 300e6  # heads * tokens * dk * dv / 16 stays under the listed cases'
        while True:
            seqs = _log(rng, 1, 64)
            groups = rng.choice([1, 1, 2, 4])
            heads = groups * rng.choice([1, 2, 3, 5, 8, 16, 20])
            if rng.random() < 0.3:
                groups = heads
            dk, dv = rng.choice([16, 32, 64, 128, 128, 256]), rng.choice([16, 32, 64, 64, 128, 256])
            tokens = seqs if op == "scan" and rng.random() < 0.25 else seqs * _log(rng, 2, 4096) + rng.randrange(2)
            if heads * tokens * dk * dv / 16 <= most and seqs * heads * dk * dv <= 70e6:
                break
        ragged = rng.randrange(1, 1 << 20) if tokens % seqs or rng.random() < 0.5 else 0
        return _scan(None, op, seqs, tokens, heads, dk, dv, groups, ragged=ragged, decay=rng.random() < 0.4,
                     state=rng.random() < 0.6) | {"name": "drawn"}
    while True:
        width = 8 * _log(rng, 2, 1024) if rng.random() < 0.7 else _log(rng, 16, 8192)
        parts = rng.choice([1, 1, 2, 4, 16]) if op.startswith("gated") else 1
        rows = _log(rng, 1, 30000)
        if width % parts == 0 and rows * width <= 40e6:
            break
    return _norm(None, op, rows, width, width // parts, first=rng.random() < 0.5, x=rng.choice(["bf16", "f32"]),
                 side=rng.choice(["bf16", "f32"]), scale=rng.random() < 0.5) | {"name": "drawn"}


def _bounds(c):
    """The host's list of sequence bounds."""
    n, total = c["seqs"], c["tokens"]
    if not c["ragged"]:
        return [total // n * i for i in range(n + 1)]
    cut = np.random.RandomState(c["ragged"]).randint(0, total + 1, n - 1)
    return [0] + sorted(int(v) for v in cut) + [total]


def work(c):
    if c["op"].startswith("scan"):
        T, H, N, P, G = c["tokens"], c["heads"], c["dk"], c["dv"], c["groups"]
        gates = 4 * T * H
        states = 4 * c["seqs"] * H * N * P
        if c["op"] == "scan":
            return {"bytes": T * H * P * 4 + T * G * N * 4 + gates + states * (2 if c["state"] else 1),
                    "flops": 4.0 * T * H * N * P}
        return {"bytes": T * H * P * 6 + T * G * N * 8 + 2 * gates + states * (3 if c["state"] else 0),
                "flops": 12.0 * T * H * N * P}
    n = c["rows"] * c["width"]
    x, s = (4 if c["x"] == "f32" else 2), (4 if c["side"] == "f32" else 2)
    if c["op"] == "gated_norm":
        return {"bytes": n * (x + s + 2), "flops": 8.0 * n}
    if c["op"] == "gated_norm_backward":
        return {"bytes": n * (2 * x + 2 * s + 2), "flops": 20.0 * n}
    if c["op"] == "residual_norm":
        return {"bytes": n * (x + 2 * s + 2), "flops": 6.0 * n}
    # x is read for the gradient of the scale alone
    return {"bytes": n * ((2 if c["scale"] else 1) * x + 3 * s + 2), "flops": 12.0 * n}


# --------------------------------------------------------------------------------------------- inputs
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    f32 = torch.float32
    s = {"case": c}
    if c["op"].startswith("scan"):
        T, H, N, P, G, n = c["tokens"], c["heads"], c["dk"], c["dv"], c["groups"], c["seqs"]
        s["x"] = normal(T, H, P)
        s["Bm"], s["Cm"] = normal(T, G, N), normal(T, G, N)
        if c["decay"]:
            s["Bm"] = torch.nn.functional.normalize(s["Bm"].float(), dim=-1).to(torch.bfloat16)
            s["dt"] = s["A"] = s["D"] = None
            gamma = 1 - 2.0 ** -torch.linspace(3, 9, H, device="cuda")
            s["decay"] = (gamma + 0.02 * (torch.rand(T, H, generator=g, device="cuda") - 0.9)).clamp(0.5, 1.0)
        else:
            s["dt"] = torch.nn.functional.softplus(normal(T, H, dtype=f32, mean=-2.0))
            s["A"] = -torch.exp(2.8 * torch.rand(H, generator=g, device="cuda"))
            s["D"] = normal(H, dtype=f32, std=0.1, mean=1.0)
            s["decay"] = None
        s["state_in"] = normal(n, H, N, P, dtype=f32) if c["state"] else None
        s["bounds"] = torch.tensor(_bounds(c), dtype=torch.int32, device="cuda")
        s["longest"] = max(b - a for a, b in zip(_bounds(c), _bounds(c)[1:]))
        if c["op"] == "scan_backward":
            s["dout"] = normal(T, H, P)
            s["dstate_out"] = normal(n, H, N, P, dtype=f32, std=0.1) if c["state"] else None
        return s
    R, W = c["rows"], c["width"]
    s["w"] = normal(W, dtype=f32, std=0.2, mean=1.0)
    s["x"] = normal(R, W, dtype=_dtype(c["x"]), std=1.5)
    s["side"] = normal(R, W, dtype=_dtype(c["side"]))
    s["scale"] = normal(W, dtype=f32, std=0.1, mean=0.7) if c["scale"] else None
    if c["op"].endswith("backward"):
        s["dy"] = normal(R, W)
        if c["op"] == "residual_norm_backward":
            s["dh"] = normal(R, W, dtype=_dtype(c["side"]))
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _padded(bounds, longest):
    """Token index and validity of place t of every sequence, padded to whole chunks."""
    length = -(-max(longest, 1) // CHUNK) * CHUNK
    at = bounds[:-1, None].long() + torch.arange(length, device=bounds.device)
    ok = at < bounds[1:, None]
    return torch.where(ok, at, torch.zeros_like(at)), ok


def _plain_scan(x, Bm, Cm, dt, log_a, D, state, bounds, longest):
    """x [T,H,P], Bm, Cm [T,G,N], dt [T,H] or None, log_a [T,H] float64, all differentiable float32:
    outputs in chunks, the states between chunks by the matrix of decays between them."""
    T, H, P = x.shape
    per = H // Bm.shape[1]
    at, ok = _padded(bounds, longest)
    n, length = at.shape
    m = ok[..., None]
    xs = (x[at] * m[..., None]).view(n, -1, CHUNK, H, P).transpose(2, 3)
    k = (Bm[at] * m[..., None]).view(n, -1, CHUNK, *Bm.shape[1:]).transpose(2, 3)
    q = Cm[at].view(n, -1, CHUNK, *Cm.shape[1:]).transpose(2, 3)
    b = (log_a[at] * m).view(n, -1, CHUNK, H).transpose(2, 3).cumsum(-1)
    u = xs if dt is None else xs * (dt[at] * m).view(n, -1, CHUNK, H).transpose(2, 3)[..., None]
    keep = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    between = torch.where(keep, b[..., :, None] - b[..., None, :], float("-inf")).exp().float()
    y = ((q @ k.transpose(-1, -2)).repeat_interleave(per, 2) * between) @ u
    k, q = k.repeat_interleave(per, 2), q.repeat_interleave(per, 2)
    local = (k * (b[..., -1:] - b).exp().float()[..., None]).transpose(-1, -2) @ u  # [n,c,H,N,P]
    first = torch.zeros_like(local[:, :1]) if state is None else state[:, None]
    parts = torch.cat([first, local], 1).transpose(1, 2).flatten(3)                # [n,H,c+1,N*P]
    end = torch.cat([torch.zeros_like(b[:, :1, :, -1]), b[..., -1]], 1).cumsum(1).transpose(1, 2)
    c1 = end.shape[-1]
    keep = torch.ones(c1, c1, dtype=torch.bool, device=x.device).tril()
    hops = torch.where(keep, end[..., :, None] - end[..., None, :], float("-inf")).exp().float()
    states = (hops @ parts).view(n, H, c1, *local.shape[-2:]).transpose(1, 2)
    y = y + b.exp().float()[..., None] * (q @ states[:, :-1])
    y = y if D is None else y + D[:, None, None] * xs
    y = y.transpose(2, 3).reshape(n, length, H, P)
    out = x.new_zeros(T, H, P).index_put((at[ok],), y[ok])
    return out, states[:, -1]


def _leaf(t):
    return None if t is None else t.float().detach().requires_grad_()


def _plain(s):
    c = s["case"]
    if c["op"] == "scan":
        f = {k: None if s[k] is None else s[k].float() for k in ("x", "Bm", "Cm", "dt", "A", "D", "decay")}
        log_a = f["decay"].double().log() if c["decay"] else f["dt"].double() * f["A"].double()
        y, state = _plain_scan(f["x"], f["Bm"], f["Cm"], f["dt"], log_a, f["D"], s["state_in"], s["bounds"], s["longest"])
        return {"out": y.bfloat16(), "state": state}
    if c["op"] == "scan_backward":
        f = {k: _leaf(s[k]) for k in ("x", "Bm", "Cm", "dt", "A", "D", "state_in")}
        if c["decay"]:
            log_a = s["decay"].double().log().requires_grad_()
        else:
            log_a = f["dt"].double() * f["A"].double()
        y, state = _plain_scan(f["x"], f["Bm"], f["Cm"], f["dt"], log_a, f["D"], f["state_in"], s["bounds"], s["longest"])
        names = ["x", "Bm", "Cm"] + ([] if c["decay"] else ["dt", "A", "D"]) + (["state_in"] if c["state"] else [])
        leaves = [f[k] for k in names] + ([log_a] if c["decay"] else [])
        outs = [y] + ([state] if c["state"] else [])
        grads = torch.autograd.grad(outs, leaves, [s["dout"].float()] + ([s["dstate_out"]] if c["state"] else []))
        got = dict(zip(names + (["log_decay"] if c["decay"] else []), grads))
        return {"d" + k: v.bfloat16() if k in ("x", "Bm", "Cm") else v.float() for k, v in got.items()}
    x, side, w, group = s["x"].float(), s["side"].float(), s["w"], c["group"]
    back = c["op"].endswith("backward")
    if c["op"].startswith("gated"):
        leaves = [t.detach().requires_grad_() for t in (x, side, w)] if back else [x, side, w]
        y = _plain_gated(*leaves, group, c["first"])
        if not back:
            return {"y": y.bfloat16()}
        dx, dz, dw = torch.autograd.grad(y, leaves, s["dy"].float())
        return {"dx": dx.to(s["x"].dtype), "dz": dz.to(s["side"].dtype), "dw": dw}
    if not back:
        h = (side + (x if s["scale"] is None else x * s["scale"])).to(s["side"].dtype)
        return {"h": h, "y": _plain_norm(h.float(), w).bfloat16()}
    # the backward pass has the forward's h: here `side`
    h, w = side.detach().requires_grad_(), w.detach().requires_grad_()
    dh, dw = torch.autograd.grad(_plain_norm(h, w), [h, w], s["dy"].float())
    dh = dh + s["dh"].float()
    got = {"dresidual": dh.to(s["side"].dtype), "dw": dw,
           "dx": (dh if s["scale"] is None else dh * s["scale"]).to(s["x"].dtype)}
    if s["scale"] is not None:
        got["dscale"] = (dh * x).sum(0)
    return got


def _plain_norm(u, w):
    return u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-5) * w


def _plain_gated(x, z, w, group, first):
    z = z * torch.sigmoid(z)
    u = (x * z if first else x).unflatten(-1, (-1, group))
    y = _plain_norm(u, w.view(-1, group)).flatten(-2)
    return y if first else y * z


# ------------------------------------------------------------------------------ the framework's calls
def _own(s):
    import ssm_decode_02_b200 as rsq
    c = s["case"]
    new = torch.empty_like
    if c["op"].startswith("scan"):
        back = c["op"] == "scan_backward"
        if "scan" not in s:  # the handle and the workspace that a program keeps
            s["scan"] = rsq.Scan(c["seqs"], c["tokens"], c["heads"], c["dk"], c["dv"], ngroups=c["groups"],
                                 ragged=bool(c["ragged"]))
            s["workspace"] = s["scan"].alloc_workspace(backward=back)
        cu = s["bounds"] if c["ragged"] else None
        ins = rsq.scan_inputs(s["x"], s["Bm"], s["Cm"], s["dt"], s["A"], s["D"], s["decay"])
        if not back:
            out = new(s["x"])
            state = torch.empty((c["seqs"], c["heads"], c["dk"], c["dv"]), dtype=torch.float32, device="cuda")
            s["scan"].forward(ins, out, state_in=s["state_in"], state_out=state, cu_seqlens=cu, workspace=s["workspace"])
            return {"out": out, "state": state}
        got = {"dx": new(s["x"]), "dBm": new(s["Bm"]), "dCm": new(s["Cm"])}
        if c["decay"]:
            got["dlog_decay"] = new(s["decay"])
        else:
            got |= {"ddt": new(s["dt"]), "dA": new(s["A"]), "dD": new(s["D"])}
        if c["state"]:
            got["dstate_in"] = new(s["state_in"])
        s["scan"].backward(ins, s["dout"], rsq.scan_grads(**got), state_in=s["state_in"], dstate_out=s["dstate_out"],
                           cu_seqlens=cu, workspace=s["workspace"])
        return got
    cfg = rsq.norm_config(s["x"], s["side"], torch.bfloat16, group=c["group"], eps=1e-5,
                          order=rsq.RSQ_GATE_NORM if c["first"] else rsq.RSQ_NORM_GATE)
    if c["op"].endswith("backward") and "workspace" not in s:
        s["workspace"] = torch.empty(rsq.rsq_norm_workspace(cfg), dtype=torch.uint8, device="cuda")
    x, side, w = s["x"], s["side"], s["w"]
    if c["op"] == "gated_norm":
        y = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        rsq.rsq_gated_norm(cfg, x, side, w, y)
        return {"y": y}
    if c["op"] == "gated_norm_backward":
        got = {"dx": new(x), "dz": new(side), "dw": new(w)}
        rsq.rsq_gated_norm_backward(cfg, x, side, w, s["dy"], got["dx"], got["dz"], got["dw"], s["workspace"])
        return got
    if c["op"] == "residual_norm":
        got = {"h": new(side), "y": torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")}
        rsq.rsq_residual_norm(cfg, x, side, s["scale"], w, got["h"], got["y"])
        return got
    got = {"dresidual": new(side), "dw": new(w), "dx": new(x)}
    if s["scale"] is not None:
        got["dscale"] = new(s["scale"])
    rsq.rsq_residual_norm_backward(cfg, x, side, s["scale"], w, s["dy"], s["dh"], got["dx"], got["dresidual"],
                                   got.get("dscale"), got["dw"], s["workspace"])
    return got


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------------------------ 64-bit definitions
def _exact_scan(c, s):
    """The recurrence token by token, all sequences side by side; backward by the reverse recurrence."""
    lo, hi = s["bounds"][:-1].long(), s["bounds"][1:].long()
    per = c["heads"] // c["groups"]
    d = {k: s[k].double() for k in ("x", "Bm", "Cm", "dt", "A", "D", "decay", "state_in", "dout", "dstate_out")
         if s.get(k) is not None}
    T, H, P = s["x"].shape
    N, n = c["dk"], c["seqs"]
    a = d["decay"] if c["decay"] else torch.exp(d["dt"] * d["A"])
    dt = d.get("dt", torch.ones_like(a))
    zero = torch.zeros(n, H, N, P, dtype=torch.float64, device="cuda")
    S = d.get("state_in", zero).clone()

    def heads(t):
        return t.repeat_interleave(per, 1)

    out = torch.zeros_like(d["x"])
    dq = torch.zeros(T, H, N, dtype=torch.float64, device="cuda")
    back = c["op"] == "scan_backward"
    order = torch.argsort(hi - lo, descending=True)  # longest first: the live sequences are a prefix
    lens = (hi - lo)[order].tolist()
    live = sum(v > 0 for v in lens)
    S = S[order]
    for t in range(max(lens)):
        while live and lens[live - 1] <= t:
            live -= 1
        i = lo[order[:live]] + t
        k, q, x = heads(d["Bm"][i]), heads(d["Cm"][i]), d["x"][i]
        S[:live] *= a[i][..., None, None]
        S[:live] += (dt[i][..., None] * k)[..., None] * x[..., None, :]
        if back:
            dq[i] = (S[:live] @ d["dout"][i][..., None])[..., 0]
        else:
            out[i] = (q[..., None, :] @ S[:live])[..., 0, :] + (0 if "D" not in d else d["D"][:, None] * x)
    final = torch.empty_like(S)
    final[order] = S
    if not back:
        return {"out": out, "state": final}
    R = d.get("dstate_out", zero).clone()
    total = (final * R).sum((-1, -2))
    R = R[order]
    dk, du = torch.zeros_like(dq), torch.zeros_like(d["x"])
    da_next = torch.ones(n, H, dtype=torch.float64, device="cuda")
    live = 0
    for t in range(max(lens) - 1, -1, -1):
        while live < n and lens[live] > t:
            live += 1
        i = lo[order[:live]] + t
        k, q, x, dy = heads(d["Bm"][i]), heads(d["Cm"][i]), d["x"][i], d["dout"][i]
        R[:live] *= da_next[:live, :, None, None]
        R[:live] += q[..., None] * dy[..., None, :]
        du[i] = (k[..., None, :] @ R[:live])[..., 0, :]
        dk[i] = dt[i][..., None] * (R[:live] @ x[..., None])[..., 0]
        da_next[:live] = a[i]
    dstate = torch.empty_like(R)
    empty = torch.tensor([v == 0 for v in lens], device="cuda")
    dstate[order] = R * torch.where(empty[:, None], torch.ones_like(da_next), da_next)[..., None, None]
    # a decay scales what earlier tokens (and the initial state) give to later outputs and the final state
    k, q = heads(d["Bm"]), heads(d["Cm"])
    part = (q * dq).sum(-1) - (k * dk).sum(-1)
    run_sum = part.flip(0).cumsum(0).flip(0)
    run_sum = torch.cat([run_sum, torch.zeros_like(run_sum[:1])])
    at = torch.arange(T, device="cuda")
    seq = (torch.searchsorted(hi, at, right=True)).clamp(max=n - 1)
    dlog = run_sum[:-1] - run_sum[hi[seq]] + total[seq]
    group = lambda t: t.view(T, c["groups"], per, N).sum(2)  # noqa: E731
    got = {"dx": dt[..., None] * du + (d["D"][:, None] * d["dout"] if "D" in d else 0), "dBm": group(dk), "dCm": group(dq)}
    if c["decay"]:
        got["dlog_decay"] = dlog
    else:
        got |= {"ddt": (d["x"] * du).sum(-1) + d["A"] * dlog, "dA": (dt * dlog).sum(0),
                "dD": (d["x"] * d["dout"]).sum((0, 2))}
    if c["state"]:
        got["dstate_in"] = dstate
    return got


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"].startswith("scan"):
        return _exact_scan(c, s)
    x, side, w = s["x"].double(), s["side"].double(), s["w"].double()
    R, W, m = c["rows"], c["width"], c["group"]

    def inv(v):
        return 1 / (v.view(R, -1, m).pow(2).sum(-1, keepdim=True) / m + 1e-5).sqrt()

    def wide(v):
        return v.expand(R, W // m, m).reshape(R, W)

    if c["op"] == "residual_norm":
        h = side + x * (1 if s["scale"] is None else s["scale"].double())
        kept = h.to(s["side"].dtype) if s["side"].dtype == torch.float32 else h.float().to(s["side"].dtype)
        return {"h": h, "y": kept.double() * wide(inv(kept.double())) * w}
    if c["op"] == "residual_norm_backward":
        r, dy, n = wide(inv(side)), s["dy"].double(), side * wide(inv(side))
        dh = s["dh"].double() + r * (dy * w - n * (dy * w * n).mean(-1, keepdim=True))
        sc = 1 if s["scale"] is None else s["scale"].double()
        got = {"dresidual": dh, "dw": (dy * n).sum(0), "dx": dh * sc}
        if s["scale"] is not None:
            got["dscale"] = (dh * x).sum(0)
        return got
    sig = 1 / (1 + torch.exp(-side))
    gate = side * sig
    slope = sig * (1 + side * (1 - sig))
    u = x * gate if c["first"] else x
    r = wide(inv(u))
    n = u * r
    if c["op"] == "gated_norm":
        return {"y": n * w * (1 if c["first"] else gate)}
    dy = s["dy"].double()
    dn = dy * w * (1 if c["first"] else gate)
    mean = (dn * n).view(R, -1, m).mean(-1, keepdim=True)
    du = r * (dn - n * wide(mean))
    if c["first"]:
        return {"dx": du * gate, "dz": du * x * slope, "dw": (dy * n).sum(0)}
    return {"dx": du, "dz": dy * n * w * slope, "dw": (dy * n * gate).sum(0)}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(case, work(case))
