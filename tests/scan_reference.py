"""The scan and the norms from their definitions, in 64 bits on the CPU (torch
double, differentiable), and the error bounds that the tests hold the kernels to.
"""
import torch

U16 = 2.0 ** -8    # half a step of bf16 relative to the value
U32 = 2.0 ** -24   # half a step of binary32


def scan64(x, Bm, Cm, dt=None, A=None, D=None, decay=None, state_in=None, bounds=None):
    """x [T,H,P], Bm, Cm [T,G,N], all double.  Token by token: (out, state_out [n,H,N,P])."""
    T, H, P = x.shape
    per = H // Bm.shape[1]
    N = Bm.shape[2]
    a = decay if decay is not None else torch.exp(dt * A)
    u = x if dt is None else dt[..., None] * x
    rows, finals = [None] * T, []
    zero = torch.zeros(P, dtype=torch.float64)
    for i, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        S = torch.zeros(H, N, P, dtype=torch.float64) if state_in is None else state_in[i]
        for t in range(lo, hi):
            k, q = Bm[t].repeat_interleave(per, 0), Cm[t].repeat_interleave(per, 0)
            S = a[t][:, None, None] * S + k[:, :, None] * u[t][:, None, :]
            rows[t] = (q[:, :, None] * S).sum(1) + (0 if D is None else D[:, None] * x[t])
        finals.append(S)
    out = torch.stack([zero.expand(H, P) if r is None else r for r in rows]) if T else x.clone()
    return out, torch.stack(finals)


def magnitude(x, Bm, Cm, dt=None, A=None, D=None, decay=None, state_in=None, bounds=None):
    """The same sums over absolute values: what rounding errors of the terms add up to at most."""
    f = lambda t: None if t is None else t.abs()  # noqa: E731
    a = decay if decay is not None else torch.exp(dt * A)
    return scan64(f(x), f(Bm), f(Cm), f(dt), None, f(D), a, f(state_in), bounds)


def silu(z):
    return z / (1 + torch.exp(-z))


def norm64(u, w, group, eps):
    v = u.unflatten(-1, (-1, group))
    return (v / (v.pow(2).mean(-1, keepdim=True) + eps).sqrt()).flatten(-2) * w


def gated64(x, z, w, group, eps, gate_first):
    if z is None:
        return norm64(x, w, group, eps)
    return norm64(x * silu(z), w, group, eps) if gate_first else norm64(x, w, group, eps) * silu(z)


def rel(got, want):
    """2-norm of the difference over the 2-norm of the value."""
    got, want = got.double().cpu(), want.double().cpu()
    n = want.norm().item()
    return (got - want).norm().item() / n if n else got.norm().item()
