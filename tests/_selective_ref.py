"""Plain 64-bit forms of the selective scan, its convolution and the block
norm, one token after another, on the CPU; gradients by differentiating them."""
import math

import torch

# A rounding to the type is off by at most half a step relative to the value; fp32
# results are held to the library's fp32 bound (1e-5 of the norm, 1e-4 of the largest).
HALF_STEP = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
REL, MAX = 1e-5, 1e-4


def close(got, ref, what=""):
    got64, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got64.shape == ref.shape, (what, got64.shape, ref.shape)
    assert torch.isfinite(got64).all(), f"{what}: not finite"
    half = HALF_STEP[got.dtype]
    diff, norm = (got64 - ref).norm().item(), ref.norm().item()
    assert diff <= (half + REL) * norm + 1e-30, f"{what}: relative difference {diff / max(norm, 1e-300):.2e}"
    if ref.numel():
        bound = half * ref.abs() + MAX * ref.abs().max()
        assert (got64 - ref).abs().le(bound + 1e-30).all(), f"{what}: largest difference {(got64 - ref).abs().max():.2e}"


def of(t):
    """A 64-bit copy on the CPU (None stays None)."""
    return None if t is None else t.detach().cpu().double()


def step_of(dt, bias, softplus, limit):
    v = dt if bias is None else dt + bias
    if softplus:
        v = torch.logaddexp(v, torch.zeros((), dtype=v.dtype))
    lo, hi = limit
    return v if (lo, hi) == (0.0, math.inf) else v.clamp(lo, hi)


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None, softplus=True, limit=(0.0, math.inf)):
    Bb, L, Dm = x.shape
    G, N = B.shape[2:]
    of_g = torch.arange(Dm) // (Dm // G)
    h = h0 if h0 is not None else torch.zeros((Bb, Dm, N), dtype=x.dtype)
    ys = []
    for t in range(L):
        d = step_of(dt[:, t], dt_bias, softplus, limit)
        new = torch.exp(d[:, :, None] * A) * h + (d * x[:, t])[:, :, None] * B[:, t, of_g]
        y = (new * C[:, t, of_g]).sum(-1)
        if D is not None:
            y = y + D * x[:, t]
        if z is not None:
            y = y * z[:, t] * torch.sigmoid(z[:, t])
        if lengths is not None:
            on = (lengths > t)[:, None]
            new, y = torch.where(on[:, :, None], new, h), torch.where(on, y, torch.zeros_like(y))
        h = new
        ys.append(y)
    return torch.stack(ys, 1), h


def conv(x, w, bias=None, h0=None, lengths=None, silu=True):
    Bb, L, C = x.shape
    W = w.shape[1]
    ys, ends = [], []
    for b in range(Bb):
        n = L if lengths is None else int(lengths[b])
        front = h0[b] if h0 is not None else torch.zeros((W - 1, C), dtype=x.dtype)
        v = torch.cat([front, x[b, :n]], 0)
        rows = []
        for t in range(n):
            a = (w.t() * v[t:t + W]).sum(0)
            a = a if bias is None else a + bias
            rows.append(a * torch.sigmoid(a) if silu else a)
        rows += [torch.zeros(C, dtype=x.dtype)] * (L - n)
        ys.append(torch.stack(rows))
        ends.append(v[n:])
    return torch.stack(ys), torch.stack(ends)


def norm(o, r, w_pre, w_post=None, gate=None, scale=None, eps=1e-5):
    """(n of the unrounded r', r')."""
    if o is not None:
        p = o if w_post is None else o / torch.sqrt((o * o).mean(-1, keepdim=True) + eps) * w_post
        if scale is not None:
            p = p * scale
        if gate is not None:
            p = p * (gate if gate.dim() == r.dim() else gate.reshape(gate.shape[0], *[1] * (r.dim() - 2), gate.shape[1]))
        r = r + p
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w_pre, r


def gradients(f, inputs, outs):
    """Gradients of sum(out * weight) over (out, weight) of f(inputs), for the
    inputs (a dict) that are given."""
    leaves = {k: v.clone().requires_grad_(True) for k, v in inputs.items() if v is not None}
    got = f(**leaves, **{k: None for k, v in inputs.items() if v is None})
    loss = sum((g * w).sum() for g, w in zip(got, outs) if w is not None)
    grads = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return {k: torch.zeros_like(v) if g is None else g for (k, v), g in zip(leaves.items(), grads)}
