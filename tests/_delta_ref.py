"""Plain 64-bit forms of the gated delta rule and of the norm of queries and keys,
token by token on the CPU; gradients by differentiating them."""
import torch


def delta(q, k, v, g, beta, h0=None, lengths=None, scale=None):
    """(y, final state): S' = e^g S, u = beta (v - S' k), S = S' + u k^T, y = scale S q."""
    (B, L, G, N), (H, P) = q.shape, v.shape[2:]
    of = torch.arange(H) // (H // G)
    scale = N ** -0.5 if scale is None else scale
    S = h0 if h0 is not None else torch.zeros((B, H, P, N), dtype=q.dtype)
    ys = []
    for t in range(L):
        kt, qt = k[:, t, of], q[:, t, of]
        new = torch.exp(g[:, t])[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (new * kt[:, :, None]).sum(-1))
        new = new + u[..., None] * kt[:, :, None]
        y = scale * (new * qt[:, :, None]).sum(-1)
        if lengths is not None:
            on = (lengths > t)[:, None, None]
            new, y = torch.where(on[..., None], new, S), torch.where(on, y, torch.zeros_like(y))
        S = new
        ys.append(y)
    return torch.stack(ys, 1), S


def qk_norm(q, k, w_q=None, w_k=None, norm="rms", eps=1e-6, freqs=None, positions=None, interleaved=False):
    if freqs is not None and positions is None:
        positions = torch.arange(q.shape[1]).expand(q.shape[:2])

    def one(x, w):
        sq = (x * x).sum(-1, keepdim=True)
        x = x / torch.sqrt((sq / x.shape[-1] if norm == "rms" else sq) + eps)
        if w is not None:
            x = x * w
        if freqs is None:
            return x
        R = freqs.shape[0]
        angle = positions.to(x.dtype)[..., None, None] * freqs
        c, s = torch.cos(angle), torch.sin(angle)
        a, b = (x[..., 0:2 * R:2], x[..., 1:2 * R:2]) if interleaved else (x[..., :R], x[..., R:2 * R])
        turned = [a * c - b * s, b * c + a * s]
        turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
        return torch.cat([turned, x[..., 2 * R:]], -1)

    return one(q, w_q), one(k, w_k)
