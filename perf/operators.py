"""Cases and plain forms of the selective scan with its short convolution, and of the block norm.

The operators, with u the scan's input, d = softplus(dt + dt_bias) and group g = c / (D / G):

    scan      h_t[c,:] = exp(d_t[c] A[c,:]) h_{t-1}[c,:] + d_t[c] u_t[c] B_t[g,:]
              y_t[c] = (h_t[c,:] . C_t[g,:] + D[c] u_t[c]) silu(z_t[c])
    conv      y_t[c] = silu(bias[c] + sum_k w[c,k] x_{t-(W-1)+k}[c]), x before the first token from a carried state
    norm      r' = r + scale gate (o / rms(o)) w_post,   n = (r' / rms(r')) w_pre

each for prompts, for single tokens where that differs, and with its gradients.  `run` computes them
with elementary torch operations, or, where `own` is true, through this package's public calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # a batch of prompts through one layer, every option on: the size at which throughput counts
        dict(name="scan_prompts", op="scan", type="bf16", B=8, L=4096, D=4096, N=16, G=1, z=True, h0=False, ragged=False),
        # one long document continued from a carried state: too few channels to fill the card without cutting the sequence
        dict(name="scan_long", op="scan", type="bf16", B=1, L=16384, D=2048, N=16, G=1, z=True, h0=True, ragged=False),
        # a few short prompts of unequal lengths (one of them empty) in 32 bits, odd sizes, two groups of B and C
        dict(name="scan_ragged", op="scan", type="f32", B=3, L=517, D=202, N=12, G=2, z=False, h0=True, ragged=True),
        # the gradients of a training step's layer
        dict(name="scan_grad", op="scan_bwd", type="bf16", B=4, L=2048, D=4096, N=16, G=1, z=True, h0=False, ragged=False),
        # the gradients of a small model in 32 bits, odd sizes, no gate, with the carried state's gradient
        dict(name="scan_grad_small", op="scan_bwd", type="f32", B=2, L=333, D=328, N=8, G=1, z=False, h0=True, ragged=False),
        # one token of one sequence: latency
        dict(name="step_one", op="scan_step", type="bf16", B=1, L=1, D=2048, N=16, G=1, z=True),
        # one token of each of many sequences, their states in a shared pool: the state's bytes count
        dict(name="step_many", op="scan_step", type="f16", B=256, L=1, D=8192, N=16, G=1, z=True),
        # the convolution in front of the scan over prompts that continue earlier ones
        dict(name="conv_prompts", op="conv", type="bf16", B=2, L=8192, D=8192, W=4, h0=True, ragged=False),
        # the convolution's gradients in a training step
        dict(name="conv_grad", op="conv_bwd", type="bf16", B=4, L=2048, D=4096, W=4, h0=False, ragged=False),
        # the convolution of one token of each of many sequences
        dict(name="conv_step", op="conv_step", type="f16", B=64, L=1, D=8192, W=4),
        # the end of a block and the norm before the next over a batch of prompts; a gate per sequence, the stream in 32 bits
        dict(name="norm_prompts", op="norm", type="bf16", stream="f32", B=8, L=4096, D=2048, gate="sequence"),
        # its gradients in a training step; a gate per token
        dict(name="norm_grad", op="norm_bwd", type="bf16", stream="bf16", B=4, L=2048, D=2048, gate="token"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_bwd", "scan_bwd", "scan_step", "conv", "conv_bwd", "conv_step", "norm", "norm_bwd"])
    case = dict(op=op, type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op.endswith("_step"):
        case.update(B=_spread(rng, 1, 256), L=1, D=_spread(rng, 64, 8192))
    else:
        case.update(B=_spread(rng, 1, 8), L=_spread(rng, 1, 16384), D=_spread(rng, 64, 8192))
    if op.startswith("scan"):
        case.update(N=rng.choice([4, 8, 12, 16, 16, 16, 24, 32, 64]), G=rng.choice([1, 1, 2]), z=rng.random() < 0.6)
        case["D"] += case["D"] % case["G"]
        most = {"scan": 8 * 4096 * 4096 * 16, "scan_bwd": 4 * 2048 * 4096 * 16, "scan_step": 256 * 8192 * 16}[op]
        one = case["D"] * case["N"]
    else:
        if op.startswith("conv"):
            case["W"] = rng.choice([2, 3, 4, 4, 4])
        else:
            case.update(stream=rng.choice(["f32", case["type"]]), gate=rng.choice(["none", "sequence", "token"]))
        most = {"conv": 2 * 8192 * 8192, "conv_bwd": 4 * 2048 * 4096, "conv_step": 64 * 8192,
                "norm": 8 * 4096 * 2048, "norm_bwd": 4 * 2048 * 2048}[op]
        one = case["D"]
    if op.endswith("_step"):  # fewer sequences, or shorter ones, where the case would cost more than the largest listed one
        case["B"] = max(1, min(case["B"], most // one))
    else:
        case["L"] = max(1, min(case["L"], most // (one * case["B"])))
    if op in ("scan", "scan_bwd", "conv", "conv_bwd"):
        case.update(h0=rng.random() < 0.5, ragged=rng.random() < 0.3)
    return case


def work(case):
    B, L, D = case["B"], case["L"], case["D"]
    s, n = (2 if case["type"] != "f32" else 4), B * L * D
    if case["op"].startswith("scan"):
        N, bc, st = case["N"], 2 * B * L * case["G"] * case["N"] * s, 4 * B * D * case["N"]
        z, par = int(case["z"]), 4 * D * (case["N"] + 2)
        # per state element: the decay's product and exponential, the input's product and sum, the output's product and sum
        if case["op"] == "scan_step":
            return {"bytes": n * s * (3 + z) + bc + 2 * st + par, "flops": 7 * n * N}
        h0 = int(case["h0"])
        if case["op"] == "scan":
            return {"bytes": n * s * (3 + z) + bc + st * (1 + h0) + par, "flops": 7 * n * N}
        # u, dt, z, dy read, du, ddt, dz written; B, C read, dB, dC written; the states' gradients; 22 operations a state element
        return {"bytes": n * s * (5 + 2 * z) + 2 * bc + 3 * st * h0 + 2 * par, "flops": 22 * n * N}
    if case["op"].startswith("conv"):
        W = case["W"]
        st, par = B * (W - 1) * D * s, 4 * D * (W + 1)
        if case["op"] == "conv_step":
            return {"bytes": 2 * n * s + 2 * st + par, "flops": n * (2 * W + 4)}
        h0 = int(case["h0"])
        if case["op"] == "conv":
            return {"bytes": 2 * n * s + st * (1 + h0) + par, "flops": n * (2 * W + 4)}
        return {"bytes": 3 * n * s + 3 * st * h0 + 2 * par, "flops": n * (6 * W + 10)}
    q = 2 if case["stream"] != "f32" else 4
    gate = {"none": 0, "sequence": B * D * s, "token": n * s}[case["gate"]]
    if case["op"] == "norm":  # o, r, gate read; n, r' written
        return {"bytes": n * (2 * s + 2 * q) + gate + 12 * D, "flops": 11 * n}
    return {"bytes": n * (3 * s + 3 * q) + 2 * gate + 24 * D, "flops": 30 * n}


# ---- inputs --------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, L, D, t = case["B"], case["L"], case["D"], TYPES[case["type"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    st = dict(case=case)
    f32 = torch.float32
    step = case["op"].endswith("_step")
    rows = (B,) if step else (B, L)
    if case["op"].startswith("scan"):
        N, G = case["N"], case["G"]
        st["x"] = torch.nn.functional.silu(normal(*rows, D, dtype=f32)).to(t)
        st["dt"] = normal(*rows, D, scale=0.5)
        d = torch.exp(math.log(1e-3) + uniform(D) * math.log(100.0))  # steps of 0.001 to 0.1
        st["dt_bias"] = d + torch.log(-torch.expm1(-d))
        st["A"] = -(torch.arange(1, N + 1, device="cuda") * (0.75 + 0.5 * uniform(D, N)))
        st["Bm"], st["Cm"] = normal(*rows, G, N), normal(*rows, G, N)
        st["D"] = 1.0 + 0.1 * normal(D, dtype=f32)
        st["z"] = normal(*rows, D) if case["z"] else None
        if step:
            st["state"] = normal(B, D, N, scale=0.3, dtype=f32)
            st["state_out"] = torch.empty_like(st["state"])
            st["slots"] = torch.randperm(B, generator=gen, device="cuda").to(torch.int32)
        else:
            st["h0"] = normal(B, D, N, scale=0.3, dtype=f32) if case["h0"] else None
        if case["op"] == "scan_bwd":
            st["dy"] = normal(B, L, D)
            st["dfinal"] = normal(B, D, N, dtype=f32) if case["h0"] else None
    elif case["op"].startswith("conv"):
        W = case["W"]
        st["x"] = normal(*rows, D)
        st["w"], st["bias"] = normal(D, W, scale=W ** -0.5, dtype=f32), normal(D, scale=0.1, dtype=f32)
        if step:
            st["state"] = normal(B, W - 1, D)
            st["state_out"] = torch.empty_like(st["state"])
            st["slots"] = torch.randperm(B, generator=gen, device="cuda").to(torch.int32)
        else:
            st["h0"] = normal(B, W - 1, D) if case["h0"] else None
        if case["op"] == "conv_bwd":
            st["dy"] = normal(B, L, D)
            st["dfinal"] = normal(B, W - 1, D) if case["h0"] else None
    else:
        q = TYPES[case["stream"]]
        st["o"], st["w_post"], st["w_pre"] = normal(B, L, D), 1.0 + 0.1 * normal(D, dtype=f32), 1.0 + 0.1 * normal(D, dtype=f32)
        st["scale"] = 0.5 + 0.1 * normal(D, dtype=f32)
        st["gate"] = None if case["gate"] == "none" else normal(*((B, D) if case["gate"] == "sequence" else (B, L, D)))
        st["r"] = normal(B, L, D, scale=2.0, dtype=q)
        if case["op"] == "norm_bwd":  # the stream after the block, as the forward leaves it, and the gradients from above
            st["r_out"] = _norm(st)[1]
            st["dn"], st["dr_out"] = normal(B, L, D), normal(B, L, D, dtype=q)
    st["lengths"] = None
    if case.get("ragged"):
        lengths = (uniform(B) * (L + 1)).to(torch.int32).clamp_(max=L)
        lengths[0] = L
        if B > 2:
            lengths[1] = 0
        st["lengths"] = lengths
    return st


# ---- plain forms ---------------------------------------------------------------------------------

def _scan_up(a, b):
    """h_t = a_t h_{t-1} + b_t from h = 0 along dimension 1, in log2(L) doublings."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])], 1)
        if 2 * k < a.shape[1]:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _live(st):
    """[B,L,1]: 1 on a row's tokens, 0 on its padding."""
    B, L = st["x"].shape[:2]
    if st["lengths"] is None:
        return torch.ones((B, L, 1), device="cuda")
    return (torch.arange(L, device="cuda")[None, :] < st["lengths"][:, None]).float()[:, :, None]


def _per_channel(m, D):
    """[..., G, N] to [..., D, N]: the group of each channel."""
    G, N = m.shape[-2:]
    return m.float()[..., :, None, :].expand(*m.shape[:-1], D // G, N).reshape(*m.shape[:-2], D, N)


def _states(st):
    """What both directions need: u, d, the decays, every state, the mask."""
    live = _live(st)
    u = torch.where(live > 0, st["x"].float(), 0.0)
    raw = st["dt"].float() + st["dt_bias"]
    d = torch.nn.functional.softplus(raw, threshold=40.0) * live
    a = torch.exp(d[..., None] * st["A"])
    b = (d * u)[..., None] * _per_channel(st["Bm"], u.shape[-1])
    if st["h0"] is not None:
        b[:, 0] += a[:, 0] * st["h0"]
    return live, u, raw, d, a, _scan_up(a, b)


def _scan(st):
    live, u, _, _, _, h = _states(st)
    s = (h * _per_channel(st["Cm"], u.shape[-1])).sum(-1) + st["D"] * u
    if st["z"] is not None:
        z = st["z"].float()
        s = s * z * torch.sigmoid(z)
    return torch.where(live > 0, s, 0.0).to(st["x"].dtype), h[:, -1].clone()


def _scan_bwd(st):
    live, u, raw, d, a, h = _states(st)
    t, (B, L, D), G = st["x"].dtype, u.shape, st["Bm"].shape[2]
    Bd, Cd = _per_channel(st["Bm"], D), _per_channel(st["Cm"], D)
    dy = torch.where(live > 0, st["dy"].float(), 0.0)
    out = {}
    ds = dy
    if st["z"] is not None:
        z = st["z"].float()
        sig = torch.sigmoid(z)
        s = (h * Cd).sum(-1) + st["D"] * u
        out["dz"] = (dy * s * sig * (1 + z * (1 - sig))).to(t)
        ds = dy * z * sig
    # the adjoint states, by the same scan over the reversed tokens
    carry = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1)
    e = ds[..., None] * Cd
    if st["dfinal"] is not None:
        e[:, -1] += st["dfinal"]
    q = _scan_up(carry, e.flip(1)).flip(1)
    before = torch.cat([(st["h0"] if st["h0"] is not None else torch.zeros_like(h[:, 0]))[:, None], h[:, :-1]], 1)
    qa = q * before * a
    qb = (q * Bd).sum(-1)
    dd = (qb * u + (qa * st["A"]).sum(-1)) * live * torch.sigmoid(raw)
    out["dx"] = torch.where(live > 0, qb * d + ds * st["D"], 0.0).to(t)
    out["ddt"] = dd.to(t)
    out["dA"] = (qa * d[..., None]).sum((0, 1))
    out["dB"] = (q * (d * u)[..., None]).reshape(B, L, G, D // G, -1).sum(3).to(t)
    out["dC"] = (h * ds[..., None]).reshape(B, L, G, D // G, -1).sum(3).to(t)
    out["dD"] = (ds * u).sum((0, 1))
    out["ddt_bias"] = dd.sum((0, 1))
    if st["h0"] is not None:
        out["dh0"] = q[:, 0] * a[:, 0]
    return out


def _scan_step(st):
    u, slots = st["x"].float(), st["slots"].long()
    d = torch.nn.functional.softplus(st["dt"].float() + st["dt_bias"], threshold=40.0)
    D = u.shape[-1]
    h = torch.exp(d[..., None] * st["A"]) * st["state"][slots] + (d * u)[..., None] * _per_channel(st["Bm"], D)
    st["state_out"][slots] = h
    y = (h * _per_channel(st["Cm"], D)).sum(-1) + st["D"] * u
    if st["z"] is not None:
        z = st["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(st["x"].dtype), st["state_out"]


def _conv_parts(st):
    """The tokens with the carried ones in front, padding zeroed, and the sums before the SiLU."""
    x, (B, L, D), W = st["x"], st["x"].shape, st["w"].shape[1]
    live = _live(st)
    front = st["h0"].float() if st["h0"] is not None else torch.zeros((B, W - 1, D), device="cuda")
    xs = torch.cat([front, torch.where(live > 0, x.float(), 0.0)], 1)
    return live, xs, st["bias"] + sum(st["w"][:, k] * xs[:, k:k + L] for k in range(W))


def _last_rows(st, rows, W):
    """Of each sequence's rows [B, W-1+L, D], the W-1 that its last token ends."""
    B, n, D = rows.shape
    if st["lengths"] is None:
        return rows[:, n - (W - 1):]
    at = st["lengths"].long()[:, None] + torch.arange(W - 1, device="cuda")
    return torch.gather(rows, 1, at[:, :, None].expand(B, W - 1, D))


def _conv(st):
    live, xs, pre = _conv_parts(st)
    y = torch.where(live > 0, pre * torch.sigmoid(pre), 0.0)
    return y.to(st["x"].dtype), _last_rows(st, xs, st["w"].shape[1]).to(st["x"].dtype)


def _conv_bwd(st):
    live, xs, pre = _conv_parts(st)
    t, (B, L, D), W = st["x"].dtype, st["x"].shape, st["w"].shape[1]
    sig = torch.sigmoid(pre)
    dp = torch.where(live > 0, st["dy"].float(), 0.0) * sig * (1 + pre * (1 - sig))
    dxs = sum(torch.nn.functional.pad(dp * st["w"][:, k], (0, 0, k, W - 1 - k)) for k in range(W))
    if st["dfinal"] is not None:
        ends = torch.full((B,), L, device="cuda") if st["lengths"] is None else st["lengths"].long()
        at = ends[:, None] + torch.arange(W - 1, device="cuda")
        dxs.scatter_add_(1, at[:, :, None].expand(B, W - 1, D), st["dfinal"].float())
    out = {"dx": torch.where(live > 0, dxs[:, W - 1:], 0.0).to(t), "dbias": dp.sum((0, 1)),
           "dw": torch.stack([(dp * xs[:, k:k + L]).sum((0, 1)) for k in range(W)], 1)}
    if st["h0"] is not None:
        out["dh0"] = dxs[:, :W - 1].to(t)
    return out


def _conv_step(st):
    slots = st["slots"].long()
    xs = torch.cat([st["state"][slots], st["x"][:, None]], 1)
    pre = st["bias"] + (xs.float() * st["w"].t()).sum(1)
    st["state_out"][slots] = xs[:, 1:]
    return (pre * torch.sigmoid(pre)).to(st["x"].dtype), st["state_out"]


def _rms(v):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _gate(st):
    if st["gate"] is None:
        return 1.0
    g = st["gate"].float()
    return g if g.dim() == 3 else g[:, None, :]


def _norm(st):
    """(n, r'): the norm is of the rounded r', which is what the next block adds to."""
    r_out = (st["r"].float() + st["scale"] * _gate(st) * _rms(st["o"].float()) * st["w_post"]).to(st["r"].dtype)
    return (_rms(r_out.float()) * st["w_pre"]).to(st["o"].dtype), r_out


def _rms_bwd(v, dv):
    """The gradient of v / rms(v) against dv."""
    inv = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return inv * (dv - v * inv * inv * (v * dv).mean(-1, keepdim=True))


def _norm_bwd(st):
    t, o, r_out, dn, g = st["o"].dtype, st["o"].float(), st["r_out"].float(), st["dn"].float(), _gate(st)
    out = {"dw_pre": (dn * _rms(r_out)).sum((0, 1))}
    dr = st["dr_out"].float() + _rms_bwd(r_out, dn * st["w_pre"])
    hat = _rms(o)
    dp = dr * st["scale"] * g
    out["dr"] = dr.to(st["r"].dtype)
    out["do"] = _rms_bwd(o, dp * st["w_post"]).to(t)
    out["dw_post"] = (dp * hat).sum((0, 1))
    out["dscale"] = (dr * g * hat * st["w_post"]).sum((0, 1))
    if st["gate"] is not None:
        dg = dr * st["scale"] * hat * st["w_post"]
        out["dgate"] = (dg if st["gate"].dim() == 3 else dg.sum(1)).to(t)
    return out


PLAIN = {"scan": _scan, "scan_bwd": _scan_bwd, "scan_step": _scan_step, "conv": _conv, "conv_bwd": _conv_bwd,
         "conv_step": _conv_step, "norm": _norm, "norm_bwd": _norm_bwd}


# ---- the framework's calls -----------------------------------------------------------------------

def _own(op, st):
    import mamba_ssd_chunked_fwd_gb300 as ssd
    if op == "scan":
        return ssd.selective_scan(st["x"], st["dt"], st["A"], st["Bm"], st["Cm"], dt_softplus=True, return_final_state=True,
                                  D=st["D"], z=st["z"], dt_bias=st["dt_bias"], initial_states=st["h0"], lengths=st["lengths"])
    if op == "scan_bwd":
        return ssd.selective_scan_bwd(st["x"], st["dt"], st["A"], st["Bm"], st["Cm"], st["dy"], dt_softplus=True,
                                      dfinal=st["dfinal"], D=st["D"], z=st["z"], dt_bias=st["dt_bias"],
                                      initial_states=st["h0"], lengths=st["lengths"])
    if op == "scan_step":
        y = ssd.selective_scan_step(st["x"], st["dt"], st["A"], st["Bm"], st["Cm"], st["state"], dt_softplus=True,
                                    state_out=st["state_out"], slots=st["slots"], D=st["D"], z=st["z"], dt_bias=st["dt_bias"])
        return y, st["state_out"]
    if op == "conv":
        return ssd.causal_conv1d_carry(st["x"], st["w"], st["bias"], initial_state=st["h0"], lengths=st["lengths"],
                                       return_final_state=True)
    if op == "conv_bwd":
        return ssd.causal_conv1d_bwd(st["x"], st["w"], st["dy"], st["bias"], dfinal=st["dfinal"], initial_state=st["h0"],
                                     lengths=st["lengths"])
    if op == "conv_step":
        y = ssd.causal_conv1d_step(st["x"], st["state"], st["w"], st["bias"], state_out=st["state_out"], slots=st["slots"])
        return y, st["state_out"]
    if op == "norm":
        return ssd.block_norm(st["o"], st["r"], st["w_pre"], w_post=st["w_post"], gate=st["gate"], scale=st["scale"], eps=EPS)
    return ssd.block_norm_bwd(st["dn"], st["dr_out"], st["o"], st["r_out"], st["w_pre"], w_post=st["w_post"], gate=st["gate"],
                              scale=st["scale"], eps=EPS)


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return PLAIN[op](state)


# ---- in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    """The definitions token by token in 64 bits; gradients by differentiating them."""
    st = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op.startswith("scan"):
        return _exact_scan(st, op)
    if op.startswith("conv"):
        return _exact_conv(st, op)
    return _exact_norm(st, op)


def _leaves(st, names):
    kept = {}
    for n in names:
        if st.get(n) is not None:
            kept[n] = st[n] = st[n].detach().requires_grad_(True)
    return kept


def _exact_scan(st, op):
    D, G, N = st["A"].shape[0], st["Bm"].shape[-2], st["A"].shape[1]
    of = torch.arange(D, device="cuda") // (D // G)

    def token(h, x, dt, Bt, Ct):
        d = torch.logaddexp(dt + st["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
        h = torch.exp(d[:, :, None] * st["A"]) * h + (d * x)[:, :, None] * Bt[:, of]
        return h, torch.einsum("bcn,bcn->bc", h, Ct[:, of]) + st["D"] * x

    def gated(y, z):
        return y if z is None else y * z / (1 + torch.exp(-z))

    if op == "scan_step":
        at = st["slots"].long()
        h, y = token(st["state"][at], st["x"], st["dt"], st["Bm"], st["Cm"])
        st["state_out"][at] = h
        return gated(y, st["z"]), st["state_out"]
    grad = op == "scan_bwd"
    leaves = _leaves(st, ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0"]) if grad else {}
    with torch.set_grad_enabled(grad):
        B = st["x"].shape[0]
        h = st["h0"] if st["h0"] is not None else torch.zeros((B, D, N), dtype=torch.float64, device="cuda")
        ys, ends = [], None if st["lengths"] is None else st["lengths"].long()
        for t, (x, dt, Bt, Ct) in enumerate(zip(*(st[k].unbind(1) for k in ("x", "dt", "Bm", "Cm")))):
            new, y = token(h, x, dt, Bt, Ct)
            if ends is not None:
                on = (ends > t)[:, None]
                new, y = torch.where(on[:, :, None], new, h), torch.where(on, y, torch.zeros_like(y))
            h = new
            ys.append(y)
        y = gated(torch.stack(ys, 1), st["z"])
    if not grad:
        return y, h
    names = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias", "h0": "dh0"}
    loss = (y * st["dy"]).sum() + (0 if st["dfinal"] is None else (h * st["dfinal"]).sum())
    return {names[k]: g for k, g in zip(leaves, torch.autograd.grad(loss, list(leaves.values())))}


def _exact_conv(st, op):
    W = st["w"].shape[1]

    def silu(v):
        return v / (1 + torch.exp(-v))

    if op == "conv_step":
        at = st["slots"].long()
        s = st["state"][at]
        y = silu(st["bias"] + torch.einsum("bkc,ck->bc", s, st["w"][:, :-1]) + st["w"][:, -1] * st["x"])
        st["state_out"][at] = torch.cat([s[:, 1:], st["x"][:, None]], 1)
        return y, st["state_out"]
    grad = op == "conv_bwd"
    leaves = _leaves(st, ["x", "w", "bias", "h0"]) if grad else {}
    with torch.set_grad_enabled(grad):
        B, L, D = st["x"].shape
        ys, ends = [], []
        for b in range(B):  # one sequence after another, each as long as it is
            n = L if st["lengths"] is None else int(st["lengths"][b])
            front = st["h0"][b] if st["h0"] is not None else torch.zeros((W - 1, D), dtype=torch.float64, device="cuda")
            xs = torch.cat([front, st["x"][b, :n]], 0)
            y = silu(st["bias"] + torch.einsum("tck,ck->tc", xs.unfold(0, W, 1), st["w"])) if n else xs[:0]
            ys.append(torch.cat([y, torch.zeros((L - n, D), dtype=torch.float64, device="cuda")], 0))
            ends.append(xs[n:])
        y, end = torch.stack(ys), torch.stack(ends)
    if not grad:
        return y, end
    loss = (y * st["dy"]).sum() + (0 if st["dfinal"] is None else (end * st["dfinal"]).sum())
    got = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    out = {"dx": got["x"], "dbias": got["bias"], "dw": got["w"]}
    return out if st["h0"] is None else {**out, "dh0": got["h0"]}


def _exact_norm(st, op):
    def unit(v):
        return v / torch.sqrt(torch.linalg.vecdot(v, v)[..., None] / v.shape[-1] + EPS)

    def gate():
        return 1.0 if st["gate"] is None else st["gate"] if st["gate"].dim() == 3 else st["gate"].unsqueeze(1)

    if op == "norm":
        r_out = st["r"] + st["scale"] * gate() * unit(st["o"]) * st["w_post"]
        return unit(r_out) * st["w_pre"], r_out
    # around the stream that the forward left: r' enters as a value of its own, and the branch as its change
    leaves = _leaves(st, ["o", "w_post", "w_pre", "scale", "gate", "r_out"])
    with torch.enable_grad():
        branch = st["scale"] * gate() * unit(st["o"]) * st["w_post"]
        r_new = st["r_out"] + branch - branch.detach()
        loss = (unit(r_new) * st["w_pre"] * st["dn"]).sum() + (r_new * st["dr_out"]).sum()
        got = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    out = {"dw_pre": got["w_pre"], "dr": got["r_out"], "do": got["o"], "dw_post": got["w_post"], "dscale": got["scale"]}
    return out if st["gate"] is None else {**out, "dgate": got["gate"]}
