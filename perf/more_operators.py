"""Cases and plain forms of the gated delta rule, and of the norm of queries and keys with its rotation.

The operators, for a head h that reads the queries and keys of group h / (H / G), with S a state of P x N:

    delta     S' = exp(g_t) S_{t-1},   u_t = beta_t (v_t - S' k_t),   S_t = S' + u_t k_t^T,   y_t = scale S_t q_t
    norm      x' = rot(x / sqrt(mean(x^2) + eps) * w)       for every head of the queries and of the keys; the sum
              in place of the mean where the norm is that of the vector, and rot turns pair i by position * freqs[i]

the first for prompts, single tokens and with its gradients, the second forward and backward.  `run`
computes them with elementary torch operations, or, where `own` is true, through this package's public calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
C = 64  # tokens of a chunk in the plain form


def listed():
    return [
        # a batch of prompts through one layer, two value heads to each key head: the size at which throughput counts
        dict(name="delta_prompts", op="delta", type="bf16", B=4, L=4096, H=32, G=16, N=128, P=128, h0=False, ragged=False),
        # one long document continued from a carried state: few heads, many tokens
        dict(name="delta_long", op="delta", type="bf16", B=1, L=16384, H=16, G=16, N=128, P=128, h0=True, ragged=False),
        # a few short prompts of unequal lengths (one of them empty) in 32 bits, odd sizes
        dict(name="delta_ragged", op="delta", type="f32", B=3, L=517, H=6, G=3, N=100, P=72, h0=True, ragged=True),
        # the gradients of a training step's layer
        dict(name="delta_grad", op="delta_bwd", type="bf16", B=4, L=2048, H=16, G=16, N=128, P=128, h0=False, ragged=False),
        # the gradients of a small model in 32 bits, odd length, shared keys, with the carried state's gradient
        dict(name="delta_grad_small", op="delta_bwd", type="f32", B=2, L=333, H=6, G=3, N=64, P=64, h0=True, ragged=False),
        # one token of one sequence: latency
        dict(name="delta_step_one", op="delta_step", type="bf16", B=1, L=1, H=16, G=16, N=128, P=128),
        # one token of each of many sequences, their states in a shared pool: the state's bytes count
        dict(name="delta_step_many", op="delta_step", type="f16", B=256, L=1, H=32, G=16, N=128, P=128),
        # queries and keys of a batch of prompts: root mean square with weights, half of each head rotated
        dict(name="norm_prompts", op="norm", type="bf16", B=8, L=4096, H=32, G=8, N=128, kind="rms", w=True, rot=64, interleaved=False),
        # vectors of length one for a delta layer's few heads, in 32 bits, an odd width, no rotation
        dict(name="norm_vectors", op="norm", type="f32", B=2, L=777, H=6, G=6, N=100, kind="l2", w=False, rot=0, interleaved=False),
        # the gradients in a training step, whole heads rotated, pairs side by side
        dict(name="norm_grad", op="norm_bwd", type="bf16", B=4, L=2048, H=16, G=16, N=128, kind="rms", w=True, rot=128, interleaved=True),
        # the queries and keys of one token of each of many sequences at positions of their own
        dict(name="norm_step", op="norm", type="f16", B=64, L=1, H=32, G=8, N=128, kind="rms", w=True, rot=128, interleaved=False),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_bwd", "delta_bwd", "delta_step", "norm", "norm_bwd"])
    case = dict(op=op, type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    case["G"] = _spread(rng, 1, 32)
    case["H"] = case["G"] * rng.choice([1, 1, 2, 4])
    case["N"] = rng.choice([16, 40, 64, 64, 100, 128, 128, 128])
    if op.startswith("norm"):
        case.update(B=_spread(rng, 1, 64), L=_spread(rng, 1, 16384), kind=rng.choice(["rms", "rms", "l2"]), w=rng.random() < 0.7,
                    rot=2 * rng.choice([0, case["N"] // 4, case["N"] // 2]), interleaved=rng.random() < 0.3)
        most = {"norm": 8 * 4096 * 40 * 128, "norm_bwd": 4 * 2048 * 32 * 128}[op]
        one = (case["H"] + case["G"]) * case["N"]
    else:
        case["P"] = rng.choice([16, 64, 72, 128, 128, 128, 200, 256])
        case.update(B=_spread(rng, 1, 256 if op == "delta_step" else 8), L=1 if op == "delta_step" else _spread(rng, 1, 16384))
        most = {"delta": 4 * 4096 * 32 * 128 * 128, "delta_bwd": 4 * 2048 * 16 * 128 * 128, "delta_step": 256 * 32 * 128 * 128}[op]
        one = case["H"] * case["P"] * case["N"]
        if op != "delta_step":
            case.update(h0=rng.random() < 0.5, ragged=rng.random() < 0.3)
    # fewer sequences, or shorter ones, where the case would cost more than the largest listed one
    case["B"] = max(1, min(case["B"], most // one))
    case["L"] = max(1, min(case["L"], most // (one * case["B"])))
    return case


def work(case):
    B, L, H, G, N = (case[k] for k in "BLHGN")
    s, qk = (2 if case["type"] != "f32" else 4), B * L * (H + G) * N
    if case["op"] == "norm":  # four bytes a position
        return {"bytes": 2 * qk * s + (4 * B * L if case["rot"] else 0) + 8 * N, "flops": 8 * qk}
    if case["op"] == "norm_bwd":
        return {"bytes": 3 * qk * s + (4 * B * L if case["rot"] else 0) + 16 * N, "flops": 20 * qk}
    P = case["P"]
    qkv, vec, st = 2 * B * L * G * N * s, B * L * H * P * s, 4 * B * H * P * N
    gates = B * L * H * (4 + s)  # g in 32 bits, beta
    # the three products of a token with the state: S' k, u k^T, S q
    flops = 6 * B * L * H * P * N
    if case["op"] == "delta_step":
        return {"bytes": qkv + 2 * vec + gates + 2 * st, "flops": flops}
    h0 = int(case["h0"])
    if case["op"] == "delta":
        return {"bytes": qkv + 2 * vec + gates + st * (1 + h0), "flops": flops}
    # the states again, their adjoint's three products, and three more for the keys' and queries' gradients
    return {"bytes": 2 * (qkv + gates) + 3 * vec + 3 * st * h0, "flops": 16 * B * L * H * P * N}


# ---- inputs --------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, L, H, G, N, t = *(case[k] for k in "BLHGN"), TYPES[case["type"]]
    f32 = torch.float32

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    st = dict(case=case)
    step = L == 1 and case["op"] in ("delta_step", "norm")
    rows = (B,) if step else (B, L)
    if case["op"].startswith("norm"):
        st["q"], st["k"] = normal(*rows, H, N, scale=2.0), normal(*rows, G, N, scale=2.0)
        st["w_q"], st["w_k"] = (1.0 + 0.1 * normal(N, dtype=f32), 1.0 + 0.1 * normal(N, dtype=f32)) if case["w"] else (None, None)
        st["freqs"] = st["positions"] = None
        if case["rot"]:
            half = case["rot"] // 2
            st["freqs"] = torch.pow(10000.0, -torch.arange(half, device="cuda", dtype=torch.float64) / half).float()
            # every sequence somewhere in a document of up to a million tokens
            st["positions"] = (uniform(B) * 1e6).to(torch.int32)
            if not step:
                st["positions"] = st["positions"][:, None] + torch.arange(L, device="cuda", dtype=torch.int32)
        if case["op"] == "norm_bwd":
            st["dq_out"], st["dk_out"] = normal(*rows, H, N), normal(*rows, G, N)
        return st

    P = case["P"]

    def directions(heads):  # what a layer's convolution, SiLU and norm leave: mostly positive, of length one
        v = torch.nn.functional.silu(normal(*rows, heads, N, dtype=f32) + 0.2)
        return (v / (v * v).sum(-1, keepdim=True).add(EPS).sqrt()).to(t)

    st["q"], st["k"], st["v"] = directions(G), directions(G), normal(*rows, H, P)
    d = torch.exp(math.log(1e-3) + uniform(H) * math.log(100.0))  # steps of 0.001 to 0.1 at the middle
    a = 1.0 + 15.0 * uniform(H)
    st["g"] = -a * torch.nn.functional.softplus(d + torch.log(-torch.expm1(-d)) + normal(*rows, H, scale=0.5, dtype=f32))
    st["beta"] = torch.sigmoid(normal(*rows, H, dtype=f32)).to(t)
    if step:
        st["state"] = normal(B, H, P, N, scale=0.3, dtype=f32)
        st["state_out"] = torch.empty_like(st["state"])
        st["slots"] = torch.randperm(B, generator=gen, device="cuda").to(torch.int32)
        return st
    st["h0"] = normal(B, H, P, N, scale=0.3, dtype=f32) if case["h0"] else None
    if case["op"] == "delta_bwd":
        st["dy"] = normal(B, L, H, P)
        st["dfinal"] = normal(B, H, P, N, dtype=f32) if case["h0"] else None
    st["lengths"] = None
    if case["ragged"]:
        lengths = (uniform(B) * (L + 1)).to(torch.int32).clamp_(max=L)
        lengths[0] = L
        if B > 2:
            lengths[1] = 0
        st["lengths"] = lengths
    return st


# ---- plain forms ---------------------------------------------------------------------------------

def _live(st):
    """[B,L]: which tokens are a row's own."""
    B, L = st["v"].shape[:2]
    if st["lengths"] is None:
        return torch.ones((B, L), dtype=torch.bool, device="cuda")
    return torch.arange(L, device="cuda")[None, :] < st["lengths"][:, None]


def _chunks(x, live):
    """[B,L,H,...] to [B,H,chunk,C,...] in 32 bits, zeros past a row's end."""
    x = torch.where(live.reshape(*live.shape, *[1] * (x.dim() - 2)), x.float(), 0.0)
    pad = -x.shape[1] % C
    x = torch.cat([x, x.new_zeros((x.shape[0], pad, *x.shape[2:]))], 1)
    return x.unflatten(1, (-1, C)).movedim(3, 1)


def _tokens(x, L):
    """The way back: [B,H,chunk,C,...] to [B,L,H,...]."""
    return x.movedim(1, 3).flatten(1, 2)[:, :L]


def _heads(x, H):
    """[..., G, N] to [..., H, N]: the group of each head."""
    return x.repeat_interleave(H // x.shape[-2], -2)


def _inverse(A):
    """(I + A)^-1 for A [..., C, C] strictly below the diagonal: pairs of blocks of 1, 2, 4 ... rows joined."""
    T = torch.eye(C, device="cuda").expand(A.shape).clone()
    s = 1
    while s < C:
        first = torch.arange(0, C, 2 * s, device="cuda")[:, None] + torch.arange(s, device="cuda")
        up, low = first, first + s
        block = lambda m, r, c: m[..., r[:, :, None], c[:, None, :]]  # noqa: E731
        T[..., low[:, :, None], up[:, None, :]] = -(block(T, low, low) @ block(A, low, up) @ block(T, up, up))
        s *= 2
    return T


def _parts(st):
    """What both directions need of every chunk."""
    live, H, N = _live(st), st["v"].shape[2], st["q"].shape[-1]
    q, k = _chunks(_heads(st["q"], H), live), _chunks(_heads(st["k"], H), live)
    v, beta = _chunks(st["v"], live), _chunks(st["beta"], live)
    G = _chunks(st["g"], live).double().cumsum(-1)
    below = torch.ones((C, C), dtype=torch.bool, device="cuda").tril()
    decay = torch.exp(torch.where(below, G[..., :, None] - G[..., None, :], -math.inf)).float()
    into, out, over = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float(), torch.exp(G[..., -1]).float()
    T = _inverse((beta[..., None] * decay * (k @ k.mT)).tril(-1))
    return live, q, k, v, beta, decay, into, out, over, T, N ** -0.5


def _delta(st, states=False):
    live, q, k, v, beta, decay, into, out, over, T, scale = _parts(st)
    B, H, n = k.shape[:3]
    S = st["h0"].clone() if st["h0"] is not None else torch.zeros((B, H, v.shape[-1], k.shape[-1]), device="cuda")
    M = decay * (q @ k.mT)
    y, before, us, ws = torch.empty_like(v), [], [], []
    for c in range(n):
        w = v[:, :, c] - into[:, :, c, :, None] * (k[:, :, c] @ S.mT)
        u = T[:, :, c] @ (beta[:, :, c, :, None] * w)
        y[:, :, c] = scale * (into[:, :, c, :, None] * (q[:, :, c] @ S.mT) + M[:, :, c] @ u)
        if states:
            before.append(S)
            us.append(u)
            ws.append(w)
        S = over[:, :, c, None, None] * S + (out[:, :, c, :, None] * u).mT @ k[:, :, c]
    if states:
        return before, us, ws, S
    L = st["v"].shape[1]
    return torch.where(live[..., None, None], _tokens(y, L), 0.0).to(st["v"].dtype), S


def _delta_bwd(st):
    live, q, k, v, beta, decay, into, out, over, T, scale = _parts(st)
    before, us, ws, last = _delta(st, True)
    n, (B, L, H, P), G, N = k.shape[2], st["v"].shape, st["q"].shape[2], st["q"].shape[3]
    dy = scale * _chunks(st["dy"], live)
    M = decay * (q @ k.mT)
    dS = st["dfinal"].clone() if st["dfinal"] is not None else torch.zeros_like(last)
    dq, dk, dv, dbeta, dg = (torch.empty_like(x) for x in (q, k, v, beta, beta))
    after = last
    for c in reversed(range(n)):
        i, o, b = into[:, :, c, :, None], out[:, :, c, :, None], beta[:, :, c, :, None]
        qc, kc, d, u, S = q[:, :, c], k[:, :, c], dy[:, :, c], us[c], before[c]
        dr = T[:, :, c].mT @ (M[:, :, c].mT @ d + o * (kc @ dS.mT))
        dv[:, :, c] = b * dr
        Y, Z = decay[:, :, c] * (d @ u.mT), (b * decay[:, :, c] * (dr @ u.mT)).tril(-1)
        dq[:, :, c] = i * (d @ S) + Y @ kc
        read, written = -(b * i * (dr @ S) + Z @ kc), o * (u @ dS) + Y.mT @ qc - Z.mT @ kc
        dk[:, :, c] = read + written
        w = ws[c] - (decay[:, :, c] * (kc @ kc.mT)).tril(-1) @ u
        dbeta[:, :, c] = (dr * w).sum(-1)
        each = ((qc * dq[:, :, c]).sum(-1) + (kc * read).sum(-1) - (kc * written).sum(-1)).double()
        dg[:, :, c] = ((after * dS).double().sum((-1, -2))[..., None] + each.flip(-1).cumsum(-1).flip(-1)).float()
        dS = over[:, :, c, None, None] * dS + (i * d).mT @ qc - (b * i * dr).mT @ kc
        after = S

    def back(x, like):
        x = _tokens(x, L)
        if x.shape[2:] != like.shape[2:]:  # the heads of a group
            x = x.unflatten(2, (G, H // G)).sum(3)
        return torch.where(live.reshape(B, L, *[1] * (x.dim() - 2)), x, 0.0).to(like.dtype)

    res = dict(dq=back(dq, st["q"]), dk=back(dk, st["k"]), dv=back(dv, st["v"]), dg=back(dg, st["g"]), dbeta=back(dbeta, st["beta"]))
    if st["h0"] is not None:
        res["dh0"] = dS
    return res


def _delta_step(st):
    slots, H = st["slots"].long(), st["v"].shape[1]
    q, k = _heads(st["q"].float(), H)[:, :, None], _heads(st["k"].float(), H)[:, :, None]
    S = torch.exp(st["g"])[..., None, None] * st["state"][slots]
    u = st["beta"].float()[..., None] * (st["v"].float() - (S * k).sum(-1))
    S = S + u[..., None] * k
    st["state_out"][slots] = S
    return ((S * q).sum(-1) * st["q"].shape[-1] ** -0.5).to(st["v"].dtype), st["state_out"]


def _turn(st):
    """cos and sin of every token's angles, from angles in 64 bits; None where nothing is rotated."""
    if st["freqs"] is None:
        return None
    angle = st["positions"].double()[..., None, None] * st["freqs"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(x, turn, interleaved, back=False):
    if turn is None:
        return x
    cos, sin = turn
    if back:
        sin = -sin
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _inverse_norm(x, kind):
    sq = x * x
    return torch.rsqrt((sq.mean(-1, keepdim=True) if kind == "rms" else sq.sum(-1, keepdim=True)) + EPS)


def _norm(st):
    case, turn = st["case"], _turn(st)

    def one(x, w):
        v = x.float()
        v = v * _inverse_norm(v, case["kind"])
        return _rotate(v if w is None else v * w, turn, case["interleaved"]).to(x.dtype)

    return one(st["q"], st["w_q"]), one(st["k"], st["w_k"])


def _norm_bwd(st):
    case, turn, out = st["case"], _turn(st), {}
    for n in ("q", "k"):
        x, w, d = st[n].float(), st["w_" + n], _rotate(st["d%s_out" % n].float(), turn, case["interleaved"], True)
        inv = _inverse_norm(x, case["kind"])
        if w is not None:
            out["dw_" + n] = (d * x * inv).sum((0, 1, 2))
            d = d * w
        dot = (d * x).sum(-1, keepdim=True) / (x.shape[-1] if case["kind"] == "rms" else 1)
        out["d" + n] = (inv * (d - x * (inv * inv * dot))).to(st[n].dtype)
    return out


PLAIN = {"delta": _delta, "delta_bwd": _delta_bwd, "delta_step": _delta_step, "norm": _norm, "norm_bwd": _norm_bwd}


# ---- the framework's calls -----------------------------------------------------------------------

def _own(op, st):
    import mamba_ssd_chunked_fwd_gb300 as ssd
    if op == "delta":
        return ssd.delta_rule(st["q"], st["k"], st["v"], st["g"], st["beta"], return_final_state=True, initial_states=st["h0"],
                              lengths=st["lengths"])
    if op == "delta_bwd":
        return ssd.delta_rule_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["dy"], dfinal=st["dfinal"],
                                  initial_states=st["h0"], lengths=st["lengths"])
    if op == "delta_step":
        y = ssd.delta_rule_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], state_out=st["state_out"],
                                slots=st["slots"])
        return y, st["state_out"]
    how = dict(w_q=st["w_q"], w_k=st["w_k"], norm=st["case"]["kind"], eps=EPS, freqs=st["freqs"], positions=st["positions"],
               interleaved=st["case"]["interleaved"])
    if op == "norm":
        return ssd.qk_norm(st["q"], st["k"], **how)
    return ssd.qk_norm_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"], **how)


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return PLAIN[op](state)


# ---- in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    """The definitions token by token in 64 bits; gradients by differentiating them."""
    st = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    if case["op"].startswith("norm"):
        return _exact_norm(st, case)
    return _exact_delta(st, case)


def _exact_delta(st, case):
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    of = torch.arange(H, device="cuda") // (H // G)

    def token(S, q, k, v, g, beta):
        S = S * torch.exp(g)[..., None, None]
        error = v - torch.einsum("bhpn,bhn->bhp", S, k[:, of])
        S = S + torch.einsum("bhp,bhn->bhpn", error * beta[..., None], k[:, of])
        return S, torch.einsum("bhpn,bhn->bhp", S, q[:, of]) / math.sqrt(N)

    names = ("q", "k", "v", "g", "beta")
    if case["op"] == "delta_step":
        at = st["slots"].long()
        S, y = token(st["state"][at], *(st[n] for n in names))
        st["state_out"][at] = S
        return y, st["state_out"]
    grad = case["op"] == "delta_bwd"
    B, L = case["B"], case["L"]
    x = {n: st[n].detach().requires_grad_(grad) for n in names}
    x["h0"] = (st["h0"] if st["h0"] is not None else torch.zeros((B, H, P, N), dtype=torch.float64, device="cuda")).requires_grad_(grad)
    ends = None if st["lengths"] is None else st["lengths"].long()
    with torch.set_grad_enabled(grad):
        S, ys = x["h0"], []
        for t, parts in enumerate(zip(*(x[n].unbind(1) for n in names))):
            new, y = token(S, *parts)
            if ends is not None:
                on = (ends > t)[:, None, None]
                new, y = torch.where(on[..., None], new, S), torch.where(on, y, torch.zeros_like(y))
            S = new
            ys.append(y)
        y = torch.stack(ys, 1)
    if not grad:
        return y, S
    loss = (y * st["dy"]).sum() + (0 if st["dfinal"] is None else (S * st["dfinal"]).sum())
    got = {"d" + n: g for n, g in zip(x, torch.autograd.grad(loss, list(x.values())))}
    if st["h0"] is None:
        del got["dh0"]
    return got


def _exact_norm(st, case):
    def one(x, w):
        size = torch.linalg.vecdot(x, x)[..., None]
        x = x / torch.sqrt((size / x.shape[-1] if case["kind"] == "rms" else size) + EPS)
        if w is not None:
            x = x * w
        if st["freqs"] is None:
            return x
        n = case["rot"]
        pairs = x[..., :n].unflatten(-1, (-1, 2)) if case["interleaved"] else x[..., :n].unflatten(-1, (2, -1)).mT
        z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                                                    st["positions"].double()[..., None, None] * st["freqs"])
        z = torch.view_as_real(z)
        return torch.cat([(z if case["interleaved"] else z.mT).flatten(-2), x[..., n:]], -1)

    if case["op"] == "norm":
        return one(st["q"], st["w_q"]), one(st["k"], st["w_k"])
    leaves = {k: st[k].detach().requires_grad_(True) for k in ("q", "k", "w_q", "w_k") if st[k] is not None}
    with torch.enable_grad():
        loss = (one(leaves["q"], leaves.get("w_q")) * st["dq_out"]).sum() + (one(leaves["k"], leaves.get("w_k")) * st["dk_out"]).sum()
        got = torch.autograd.grad(loss, list(leaves.values()))
    return {"d" + k: g for k, g in zip(leaves, got)}
