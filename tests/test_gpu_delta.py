"""GPU parity of the gated delta rule, forward, backward and single-token, against the
plain 64-bit form, at the sizes, masks and strides where it can go wrong."""
import math

import pytest
import torch

import _delta_ref as ref
from _selective_ref import close, of

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAMES = ("q", "k", "v", "g", "beta")


def ssd():
    import mamba_ssd_chunked_fwd_gb300 as m
    return m


def make(B, L, H, G, N, P, t, *, h0=True, ragged=False, g32=True, b32=False, seed=0):
    gen = torch.Generator().manual_seed(1000 * seed + 7 * B + 5 * L + 3 * H + N + P)

    def normal(*shape, s=1.0, dt=t):
        return (torch.randn(shape, generator=gen) * s).to(dt)

    def unit(*shape):  # directions that share a part, as keys behind a SiLU do
        v = torch.nn.functional.silu(torch.randn(shape, generator=gen) + 0.2)
        return (v / (v.norm(dim=-1, keepdim=True) + 1e-6)).to(t)

    k = dict(q=unit(B, L, G, N), k=unit(B, L, G, N), v=normal(B, L, H, P),
             g=(-torch.exp(torch.randn((B, L, H), generator=gen) * 2 - 2)).to(F32 if g32 else t),
             beta=torch.sigmoid(torch.randn((B, L, H), generator=gen)).to(F32 if b32 else t),
             h0=normal(B, H, P, N, s=0.5, dt=F32) if h0 else None, lengths=None)
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=gen, dtype=torch.int32)
        n[0] = L
        if B > 1:
            n[1] = 0
        k["lengths"] = n
    return k


def cuda(k):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in k.items()}


def gpu(k, **more):
    return ssd().delta_rule(*(k[n] for n in NAMES), initial_states=k["h0"], lengths=k["lengths"], return_final_state=True, **more)


def plain(k, scale=None):
    f = {n: of(v) if n != "lengths" else v for n, v in k.items()}
    return ref.delta(*(f[n] for n in NAMES), f["h0"], f["lengths"], scale)


# one token; borders of tiles, chunks and rows; odd widths; shared keys; more rows than a CTA's; wide values
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 1, 2, 1, 16, 5), (1, 15, 2, 2, 64, 64), (2, 16, 1, 1, 128, 128), (1, 17, 3, 1, 40, 72),
          (1, 63, 2, 2, 128, 64), (1, 64, 2, 1, 128, 128), (2, 65, 4, 2, 64, 128), (1, 130, 2, 2, 100, 33), (1, 200, 2, 1, 128, 200),
          (1, 70, 6, 3, 33, 16), (3, 129, 2, 2, 128, 128), (1, 90, 1, 1, 128, 300), (1, 300, 2, 2, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_prompt(shape, t):
    k = make(*shape, t)
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    assert y.dtype == t and fin.dtype == F32
    close(y, ry, "y")
    close(fin, rfin, "final state")


@pytest.mark.parametrize("opts", [dict(h0=False), dict(g32=False), dict(b32=True), dict(ragged=True), dict(ragged=True, h0=False, g32=False)])
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("shape", [(3, 150, 4, 2, 128, 128), (4, 90, 2, 2, 64, 40), (3, 77, 3, 3, 20, 128)])
def test_options(shape, t, opts):
    k = make(*shape, t, **opts)
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")


def test_scale():
    k = make(1, 70, 2, 1, 128, 128, BF16)
    close(gpu(cuda(k), scale=0.5)[0], plain(k, 0.5)[0], "y")


def grads(k, seed=9):
    gen = torch.Generator().manual_seed(seed)
    dy = torch.randn(k["v"].shape, generator=gen).to(k["v"].dtype)
    B, _, H, P = k["v"].shape
    return dy, torch.randn((B, H, P, k["q"].shape[-1]), generator=gen)


def gpu_bwd(k, dy, dfinal, **more):
    return ssd().delta_rule_bwd(*(k[n] for n in NAMES), dy, dfinal=dfinal, initial_states=k["h0"], lengths=k["lengths"], **more)


def plain_bwd(k, dy, dfinal, scale=None):
    inputs = {n: of(k[n]) for n in (*NAMES, "h0")}
    f = lambda q, k_, v, g, beta, h0: ref.delta(q, k_, v, g, beta, h0, k["lengths"], scale)  # noqa: E731
    leaves = {n: v.clone().requires_grad_(True) for n, v in inputs.items() if v is not None}
    got = f(*(leaves[n] for n in NAMES), leaves.get("h0"))
    loss = (got[0] * of(dy)).sum() + (0 if dfinal is None else (got[1] * of(dfinal)).sum())
    out = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return {"d" + n: torch.zeros_like(v) if x is None else x for (n, v), x in zip(leaves.items(), out)}


def check_bwd(k, dfinal=True, **more):
    dy, df = grads(k)
    df = df if dfinal else None
    got = gpu_bwd(cuda(k), dy.cuda(), df.cuda() if dfinal else None, **more)
    want = plain_bwd(k, dy, df)
    assert set(got) == set(want)
    for n in got:
        like = k[n[1:]]
        assert got[n].dtype == like.dtype and got[n].shape == like.shape
        close(got[n], want[n], n)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_gradients(shape, t):
    check_bwd(make(*shape, t))


@pytest.mark.parametrize("opts", [dict(h0=False), dict(g32=False), dict(b32=True), dict(ragged=True), dict(ragged=True, h0=False, g32=False)])
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("shape", [(3, 150, 4, 2, 128, 128), (4, 90, 2, 2, 64, 40)])
def test_gradients_of_options(shape, t, opts):
    check_bwd(make(*shape, t, **opts), dfinal=opts.get("h0", True))


def test_gradients_against_differences():
    """In fp32 with steps of 2^-6: a central difference of sum(dy y) + sum(dfinal final) along
    a direction errs by its third derivative over 6 times the step squared, and by the
    rounding of two sums of about 1500 products of unit size: sqrt(1500) 2^-24 39 / 2^-6 = 6e-3 at most."""
    k = make(1, 70, 2, 1, 20, 12, F32)
    dy, df = grads(k)
    got = gpu_bwd(cuda(k), dy.cuda(), df.cuda())
    gen = torch.Generator().manual_seed(4)
    for n in (*NAMES, "h0"):
        way = torch.randn(k[n].shape, generator=gen)
        way = way / way.norm()
        loss = []
        for sign in (1, -1):
            moved = dict(k)
            moved[n] = k[n] + sign * 2.0 ** -6 * way
            y, fin = gpu(cuda(moved))
            loss.append((y.double().cpu() * dy.double()).sum() + (fin.double().cpu() * df.double()).sum())
        slope = ((loss[0] - loss[1]) / 2.0 ** -5).item()
        want = (got["d" + n].double().cpu() * way.double()).sum().item()
        assert abs(slope - want) <= 0.02 * max(1.0, got["d" + n].norm().item()), (n, slope, want)


def poison(k):
    """NaN and infinities in the padding."""
    for n in NAMES:
        for b, e in enumerate(k["lengths"].tolist()):
            k[n][b, e:] = float("nan") if b % 2 == 0 else float("inf")


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("shape", [(3, 150, 4, 2, 128, 128), (3, 70, 2, 1, 40, 20)])
def test_padding_does_not_leak(shape, t):
    k = make(*shape, t, ragged=True)
    dy, df = grads(k)
    want, wantb = gpu(cuda(k)), gpu_bwd(cuda(k), dy.cuda(), df.cuda())
    poison(k)
    for b, e in enumerate(k["lengths"].tolist()):
        dy[b, e:] = float("nan")
    got, gotb = gpu(cuda(k)), gpu_bwd(cuda(k), dy.cuda(), df.cuda())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for n in gotb:
        assert torch.equal(gotb[n], wantb[n]), n
        if n != "dh0":
            for b, e in enumerate(k["lengths"].tolist()):
                assert not gotb[n][b, e:].any(), n


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("offset", [8, 1])
@pytest.mark.parametrize("shape", [(2, 150, 4, 2, 128, 128), (2, 70, 2, 1, 40, 20)])
def test_strided_inputs(shape, t, offset):
    """q, k and v as slices of one projection, g and beta as slices of another: to the bit what dense
    tensors give where the slices are aligned as those are; elsewhere another kernel may take them."""
    host = make(*shape, t, g32=False)
    k = cuda(host)
    B, L = shape[:2]
    widths = [k[n][0, 0].numel() for n in NAMES]
    wide = torch.full((B, L, sum(widths) + 5 * offset), float("nan"), device="cuda", dtype=t)
    at, s = 0, dict(k)
    for n, w in zip(NAMES, widths):
        at += offset
        wide[..., at:at + w] = k[n].reshape(B, L, w)
        s[n] = wide[..., at:at + w].unflatten(-1, k[n].shape[2:])
        at += w
    dy, df = grads(k)
    a, ab = gpu(s), gpu_bwd(s, dy.cuda(), df.cuda())
    if offset == 8 or t == F32:
        b, bb = gpu(k), gpu_bwd(k, dy.cuda(), df.cuda())
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        for n in ab:
            assert torch.equal(ab[n], bb[n]), n
        return
    for x, y in zip(a, plain(host)):
        close(x, y)
    want = plain_bwd(host, dy.cpu(), df.cpu())
    for n in ab:
        close(ab[n], want[n], n)


@pytest.mark.parametrize("t", [F32, BF16])
def test_carries_its_state(t):
    """A prompt in two parts, the second from the first one's state."""
    k = make(2, 140, 4, 2, 128, 64, t)
    y, fin = gpu(cuda(k))
    cut = lambda a, b: {n: v[:, a:b].contiguous() if n in NAMES else v for n, v in k.items()}  # noqa: E731
    y0, mid = gpu(cuda(cut(0, 75)))
    y1, end = gpu({**cuda(cut(75, 140)), "h0": mid})
    close(torch.cat([y0, y1], 1), plain(k)[0], "y")
    close(end, plain(k)[1], "state")


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("g", [0.0, -1e-4, -30.0, -200.0, -math.inf])
def test_extreme_decays(t, g):
    """No decay at all, and decays that empty the state at once, every ninth token."""
    k = make(1, 150, 2, 1, 128, 128, t, g32=True)
    k["g"] = torch.full_like(k["g"], -0.01)
    k["g"][:, ::9] = g
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    if g > -math.inf:
        check_bwd(k)


@pytest.mark.parametrize("t", [F32, BF16])
def test_alike_keys(t):
    """Every key the same and beta 1: what a token writes, the next one takes out whole.  The
    inverse of a chunk then has large powers that cancel."""
    k = make(1, 130, 2, 1, 128, 128, t)
    one = torch.zeros(128)
    one[::4] = 0.1767578125  # exact in the 16-bit types; length 1 within 2^-11
    k["k"] = one.to(t).expand_as(k["k"]).contiguous()
    k["q"] = k["k"].clone()
    k["beta"] = torch.ones_like(k["beta"])
    k["g"] = torch.zeros_like(k["g"])
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    check_bwd(k)


def test_zero_steps():
    """beta = 0 leaves the state but for its decay, and its gradient is there all the same."""
    k = make(1, 80, 2, 2, 128, 64, BF16)
    k["beta"] = torch.zeros_like(k["beta"])
    k["beta"][:, 40] = 0.5
    y, fin = gpu(cuda(k))
    close(fin, plain(k)[1], "state")
    check_bwd(k)


@pytest.mark.parametrize("t", [F32, BF16])
def test_far_tokens(t):
    """A thousand tokens of slow decay."""
    k = make(1, 1100, 1, 1, 64, 64, t)
    k["g"] = torch.full_like(k["g"], -2e-3)
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "state")


@pytest.mark.parametrize("t", [F32, BF16])
def test_deterministic(t):
    k = cuda(make(2, 200, 4, 2, 128, 128, t))
    dy, df = grads(k)
    a, b = gpu(k), gpu(k)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = (gpu_bwd(k, dy.cuda(), df.cuda()) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


# ---- single tokens

STEPS = [(1, 1, 1, 1, 1), (3, 2, 1, 16, 5), (2, 4, 2, 128, 128), (5, 3, 3, 40, 72), (2, 2, 2, 100, 33), (1, 16, 16, 128, 128), (40, 32, 16, 64, 64)]


@pytest.mark.parametrize("shape", STEPS)
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_step(shape, t):
    B, H, G, N, P = shape
    k = make(B, 1, H, G, N, P, t)
    c = cuda(k)
    one = [c[n][:, 0] for n in NAMES]
    state = c["h0"].clone()
    y = ssd().delta_rule_step(*one, state)
    ry, rfin = plain(k)
    close(y, ry[:, 0], "y")
    close(state, rfin, "state")


@pytest.mark.parametrize("t", [F32, BF16])
def test_steps_equal_the_prompt(t):
    k = make(2, 20, 4, 2, 128, 64, t)
    c = cuda(k)
    state = c["h0"].clone()
    ys = [ssd().delta_rule_step(*(c[n][:, i] for n in NAMES), state) for i in range(20)]
    ry, rfin = plain(k)
    close(torch.stack(ys, 1), ry, "y")
    close(state, rfin, "state")


def test_step_slots():
    """Rows in places of their own; one outside the pool on either side; the others left as they are."""
    B, H, G, N, P = 5, 4, 2, 128, 128
    k = make(B, 1, H, G, N, P, BF16)
    c = cuda(k)
    pool = torch.randn((9, H, P, N), device="cuda")
    slots = torch.tensor([7, -1, 3, 9, 0], dtype=torch.int32, device="cuda")
    out, before = pool.clone(), pool.clone()
    y = ssd().delta_rule_step(*(c[n][:, 0] for n in NAMES), pool, state_out=out, slots=slots)
    assert torch.equal(pool, before)
    for b, s in enumerate(slots.tolist()):
        if not 0 <= s < 9:
            assert not y[b].any()
            continue
        one = {**{n: k[n][b:b + 1] for n in NAMES}, "h0": before[s:s + 1].cpu(), "lengths": None}
        ry, rs = plain(one)
        close(y[b:b + 1], ry[:, 0], "y")
        close(out[s:s + 1], rs, "state")
    untouched = [1, 2, 4, 5, 6, 8]
    assert torch.equal(out[untouched], before[untouched])


def test_step_in_a_large_pool():
    """Offsets past 2^31 elements."""
    H, P, N = 2, 128, 128
    S = (2 ** 31) // (H * P * N) + 3
    pool = torch.zeros((S, H, P, N), device="cuda")
    k = make(2, 1, H, 1, N, P, BF16)
    c = cuda(k)
    slots = torch.tensor([S - 1, S - 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = c["h0"]
    y = ssd().delta_rule_step(*(c[n][:, 0] for n in NAMES), pool, slots=slots)
    ry, rs = plain(k)
    close(y, ry[:, 0], "y")
    close(pool[slots.long()], rs, "state")


def test_step_of_strided_rows():
    k = cuda(make(3, 2, 4, 2, 128, 64, BF16))
    rows = [k[n][:, 1] for n in NAMES]  # every second token of a prompt: rows are apart
    a, b = k["h0"].clone(), k["h0"].clone()
    assert torch.equal(ssd().delta_rule_step(*rows, a), ssd().delta_rule_step(*(r.contiguous() for r in rows), b))
    assert torch.equal(a, b)


# ---- streams, graphs

def test_other_stream_and_graph():
    k = cuda(make(2, 150, 4, 2, 128, 128, BF16))
    dy, df = grads(k)
    dy, df = dy.cuda(), df.cuda()
    want, wantb = gpu(k), gpu_bwd(k, dy, df)
    state = k["h0"].clone()
    one = [k[n][:, 0].contiguous() for n in NAMES]
    step = ssd().delta_rule_step(*one, state)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gotb = gpu(k), gpu_bwd(k, dy, df)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(gotb[n], wantb[n]) for n in wantb)
    graph = torch.cuda.CUDAGraph()
    again = k["h0"].clone()
    with torch.cuda.graph(graph):
        got, gotb = gpu(k), gpu_bwd(k, dy, df)
        y = ssd().delta_rule_step(*one, again)
    again.copy_(k["h0"])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(gotb[n], wantb[n]) for n in wantb)
    second = k["h0"].clone()
    ssd().delta_rule_step(*one, second)
    assert torch.equal(ssd().delta_rule_step(*one, second), y) and torch.equal(second, again)
