"""GPU parity of the selective scan and its convolution, forward, backward and
single-token, against the plain 64-bit forms, at the sizes, masks and strides
where they can go wrong."""
import math

import pytest
import torch

import _selective_ref as ref
from _selective_ref import close, of

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def ssd():
    import mamba_ssd_chunked_fwd_gb300 as m
    return m


def make(B, L, D, N, G, t, *, z=True, h0=True, ragged=False, dt32=False, skip=True, bias=True, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + B * 7 + L * 5 + D * 3 + N)

    def normal(*shape, s=1.0, dt=t):
        return (torch.randn(shape, generator=g) * s).to(dt)

    d = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)
    k = dict(x=normal(B, L, D), dt=normal(B, L, D, s=0.5, dt=F32 if dt32 else t),
             A=-torch.rand((D, N), generator=g) * 8 - 0.05, B=normal(B, L, G, N), C=normal(B, L, G, N),
             D=normal(D, dt=F32) if skip else None, z=normal(B, L, D) if z else None,
             dt_bias=d + torch.log(-torch.expm1(-d)) if bias else None,
             h0=normal(B, D, N, dt=F32) if h0 else None, lengths=None)
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
        n[0] = L
        if B > 1:
            n[1] = 0
        k["lengths"] = n
    return k


def cuda(k):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in k.items()}


def gpu_scan(k, softplus=True, limit=(0.0, math.inf)):
    return ssd().selective_scan(k["x"], k["dt"], k["A"], k["B"], k["C"], softplus, True, D=k["D"], z=k["z"],
                                dt_bias=k["dt_bias"], initial_states=k["h0"], lengths=k["lengths"], dt_limit=limit)


def ref_scan(k, softplus=True, limit=(0.0, math.inf)):
    f = {n: of(v) if n != "lengths" else v for n, v in k.items()}
    return ref.scan(f["x"], f["dt"], f["A"], f["B"], f["C"], f["D"], f["z"], f["dt_bias"], f["h0"], f["lengths"], softplus, limit)


# one token; tile and checkpoint borders; odd channels, states and groups; more states than lanes; cut sequences
SHAPES = [(1, 1, 1, 1, 1), (2, 1, 5, 16, 1), (2, 7, 6, 3, 2), (1, 8, 130, 4, 1), (3, 9, 64, 16, 1), (1, 15, 34, 8, 2),
          (2, 17, 256, 16, 2), (1, 33, 66, 20, 1), (2, 31, 24, 32, 1), (1, 20, 40, 64, 1), (1, 12, 20, 100, 2),
          (1, 10, 16, 128, 1), (1, 300, 12, 16, 1), (2, 150, 136, 12, 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [F32, BF16])
def test_scan(shape, t):
    k = make(*shape, t)
    y, fin = gpu_scan(cuda(k))
    ry, rfin = ref_scan(k)
    assert y.dtype == t and fin.dtype == F32
    close(y, ry, "y")
    close(fin, rfin, "final state")


@pytest.mark.parametrize("opts", [dict(z=False), dict(h0=False), dict(skip=False), dict(bias=False), dict(dt32=True),
                                  dict(ragged=True), dict(ragged=True, z=False, skip=False, dt32=True)])
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("shape", [(3, 21, 72, 16, 1), (3, 90, 10, 5, 2)])
def test_scan_options(shape, t, opts):
    k = make(*shape, t, **opts)
    y, fin = gpu_scan(cuda(k))
    ry, rfin = ref_scan(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")


@pytest.mark.parametrize("softplus,limit", [(False, (0.0, math.inf)), (False, (0.01, 0.3)), (True, (0.004, 0.05))])
def test_scan_steps(softplus, limit):
    """Steps without softplus, and clamped."""
    k = make(2, 40, 24, 16, 1, F32)
    if not softplus:
        k["dt"], k["dt_bias"] = k["dt"].abs() * 0.3, None
    y, fin = gpu_scan(cuda(k), softplus, limit)
    ry, rfin = ref_scan(k, softplus, limit)
    close(y, ry, "y")
    close(fin, rfin, "final state")


def test_scan_of_extreme_steps():
    """Steps of exp(-30) to 50: no overflow, and small ones keep their relative precision."""
    k = make(1, 24, 16, 8, 1, F32, z=False, skip=False, bias=False, h0=False)
    k["dt"] = torch.linspace(-30.0, 50.0, 24)[None, :, None].expand(1, 24, 16).contiguous()
    y, fin = gpu_scan(cuda(k))
    ry, rfin = ref_scan(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    close(y[:, :4], ry[:, :4], "the smallest steps")


def poison(k, names):
    """NaN and infinities in the padding."""
    for n in names:
        if k[n] is not None:
            for b, e in enumerate(k["lengths"].tolist()):
                k[n][b, e:] = float("nan") if b % 2 == 0 else float("inf")


@pytest.mark.parametrize("t", [F32, BF16])
def test_padding_does_not_leak(t):
    k = make(3, 37, 40, 16, 1, t, ragged=True)
    clean = cuda(k)
    bad = {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in k.items()}
    poison(bad, ["x", "dt", "z", "B", "C"])
    a, b = gpu_scan(clean), gpu_scan(cuda(bad))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[0][1] == 0).all() and torch.equal(a[1][1], clean["h0"][1])  # the empty row


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("t", [F32, BF16])
def test_strided_inputs(t, offset):
    """x, z, dt, B and C as slices of wider projections, on and off 16-byte boundaries."""
    k = cuda(make(2, 30, 48, 16, 1, t))
    wide = torch.randn((2, 30, 48 * 3 + 32 + 24 + offset), device="cuda").to(t)
    cut, at = dict(k), offset
    for n, width in (("x", 48), ("z", 48), ("dt", 48), ("B", 16), ("C", 16)):
        part = wide[..., at:at + width]
        part.copy_(k[n].reshape(2, 30, width))
        cut[n] = part.unsqueeze(2) if n in "BC" else part
        at += width
    a, b = gpu_scan(k), gpu_scan(cut)
    close(b[0], a[0].double(), "y")
    close(b[1], a[1].double(), "final state")


def test_scan_carries_its_state():
    """Two calls equal one; a transposed batch works too."""
    k = cuda(make(2, 70, 40, 16, 1, F32))
    y, fin = gpu_scan(k)
    first = {n: v[:, :33] if n in ("x", "dt", "B", "C", "z") else v for n, v in k.items()}
    y0, mid = gpu_scan(first)
    rest = {n: v[:, 33:] if n in ("x", "dt", "B", "C", "z") else v for n, v in k.items()}
    y1, end = gpu_scan({**rest, "h0": mid})
    close(torch.cat([y0, y1], 1), y.double(), "y")
    close(end, fin.double(), "final state")


def test_scan_far_tokens():
    """Token offsets past 2^31 elements."""
    k = cuda(make(1, 40, 16, 8, 1, BF16))
    wide = torch.empty((40, 60_000_000), device="cuda", dtype=BF16)
    far = wide[None, :, 7:23]
    far.copy_(k["x"])
    a, b = gpu_scan(k), gpu_scan({**k, "x": far})
    close(b[0], a[0].double(), "y")


GRADS = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias", "h0": "dh0"}


def gpu_scan_bwd(k, dy, dfinal, softplus=True, limit=(0.0, math.inf)):
    return ssd().selective_scan_bwd(k["x"], k["dt"], k["A"], k["B"], k["C"], dy, softplus, dfinal=dfinal, D=k["D"], z=k["z"],
                                    dt_bias=k["dt_bias"], initial_states=k["h0"], lengths=k["lengths"], dt_limit=limit)


def ref_scan_bwd(k, dy, dfinal, softplus=True, limit=(0.0, math.inf)):
    def f(x, dt, A, B, C, D, z, dt_bias, h0):
        return ref.scan(x, dt, A, B, C, D, z, dt_bias, h0, k["lengths"], softplus, limit)
    got = ref.gradients(f, {n: of(k[n]) for n in GRADS}, [of(dy), of(dfinal)])
    return {GRADS[n]: v for n, v in got.items()}


def grads_like(k, dfinal=True, seed=5):
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(k["x"].shape, generator=g).to(k["x"].dtype)
    return dy, torch.randn((k["x"].shape[0], *k["A"].shape), generator=g) if dfinal else None


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [F32, BF16])
def test_scan_bwd(shape, t):
    k = make(*shape, t)
    dy, df = grads_like(k)
    got = gpu_scan_bwd(cuda(k), dy.cuda(), df.cuda())
    for n, r in ref_scan_bwd(k, dy, df).items():
        close(got[n], r, n)


@pytest.mark.parametrize("opts", [dict(z=False), dict(h0=False), dict(skip=False), dict(bias=False), dict(dt32=True),
                                  dict(ragged=True), dict(ragged=True, z=False, skip=False, dt32=True)])
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("shape", [(3, 21, 72, 16, 1), (3, 90, 10, 5, 2)])
def test_scan_bwd_options(shape, t, opts):
    k = make(*shape, t, **opts)
    dy, df = grads_like(k, dfinal="h0" not in opts)
    got = gpu_scan_bwd(cuda(k), dy.cuda(), None if df is None else df.cuda())
    want = ref_scan_bwd(k, dy, df)
    assert set(got) == set(want)
    for n, r in want.items():
        close(got[n], r, n)


def test_scan_bwd_of_clamped_steps():
    k = make(2, 40, 24, 16, 1, F32)
    dy, df = grads_like(k)
    got = gpu_scan_bwd(cuda(k), dy.cuda(), df.cuda(), True, (0.004, 0.05))
    for n, r in ref_scan_bwd(k, dy, df, True, (0.004, 0.05)).items():
        close(got[n], r, n)
    assert (got["ddt"] == 0).any()


@pytest.mark.parametrize("t", [F32, BF16])
def test_scan_bwd_padding_does_not_leak(t):
    k = make(3, 37, 40, 16, 1, t, ragged=True)
    dy, df = grads_like(k)
    a = gpu_scan_bwd(cuda(k), dy.cuda(), df.cuda())
    bad = {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in k.items()}
    bad["dy"] = dy.clone()
    poison(bad, ["x", "dt", "z", "B", "C", "dy"])
    b = gpu_scan_bwd(cuda(bad), bad["dy"].cuda(), df.cuda())
    for n in a:
        assert torch.equal(a[n], b[n]), n
    for n in ("dx", "ddt", "dz", "dB", "dC"):
        assert (a[n][1] == 0).all(), n
    assert torch.equal(a["dh0"][1], df.cuda()[1])  # an empty row hands its gradient on


def test_scan_bwd_against_differences():
    """The directional derivative of the 64-bit forward along random directions."""
    k = make(1, 30, 12, 8, 2, F32)
    dy, df = grads_like(k)
    got = gpu_scan_bwd(cuda(k), dy.cuda(), df.cuda())
    g = torch.Generator().manual_seed(9)
    for n, out in GRADS.items():
        v = torch.randn(k[n].shape, generator=g, dtype=torch.float64)
        e = 1e-6

        def value(s):
            y, fin = ref_scan({**k, n: of(k[n]) + s * e * v})
            return (y * of(dy)).sum() + (fin * of(df)).sum()
        slope = ((value(1) - value(-1)) / (2 * e)).item()
        mine = (got[out].double().cpu() * v).sum().item()
        # the gradient's bound times the direction's length, and the difference's own error
        bound = ref.REL * got[out].double().norm().item() * v.norm().item() + 1e-6 * abs(slope) + 1e-6
        assert abs(slope - mine) <= bound, (out, slope, mine)


def test_scan_is_deterministic():
    k = cuda(make(2, 200, 70, 16, 1, BF16))
    dy, df = grads_like(make(2, 200, 70, 16, 1, BF16))
    a, b = gpu_scan(k), gpu_scan(k)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    p, q = gpu_scan_bwd(k, dy.cuda(), df.cuda()), gpu_scan_bwd(k, dy.cuda(), df.cuda())
    assert all(torch.equal(p[n], q[n]) for n in p)


# ---- single tokens -----------------------------------------------------------

@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("shape", [(1, 5, 1, 1), (3, 24, 16, 2), (2, 66, 20, 1), (1, 16, 128, 1), (5, 40, 7, 1)])
def test_steps_equal_the_prompt(shape, t):
    B, D, N, G = shape
    k = make(B, 6, D, N, G, t)
    want, wfin = ref_scan(k)
    k = cuda(k)
    h = k["h0"].clone()
    for i in range(6):
        y = ssd().selective_scan_step(k["x"][:, i], k["dt"][:, i], k["A"], k["B"][:, i], k["C"][:, i], h, True, D=k["D"],
                                      z=k["z"][:, i], dt_bias=k["dt_bias"])
        close(y, want[:, i], f"token {i}")
    close(h, wfin, "state")


@pytest.mark.parametrize("B", [3, 130])
def test_step_slots(B):
    """States in a pool: rows find theirs, others stay, bad slots give 0 and touch
    nothing; B = 130 takes four sequences per lane, the last block not full."""
    D, N, S = (40, 16, 7) if B == 3 else (2048, 16, 140)
    k = cuda(make(B, 1, D, N, 1, BF16, h0=False))
    pool = torch.randn((S, D, N), device="cuda")
    slots = torch.randperm(S)[:B].to(torch.int32)
    slots[1], slots[2] = -1, S
    before = pool.clone()
    out = torch.full_like(pool, 7.0)
    y = ssd().selective_scan_step(k["x"][:, 0], k["dt"][:, 0], k["A"], k["B"][:, 0], k["C"][:, 0], pool, True, state_out=out,
                                  slots=slots.cuda(), D=k["D"], z=k["z"][:, 0], dt_bias=k["dt_bias"])
    assert torch.equal(pool, before) and (y[1:3] == 0).all()
    live = [b for b in range(B) if 0 <= int(slots[b]) < S]
    part = {n: v[live] if n in ("x", "dt", "B", "C", "z") else v for n, v in k.items()}
    part["h0"] = before[[int(slots[b]) for b in live]]
    want, wfin = ref_scan(part)
    close(y[live], want[:, 0], "y")
    close(out[[int(slots[b]) for b in live]], wfin, "states")
    rest = [s for s in range(S) if s not in {int(slots[b]) for b in live}]
    assert (out[rest] == 7.0).all()


def test_step_in_a_large_pool():
    """Slot offsets past 2^31 elements."""
    D, N, S = 1024, 16, 131_100
    k = cuda(make(2, 1, D, N, 1, F32))
    pool = torch.empty((S, D, N), device="cuda")
    slots = torch.tensor([S - 1, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = k["h0"]
    y = ssd().selective_scan_step(k["x"][:, 0], k["dt"][:, 0], k["A"], k["B"][:, 0], k["C"][:, 0], pool, True, slots=slots,
                                  D=k["D"], z=k["z"][:, 0], dt_bias=k["dt_bias"])
    want, wfin = ref_scan(k)
    close(y, want[:, 0], "y")
    close(pool[slots.long()], wfin, "states")


# ---- convolution -------------------------------------------------------------

def make_conv(B, L, C, W, t, *, h0=True, ragged=False, bias=True):
    g = torch.Generator().manual_seed(B + L * 3 + C * 5 + W)
    k = dict(x=torch.randn((B, L, C), generator=g).to(t), w=torch.randn((C, W), generator=g) * 0.5,
             bias=torch.randn(C, generator=g) if bias else None,
             h0=torch.randn((B, W - 1, C), generator=g).to(t) if h0 else None, lengths=None)
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
        n[0], n[-1] = L, min(1, L)
        if B > 2:
            n[1] = 0
        k["lengths"] = n
    return k


CONVS = [(1, 1, 1, 1), (2, 1, 8, 4), (1, 2, 5, 4), (2, 3, 130, 3), (1, 31, 64, 2), (2, 33, 36, 4), (1, 70, 12, 8), (1, 150, 132, 5),
         (2, 260, 24, 4)]


@pytest.mark.parametrize("shape", CONVS)
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("opts", [dict(), dict(h0=False, bias=False), dict(ragged=True)])
def test_conv(shape, t, opts):
    k = make_conv(*shape, t, **opts)
    c = cuda(k)
    for silu in (True, False):
        y, fin = ssd().causal_conv1d_carry(c["x"], c["w"], c["bias"], silu, initial_state=c["h0"], lengths=c["lengths"],
                                           return_final_state=True)
        ry, rfin = ref.conv(of(k["x"]), of(k["w"]), of(k["bias"]), of(k["h0"]), k["lengths"], silu)
        close(y, ry, "y")
        assert torch.equal(fin.cpu().double(), rfin)


@pytest.mark.parametrize("shape", CONVS)
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("opts", [dict(), dict(h0=False, bias=False), dict(ragged=True)])
def test_conv_bwd(shape, t, opts):
    k = make_conv(*shape, t, **opts)
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(k["x"].shape, generator=g).to(t)
    df = torch.randn((shape[0], shape[3] - 1, shape[2]), generator=g).to(t) if k["h0"] is not None else None
    c = cuda(k)
    for silu in (True, False):
        got = ssd().causal_conv1d_bwd(c["x"], c["w"], dy.cuda(), c["bias"], silu, dfinal=None if df is None else df.cuda(),
                                      initial_state=c["h0"], lengths=c["lengths"])

        def f(x, w, bias, h0):
            return ref.conv(x, w, bias, h0, k["lengths"], silu)
        want = ref.gradients(f, {n: of(k[n]) for n in ("x", "w", "bias", "h0")}, [of(dy), of(df)])
        assert set(got) == {"dx", "dw"} | ({"dbias"} if k["bias"] is not None else set()) | ({"dh0"} if df is not None else set())
        for n, r in want.items():
            close(got["d" + n], r, "d" + n)


def test_conv_bwd_against_differences():
    k = make_conv(1, 40, 6, 4, F32)
    g = torch.Generator().manual_seed(4)
    dy, df = torch.randn(k["x"].shape, generator=g), torch.randn((1, 3, 6), generator=g)
    c = cuda(k)
    got = ssd().causal_conv1d_bwd(c["x"], c["w"], dy.cuda(), c["bias"], dfinal=df.cuda(), initial_state=c["h0"])
    for n in ("x", "w", "bias", "h0"):
        v, e = torch.randn(k[n].shape, generator=g, dtype=torch.float64), 1e-6

        def value(s):
            f = {m: of(k[m]) for m in ("x", "w", "bias", "h0")}
            f[n] = f[n] + s * e * v
            y, fin = ref.conv(f["x"], f["w"], f["bias"], f["h0"])
            return (y * of(dy)).sum() + (fin * of(df)).sum()
        slope = ((value(1) - value(-1)) / (2 * e)).item()
        mine = (got["d" + n].double().cpu() * v).sum().item()
        assert abs(slope - mine) <= ref.REL * got["d" + n].double().norm().item() * v.norm().item() + 1e-6 * abs(slope) + 1e-6, n


@pytest.mark.parametrize("t", [F32, BF16])
def test_conv_padding_and_strides(t):
    k = make_conv(3, 40, 24, 4, t, ragged=True)
    c = cuda(k)
    bad = c["x"].clone()
    for b, e in enumerate(k["lengths"].tolist()):
        bad[b, e:] = float("nan")
    wide = torch.zeros((3, 40, 24 * 2 + 3), device="cuda", dtype=t)
    wide[..., 3:27] = bad
    f = dict(initial_state=c["h0"], lengths=c["lengths"], return_final_state=True)
    a = ssd().causal_conv1d_carry(c["x"], c["w"], c["bias"], **f)
    for x in (bad, wide[..., 3:27]):
        b = ssd().causal_conv1d_carry(x, c["w"], c["bias"], **f)
        close(b[0], a[0].double(), "y")
        assert torch.equal(a[1], b[1])
    dy = torch.randn_like(c["x"])
    p = ssd().causal_conv1d_bwd(c["x"], c["w"], dy, c["bias"], initial_state=c["h0"], lengths=c["lengths"])
    q = ssd().causal_conv1d_bwd(bad, c["w"], torch.where(torch.isnan(bad), bad, dy), c["bias"], initial_state=c["h0"],
                                lengths=c["lengths"])
    assert all(torch.equal(p[n], q[n]) for n in p)


@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_conv_steps_equal_the_prompt(W, t):
    k = make_conv(3, 10, 37, W, t)
    want, wfin = ref.conv(of(k["x"]), of(k["w"]), of(k["bias"]), of(k["h0"]))
    c = cuda(k)
    pool = torch.zeros((5, W - 1, 37), device="cuda", dtype=t)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = c["h0"]
    for i in range(10):
        y = ssd().causal_conv1d_step(c["x"][:, i], pool, c["w"], c["bias"], slots=slots)
        close(y, want[:, i], f"token {i}")
    assert torch.equal(pool[slots.long()].double().cpu(), wfin)
    assert (pool[[1, 3]] == 0).all()
    y = ssd().causal_conv1d_step(c["x"][:, 0], pool.clone(), c["w"], c["bias"], slots=torch.tensor([-1, 5, 1], dtype=torch.int32, device="cuda"))
    assert (y[:2] == 0).all()


# ---- streams, graphs, together -------------------------------------------------

def test_other_stream_and_graph():
    """The calls follow the current stream, and a captured graph replays them on new inputs."""
    k = make(2, 64, 40, 16, 1, F32)
    c = cuda(k)
    dy, df = (v.cuda() for v in grads_like(k))
    want, grads = gpu_scan(c), gpu_scan_bwd(c, dy, df)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = gpu_scan(c)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros_like(c["x"])
    with torch.cuda.graph(graph):
        y = gpu_scan({**c, "x": x})
        g = gpu_scan_bwd({**c, "x": x}, dy, df)
    x.copy_(c["x"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    assert all(torch.equal(g[n], grads[n]) for n in grads)


def test_example_runs_them_together():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_block.py")
    spec = importlib.util.spec_from_file_location("selective_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    drift, losses = m.main()
    # bf16 activations: a few roundings of 2^-8 each per layer apart
    assert drift < 4 * 2.0 ** -8
    assert losses[-1] < losses[0]


@pytest.mark.parametrize("shape", [(1, 700, 96), (4, 130, 4096), (2, 65, 33)])
@pytest.mark.parametrize("name", ["x", "dt", "z"])
def test_scan_over_its_own_input(shape, name):
    gen = torch.Generator(device="cuda").manual_seed(3)
    B, L, D = shape
    t = {n: torch.randn(shape, generator=gen, device="cuda").bfloat16() for n in ("x", "dt", "z")}
    A = -torch.rand(D, 16, generator=gen, device="cuda")
    bc = [torch.randn(B, L, 1, 16, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    want = ssd().selective_scan(t["x"], t["dt"], A, *bc, dt_softplus=True, z=t["z"])
    got = ssd().selective_scan(t["x"], t["dt"], A, *bc, dt_softplus=True, z=t["z"], out=t[name])
    assert got.data_ptr() == t[name].data_ptr()
    assert torch.equal(got, want)


def test_conv_refuses_its_own_input_as_output():
    x = torch.randn(2, 40, 64, device="cuda")
    with pytest.raises(Exception, match="overlap"):
        ssd().causal_conv1d_carry(x, torch.ones(64, 4, device="cuda"), out=x)
