"""GPU parity of the block norm and its backward against the plain 64-bit form."""
import pytest
import torch

import _selective_ref as ref
from _selective_ref import close, of

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def ssd():
    import mamba_ssd_chunked_fwd_gb300 as m
    return m


def make(lead, D, t, q, gate, *, post=True, scale=True, o=True, seed=0):
    g = torch.Generator().manual_seed(seed + D + sum(lead))

    def normal(*shape, s=1.0, dt=t):
        return (torch.randn(shape, generator=g) * s).to(dt)
    k = dict(o=normal(*lead, D) if o else None, r=normal(*lead, D, s=2.0, dt=q), w_pre=1 + 0.1 * normal(D, dt=F32),
             w_post=1 + 0.1 * normal(D, dt=F32) if post and o else None, scale=0.5 + 0.1 * normal(D, dt=F32) if scale and o else None,
             gate=None)
    if o and gate == "sequence":
        k["gate"] = normal(lead[0], D)
    elif o and gate == "token":
        k["gate"] = normal(*lead, D)
    return k


def cuda(k):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in k.items()}


def check_fwd(k, n, r_out, t, q):
    rn, rr = ref.norm(of(k["o"]), of(k["r"]), of(k["w_pre"]), of(k["w_post"]), of(k["gate"]), of(k["scale"]))
    close(r_out, rr, "r'")
    # n is of the rounded r'
    rn, _ = ref.norm(None, of(r_out), of(k["w_pre"]))
    close(n, rn, "n")


# a single element; rows a warp takes, rows of several, odd ones; the widest
WIDTHS = [1, 5, 64, 100, 256, 258, 520, 1000, 2048, 2050, 4100, 8192, 9000, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("t,q", [(F32, F32), (BF16, F32), (F16, F16)])
def test_block_norm(D, t, q):
    for lead, gate in (((3,), "none"), ((2, 5), "sequence"), ((2, 3), "token")):
        k = make(lead, D, t, q, gate)
        c = cuda(k)
        n, r = ssd().block_norm(c["o"], c["r"], c["w_pre"], w_post=c["w_post"], gate=c["gate"], scale=c["scale"])
        assert n.dtype == t and r.dtype == q
        check_fwd(k, n, r, t, q)


@pytest.mark.parametrize("opts", [dict(post=False), dict(scale=False), dict(o=False), dict(post=False, scale=False)])
@pytest.mark.parametrize("D", [6, 300, 3001])
def test_block_norm_options(D, opts):
    k = make((2, 4), D, BF16, F32, "none", **opts)
    c = cuda(k)
    n, r = ssd().block_norm(c["o"], c["r"], c["w_pre"], w_post=c["w_post"], gate=c["gate"], scale=c["scale"], dtype=BF16)
    check_fwd(k, n, r, BF16, F32)
    if k["o"] is None:
        assert r is c["r"]


def test_block_norm_in_place_and_many_rows():
    k = make((7, 301), 264, BF16, F32, "sequence")
    c = cuda(k)
    want = ssd().block_norm(c["o"], c["r"], c["w_pre"], w_post=c["w_post"], gate=c["gate"], scale=c["scale"])
    check_fwd(k, *want, BF16, F32)
    r = c["r"].clone()
    got = ssd().block_norm(c["o"], r, c["w_pre"], w_post=c["w_post"], gate=c["gate"], scale=c["scale"], r_out=r)
    assert got[1] is r and torch.equal(got[0], want[0]) and torch.equal(r, want[1])


def ref_bwd(k, dn, dr_out, r_out):
    """Around the stored r': it enters as a value of its own, the branch as its change."""
    def f(o, r_out, w_pre, w_post, gate, scale):
        r_new = r_out
        if o is not None:
            branch = ref.norm(o, torch.zeros_like(r_out), w_pre, w_post, gate, scale)[1]
            r_new = r_out + branch - branch.detach()
        return ref.norm(None, r_new, w_pre)[0], r_new
    names = {"o": "do", "r_out": "dr", "w_pre": "dw_pre", "w_post": "dw_post", "gate": "dgate", "scale": "dscale"}
    inputs = {n: of(k[n]) for n in ("o", "w_pre", "w_post", "gate", "scale")}
    inputs["r_out"] = of(r_out)
    got = ref.gradients(f, {n: inputs[n] for n in names}, [of(dn), of(dr_out)])
    return {names[n]: v for n, v in got.items()}


def check_bwd(k, t, q, with_dr=True, seed=1):
    c = cuda(k)
    _, r_out = ssd().block_norm(c["o"], c["r"], c["w_pre"], w_post=c["w_post"], gate=c["gate"], scale=c["scale"], dtype=t)
    g = torch.Generator().manual_seed(seed)
    dn = torch.randn(k["r"].shape, generator=g).to(t)
    dr = torch.randn(k["r"].shape, generator=g).to(q) if with_dr else None
    got = ssd().block_norm_bwd(dn.cuda(), None if dr is None else dr.cuda(), c["o"], r_out, c["w_pre"], w_post=c["w_post"],
                               gate=c["gate"], scale=c["scale"])
    want = ref_bwd(k, dn, dr, r_out)
    assert set(got) == set(want)
    for n, v in want.items():
        close(got[n], v, n)
    return got


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("t,q", [(F32, F32), (BF16, F32), (F16, F16)])
def test_block_norm_bwd(D, t, q):
    if D == 1:
        pytest.skip("a row of one element: its norm is a sign, its gradient a difference of equal numbers")
    for lead, gate in (((3,), "none"), ((2, 5), "sequence"), ((2, 3), "token")):
        check_bwd(make(lead, D, t, q, gate), t, q)


@pytest.mark.parametrize("opts", [dict(post=False), dict(scale=False), dict(o=False), dict(post=False, scale=False)])
@pytest.mark.parametrize("D", [6, 300, 3001])
def test_block_norm_bwd_options(D, opts):
    check_bwd(make((2, 4), D, BF16, F32, "none", **opts), BF16, F32, with_dr=False)


@pytest.mark.parametrize("gate", ["none", "sequence", "token"])
def test_block_norm_bwd_many_rows(gate):
    """More rows than chunks; sequences that chunks divide unevenly."""
    a = check_bwd(make((3, 701), 264, BF16, F32, gate), BF16, F32)
    b = check_bwd(make((3, 701), 264, BF16, F32, gate), BF16, F32)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_block_norm_bwd_against_differences():
    k = make((2, 3), 40, F32, F32, "sequence")
    c = cuda(k)
    _, r_out = ssd().block_norm(c["o"], c["r"], c["w_pre"], w_post=c["w_post"], gate=c["gate"], scale=c["scale"])
    g = torch.Generator().manual_seed(2)
    dn, dr = torch.randn(k["r"].shape, generator=g), torch.randn(k["r"].shape, generator=g)
    got = ssd().block_norm_bwd(dn.cuda(), dr.cuda(), c["o"], r_out, c["w_pre"], w_post=c["w_post"], gate=c["gate"], scale=c["scale"])
    names = {"o": "do", "r": "dr", "w_pre": "dw_pre", "w_post": "dw_post", "gate": "dgate", "scale": "dscale"}
    for n, out in names.items():
        v, e = torch.randn(k[n].shape, generator=g, dtype=torch.float64), 1e-6

        def value(s):
            f = {m: of(k[m]) for m in names}
            f[n] = f[n] + s * e * v
            y, r = ref.norm(f["o"], f["r"], f["w_pre"], f["w_post"], f["gate"], f["scale"])
            return (y * of(dn)).sum() + (r * of(dr)).sum()
        slope = ((value(1) - value(-1)) / (2 * e)).item()
        mine = (got[out].double().cpu() * v).sum().item()
        assert abs(slope - mine) <= ref.REL * got[out].double().norm().item() * v.norm().item() + 1e-6 * abs(slope) + 1e-6, out
