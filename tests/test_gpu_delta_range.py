"""fp16 tensors of the gated delta rule over the range of their values.  Everything the forward gives is linear in
(v, h0), every gradient in (dy, dfinal): results keep their precision whatever the size of those, and large ones
stay finite where the results do.  Against the plain 64-bit form."""
import pytest
import torch

from _selective_ref import close
from test_gpu_delta import F16, F32, NAMES, cuda, gpu, gpu_bwd, make, plain, plain_bwd

pytestmark = pytest.mark.gpu

# whole tiles, part of them, a narrow head, rows over two tiles of 128, shared keys with a cut row
SHAPES = [(2, 150, 2, 2, 128, 128), (1, 130, 4, 2, 64, 64), (1, 100, 2, 1, 96, 40), (1, 200, 2, 2, 128, 200)]


def grads(k, s, seed=9):
    gen = torch.Generator().manual_seed(seed)
    dy = (torch.randn(k["v"].shape, generator=gen) * s).to(k["v"].dtype)
    B, _, H, P = k["v"].shape
    return dy, torch.randn((B, H, P, k["q"].shape[-1]), generator=gen) * s


# A result in fp16 below 2^-14 has steps of 2^-24, half of which it may be off by, whatever its size.
STEP = 2.0 ** -25


def near(got, want, what):
    """As `close`, with fp16's smallest steps."""
    if got.dtype == F16:
        got64, want = got.double().cpu(), want.double()
        assert torch.isfinite(got64).all(), what
        diff, norm = (got64 - want).norm().item(), want.norm().item()
        assert diff <= (2.0 ** -11 + 1e-5) * norm + STEP * want.numel() ** 0.5, (what, diff / max(norm, 1e-300))
        assert ((got64 - want).abs() <= 2.0 ** -11 * want.abs() + 1e-4 * want.abs().max() + STEP).all(), what
    else:
        close(got, want, what)


def values(k, s):
    k["v"] = (k["v"].float() * s).to(F16)
    if k["h0"] is not None:
        k["h0"] = k["h0"] * s
    return k


@pytest.mark.parametrize("s", [1e-2, 1e-3, 1e-4, 1e-5, 1e3])
@pytest.mark.parametrize("shape", SHAPES + [(1, 1300, 2, 1, 128, 128)])
def test_sizes_of_values(shape, s):
    k = values(make(*shape, F16), s)
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    near(y, ry, "y")
    near(fin, rfin, "final state")


@pytest.mark.parametrize("s", [1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 1e3])
@pytest.mark.parametrize("shape", SHAPES)
def test_sizes_of_incoming_gradients(shape, s):
    """g and beta in fp32, so that their gradients and dh0 are."""
    k = make(*shape, F16, b32=True)
    dy, df = grads(k, s)
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    assert got["dg"].dtype == got["dbeta"].dtype == got["dh0"].dtype == F32
    for n in got:
        near(got[n], want[n], n)


@pytest.mark.parametrize("s", [1e-3, 1e3])
def test_sizes_of_both(s):
    k = values(make(2, 150, 4, 2, 128, 128, F16, b32=True), s)
    dy, df = grads(k, 1e-4 / s)
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n in got:
        near(got[n], want[n], n)


def test_unlike_rows():
    """One row of the state a thousand times the others: each of the results for itself, row by row."""
    k = make(1, 200, 2, 2, 128, 128, F16)
    k["v"][..., 5] *= 1000
    k["h0"][..., 5, :] *= 1000
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    for p in (4, 5, 6, 127):
        near(y[..., p], ry[..., p], f"y, row {p}")
        near(fin[:, :, p], rfin[:, :, p], f"state, row {p}")


def test_tiles_of_unlike_size():
    """The rows' two tiles of 128 differ by 2^6 in v and, the other way round, in dy.  What a chunk computes is held to about
    2^-26 of its largest value: of the smaller tile's, 2^-20."""
    k = make(1, 150, 2, 2, 128, 200, F16, b32=True)
    k["v"][..., 128:] *= 2.0 ** -6
    k["h0"][..., 128:, :] *= 2.0 ** -6
    dy, df = grads(k, 1.0)
    dy[..., :128] *= 2.0 ** -6
    df[..., :128, :] *= 2.0 ** -6
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n in got:
        near(got[n], want[n], n)


def test_far_adjoint():
    """What is left of dy at the last tokens after a thousand: a small part of what it was."""
    k = make(1, 1000, 1, 1, 128, 128, F16, b32=True)
    k["g"] = torch.full_like(k["g"], -0.008)
    dy, df = grads(k, 1.0)
    dy[:, :-64] = 0
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    assert want["dh0"].norm() < 1e-3 * df.norm()
    for n in got:
        near(got[n], want[n], n)
    first = slice(0, 300)  # gradients of early tokens by themselves
    for n in ("dg", "dbeta"):
        near(got[n][:, first], want[n][:, first], n)


@pytest.mark.parametrize("s", [1e-2, 1e-4])
def test_small_betas(s):
    k = make(1, 200, 2, 2, 128, 128, F16, b32=True, h0=False)
    k["beta"] = k["beta"] * s
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    near(y, ry, "y")
    near(fin, rfin, "final state")
    dy, df = grads(k, 1.0)
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n in got:
        near(got[n], want[n], n)


@pytest.mark.parametrize("s", [1e-3, 60.0])
def test_sizes_of_queries(s):
    """60: products q . k of up to 60, dy M^T and D accordingly."""
    k = make(1, 150, 2, 2, 128, 128, F16, b32=True)
    k["q"] = (k["q"].float() * s).to(F16)
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    near(y, ry, "y")
    near(fin, rfin, "final state")
    dy, df = grads(k, 1.0)
    df = df * 0
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n in got:
        near(got[n], want[n], n)


def test_an_infinity_stays_in_its_row():
    """An infinite value leaves the other rows of the state what they are."""
    k = make(1, 150, 2, 2, 128, 128, F16)
    want = gpu(cuda(k))
    k["v"][0, 70, :, 9] = float("inf")
    got = gpu(cuda(k))
    rest = [p for p in range(128) if p != 9]
    assert torch.equal(got[0][..., rest], want[0][..., rest])
    assert torch.equal(got[1][:, :, rest], want[1][:, :, rest])
    assert not torch.isfinite(got[1][:, :, 9]).any()
    dy, df = grads(k, 1.0)
    k["v"] = torch.zeros_like(k["v"])
    ref = plain_bwd(k, dy, df)
    dy[0, 70, :, 9] = float("inf")
    dv = gpu_bwd(cuda(k), dy.cuda(), df.cuda())["dv"]
    near(dv[..., rest], ref["dv"][..., rest], "dv")


def test_wide_range_is_deterministic():
    k = cuda(values(make(2, 300, 2, 1, 128, 200, F16), 1e-3))
    dy, df = grads(k, 1e-4)
    a, b = (gpu_bwd(k, dy.cuda(), df.cuda()) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    assert all(torch.equal(x, y) for x, y in zip(gpu(k), gpu(k)))
    assert set(NAMES) < set(k)
