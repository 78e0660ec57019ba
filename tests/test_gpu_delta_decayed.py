"""fp16 and bf16 in chunks where gates shrink what is carried far below what is beside it: the state after a chunk against the one before it,
its adjoint against dy.  Against the plain 64-bit form, each result by itself."""
import pytest
import torch

from _selective_ref import REL
from test_gpu_delta import BF16, F16, F32, cuda, gpu, gpu_bwd, make, plain, plain_bwd
from test_gpu_delta_range import STEP, grads
from test_gpu_delta_range import near as near_f16

pytestmark = pytest.mark.gpu


def near(got, want, what, t):
    """fp16's operands keep 2^-22 of a value, and its results in 32 bits the library's bound.  bf16's keep it to half a step of
    its second term, 2^-8 of what 2^-8 of it leaves: 2^-16; a sum of products of two of them 2^-15 of the products' sizes."""
    if t == BF16 and got.dtype == F32:
        error = (got.double().cpu() - want).norm() / want.norm()
        assert error <= 2.0 ** -15, (what, error.item())
    else:
        near_f16(got, want, what)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("g", [-5.0, -9.0])
@pytest.mark.parametrize("shape", [(1, 22, 1, 1, 40, 200), (2, 65, 2, 1, 128, 128), (1, 17, 3, 3, 64, 72)])
def test_first_token_decays(shape, g, t):
    """dh0 is e^g of what dy gives the other tokens."""
    k = make(*shape, t, b32=True)
    k["g"] = k["g"].clamp(min=-0.5)
    k["g"][:, 0] = g
    dy, df = grads(k, 1e-2)
    dy = dy.to(t)
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n in got:
        near(got[n], want[n], n, t)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("at", [0, 20, 63, 64])
def test_adjoint_through_a_decay(at, t):
    """dy at the last tokens alone, and one gate of e^-9 in the chunks before."""
    k = make(1, 200, 2, 2, 128, 128, t, b32=True)
    k["g"] = torch.full_like(k["g"], -0.01)
    k["g"][:, at] = -9.0
    dy, df = grads(k, 1.0)
    dy = dy.to(t)
    dy[:, :-30] = 0
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n in got:
        near(got[n], want[n], n, t)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("at", [0, 128, 150, 191, 199])
def test_state_after_a_decay(at, t):
    """A gate of e^-9 in the last chunks, and nothing but small betas from there on: what is left of the state is small."""
    k = make(1, 200, 2, 2, 128, 128, t, b32=True)
    k["g"] = torch.full_like(k["g"], -0.01)
    k["g"][:, at] = -9.0
    k["beta"][:, at:] *= 1e-3
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    near(y, ry, "y", t)
    near(fin, rfin, "final state", t)


@pytest.mark.parametrize("t", [F16, BF16])
def test_state_far_above_the_values(t):
    """An initial state of 1000 times the values, shrunk to their size within a chunk."""
    k = make(1, 130, 2, 2, 128, 128, t)
    k["h0"] = k["h0"] * 1000
    k["g"] = torch.full_like(k["g"], -0.01)
    k["g"][:, 40] = -7.0
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    near(y, ry, "y", t)
    near(fin, rfin, "final state", t)


def test_expanding_steps(t=F16):
    """Keys of length 1.5, alike, and beta 1: a token turns what it finds under its key into -1.25 times that, and T passes the 8
    that its operand is laid out for.  A rounding of the first tokens grows as their values do.
    (bf16's terms need no powers of two, and T has no second pass there.)"""
    k = make(1, 24, 2, 1, 64, 64, t, b32=True)
    one = torch.zeros(64)
    one[::4] = 0.375  # 16 of them: length 1.5, exact
    k["k"] = one.to(t).expand_as(k["k"]).contiguous()
    k["beta"], k["g"] = torch.ones_like(k["beta"]), torch.zeros_like(k["g"])
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    assert rfin.abs().max() > 50
    near(y, ry, "y", t)
    near(fin, rfin, "final state", t)
    dy, df = grads(k, 1.0)
    dy = dy.to(t)
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n in got:
        near(got[n], want[n], n, t)


@pytest.mark.parametrize("length,beta", [(1.0, 2.0), (32.0, 2.0 ** -9), (0.03125, 2048.0)])
def test_values_that_add_up(length, beta):
    """Keys alike, values of alternating signs, and beta |k|^2 of 2: every token adds to the ones before it or cancels them, up to
    127 values in u.  Long keys with small betas, and short ones with large.  A result may be 130 terms' difference, and off by
    130 times what one of them is (in fp32, token by token, up to 3e-5 is measured)."""
    k = make(1, 130, 2, 2, 64, 64, F16, b32=True, h0=False)
    one = torch.zeros(64)
    one[::4] = 0.25 * length  # 16 of them
    k["k"] = one.to(F16).expand_as(k["k"]).contiguous()
    k["q"] = k["k"].clone()
    k["v"] = (k["v"][:, :1].float().abs() * (1 - 2 * (torch.arange(130) % 2).float())[None, :, None, None]).to(F16)
    k["beta"], k["g"] = torch.full_like(k["beta"], beta), torch.full_like(k["g"], -1e-3)
    scale = 1.0 / (16 * length ** 2)
    dy, df = grads(k, 1e-3)  # dk of the short keys is up to 24000
    (y, fin), (ry, rfin) = gpu(cuda(k), scale=scale), plain(k, scale)
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda(), scale=scale), plain_bwd(k, dy, df, scale)
    for n, a, b in [("y", y, ry), ("final", fin, rfin)] + [(n, got[n], want[n]) for n in got]:
        half, step = (2.0 ** -11, STEP * b.numel() ** 0.5) if a.dtype == F16 else (0.0, 0.0)
        a = a.double().cpu()
        assert torch.isfinite(a).all(), n
        assert (a - b).norm() <= (half + 130 * REL) * b.norm() + step, (n, ((a - b).norm() / b.norm()).item())
