"""GPU parity of the norm of queries and keys with its rotation, forward and backward,
against the plain 64-bit form."""
import pytest
import torch

import _delta_ref as ref
from _selective_ref import close, of

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def ssd():
    import mamba_ssd_chunked_fwd_gb300 as m
    return m


def make(B, L, H, G, N, R, t, *, w=True, far=0, seed=0):
    g = torch.Generator().manual_seed(100 * seed + B + 3 * L + 5 * H + 7 * N + R)
    k = dict(q=(torch.randn((B, L, H, N), generator=g) * 2).to(t), k=(torch.randn((B, L, G, N), generator=g) * 2).to(t),
             w_q=1 + 0.2 * torch.randn(N, generator=g) if w else None, w_k=1 + 0.2 * torch.randn(N, generator=g) if w else None,
             freqs=10000.0 ** (-torch.arange(R) / max(R, 1)) if R else None, positions=None)
    if far:
        k["positions"] = (far + torch.randint(0, 1000, (B, L), generator=g)).to(torch.int32)
    return k


def cuda(k):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in k.items()}


def plain(k, **how):
    f = {n: of(v) if n != "positions" else v for n, v in k.items()}
    return ref.qk_norm(**f, **how)


# one element; odd widths; quads that end inside a lane's run; part of a head turned; wide heads
SHAPES = [(1, 1, 1, 1, 1, 0), (2, 3, 2, 1, 2, 1), (1, 5, 3, 2, 7, 3), (2, 9, 4, 2, 64, 32), (1, 17, 5, 5, 128, 64), (2, 11, 8, 2, 128, 32),
          (1, 13, 3, 1, 100, 50), (1, 6, 2, 2, 100, 12), (1, 4, 2, 1, 40, 20), (1, 8, 1, 1, 256, 128), (2, 5, 3, 1, 200, 96), (1, 3, 2, 1, 255, 127),
          (1, 700, 2, 1, 12, 4)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("how", [dict(), dict(norm="l2", interleaved=True)])
def test_norm(shape, t, how):
    k = make(*shape, t, far=5000)
    for got, want in zip(ssd().qk_norm(**cuda(k), **how), plain(k, **how)):
        assert got.dtype == t and got.is_contiguous()
        close(got, want)


@pytest.mark.parametrize("opts", [dict(w=False), dict(far=1000000), dict(far=-300), dict(far=2 ** 31 - 2000), dict()])
@pytest.mark.parametrize("interleaved", [False, True])
def test_options(opts, interleaved):
    """Positions of up to 2^31: an angle is off by 2^-52 of position * freq, 5e-7 at most."""
    k = make(2, 21, 4, 2, 128, 48, F32, **opts)
    for got, want in zip(ssd().qk_norm(**cuda(k), interleaved=interleaved), plain(k, interleaved=interleaved)):
        close(got, want)


def test_eps_and_zero_vectors():
    k = make(1, 4, 2, 1, 64, 32, F32)
    k["q"][0, 1] = 0
    k["k"][0, 2] *= 1e-6
    for norm in ("rms", "l2"):
        for got, want in zip(ssd().qk_norm(**cuda(k), norm=norm, eps=1e-3), plain(k, norm=norm, eps=1e-3)):
            close(got, want)


def bwd(k, t, how):
    g = torch.Generator().manual_seed(8)
    dq, dk = (torch.randn(k[n].shape, generator=g).to(t) for n in ("q", "k"))
    got = ssd().qk_norm_bwd(dq.cuda(), dk.cuda(), **cuda(k), **how)
    names = [n for n in ("q", "k", "w_q", "w_k") if k[n] is not None]
    leaves = {n: of(k[n]).requires_grad_(True) for n in names}
    outs = ref.qk_norm(leaves["q"], leaves["k"], leaves.get("w_q"), leaves.get("w_k"), freqs=of(k["freqs"]), positions=k["positions"], **how)
    loss = (outs[0] * of(dq)).sum() + (outs[1] * of(dk)).sum()
    want = dict(zip(["d" + n for n in names], torch.autograd.grad(loss, list(leaves.values()))))
    assert set(got) == set(want)
    return got, want


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("how", [dict(), dict(norm="l2", interleaved=True)])
def test_gradients(shape, t, how):
    """A head of one element under eps = 1e-6 has a gradient of 1e-6 times its values, the rest of
    two terms that cancel: the bound there is one of the terms."""
    if shape[4] == 1:
        how = dict(how, eps=0.5)
    k = make(*shape, t, far=5000)
    got, want = bwd(k, t, how)
    for n in got:
        close(got[n], want[n], n)


def test_gradients_without_weights():
    k = make(2, 9, 4, 2, 64, 32, BF16, w=False)
    got, want = bwd(k, BF16, {})
    for n in got:
        close(got[n], want[n], n)
    k = make(2, 9, 4, 2, 64, 32, F32)
    k["w_q"] = None
    got, want = bwd(k, F32, {})
    for n in got:
        close(got[n], want[n], n)


@pytest.mark.parametrize("N,offset", [(128, 8), (128, 1), (64, 4), (20, 2)])
@pytest.mark.parametrize("t", [F32, BF16])
def test_strided_inputs(N, offset, t):
    k = cuda(make(2, 33, 4, 2, N, N // 2, t, far=100))
    wide = torch.full((2, 33, 6 * N + 2 * offset), float("nan"), device="cuda", dtype=t)
    s = dict(k)
    s["q"] = wide[..., offset:offset + 4 * N].unflatten(-1, (4, N)).copy_(k["q"])
    s["k"] = wide[..., offset + 4 * N + offset:].unflatten(-1, (2, N)).copy_(k["k"])
    for a, b in zip(ssd().qk_norm(**s), ssd().qk_norm(**k)):
        close(a, b.double())  # another path may add in another order
    dq, dk = torch.randn_like(k["q"]), torch.randn_like(k["k"])
    a, b = ssd().qk_norm_bwd(dq, dk, **s), ssd().qk_norm_bwd(dq, dk, **k)
    for n in a:
        close(a[n], b[n].double(), n)


@pytest.mark.parametrize("N", [128, 36])
def test_in_place(N):
    k = cuda(make(2, 40, 4, 2, N, N // 4, BF16))
    want = ssd().qk_norm(**k)
    got = ssd().qk_norm(**k, out_q=k["q"], out_k=k["k"])
    assert got[0].data_ptr() == k["q"].data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("B", [1, 5, 300])
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_single_tokens(B, t):
    k = make(B, 1, 8, 2, 128, 32, t, far=70000)
    one = {n: v[:, 0] if n in ("q", "k", "positions") else v for n, v in cuda(k).items()}
    for got, want in zip(ssd().qk_norm(**one), plain(k)):
        close(got, want[:, 0])
    wide = torch.zeros((B, 20, 128), device="cuda", dtype=t)
    one["q"], one["k"] = wide[:, :8].copy_(one["q"]), wide[:, 9:11].copy_(one["k"])
    for got, want in zip(ssd().qk_norm(**one), plain(k)):
        close(got, want[:, 0])


def test_many_rows():
    """More tiles than CTAs in the backward, a last tile that is not whole."""
    k = make(3, 4001, 3, 1, 32, 16, F32)
    got, want = bwd(k, F32, {})
    for n in got:
        close(got[n], want[n], n)
    for a, b in zip(ssd().qk_norm(**cuda(k)), plain(k)):
        close(a, b)


def test_deterministic_stream_and_graph():
    k = cuda(make(2, 500, 8, 2, 128, 64, BF16))
    dq, dk = torch.randn_like(k["q"]), torch.randn_like(k["k"])
    want, wantb = ssd().qk_norm(**k), ssd().qk_norm_bwd(dq, dk, **k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gotb = ssd().qk_norm(**k), ssd().qk_norm_bwd(dq, dk, **k)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(gotb[n], wantb[n]) for n in wantb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, gotb = ssd().qk_norm(**k), ssd().qk_norm_bwd(dq, dk, **k)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(gotb[n], wantb[n]) for n in wantb)
