"""The selective scan where it is cut into segments with ragged rows, where its
grid fills the GPU, and where its tensors are strided, mixed or in place."""
import ctypes
import math

import pytest
import torch

import _selective_ref as ref
from _selective_ref import close, of
from test_gpu_selective import BF16, F16, F32, GRADS, cuda, gpu_scan, gpu_scan_bwd, grads_like, make, poison, ref_scan, ref_scan_bwd, ssd

pytestmark = pytest.mark.gpu


def is_cut(k):
    """Whether the forward walks segments of this problem (its workspace holds their states)."""
    c, size = cuda(k), ctypes.c_size_t()
    a = ssd().make_scan_args(c["x"], c["dt"], c["A"], c["B"], c["C"], z=c["z"])
    assert ssd().load_library().ssd_selective_scan_workspace_size(ctypes.byref(a), ctypes.byref(size)) == 0
    return size.value > 0


CUT = (3, 400, 64, 16, 1)
ENDS = [400, 0, 37]  # a whole row, an empty one, one that ends inside an early segment


def cut_case(t, **opts):
    k = make(*CUT, t, **opts)
    k["lengths"] = torch.tensor(ENDS, dtype=torch.int32)
    assert is_cut(k)
    return k


@pytest.mark.parametrize("opts", [dict(), dict(z=False), dict(dt32=True), dict(h0=False, skip=False)])
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_cut_ragged_scan(t, opts):
    k = cut_case(t, **opts)
    y, fin = gpu_scan(cuda(k))
    ry, rfin = ref_scan(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    for b, e in enumerate(ENDS):
        assert (y[b, e:] == 0).all()


@pytest.mark.parametrize("opts", [dict(), dict(z=False), dict(dt32=True), dict(h0=False, skip=False)])
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_cut_ragged_gradients(t, opts):
    k = cut_case(t, **opts)
    dy, df = grads_like(k)
    got = gpu_scan_bwd(cuda(k), dy.cuda(), df.cuda())
    for n, r in ref_scan_bwd(k, dy, df).items():
        if n in got:
            close(got[n], r, n)
    for n in ("dx", "ddt", "dB", "dC"):
        for b, e in enumerate(ENDS):
            assert (got[n][b, e:] == 0).all(), n


@pytest.mark.parametrize("t", [F32, BF16])
def test_cut_padding_does_not_leak(t):
    k = cut_case(t)
    dy, df = grads_like(k)
    bad = {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in k.items()}
    bad["dy"] = dy.clone()
    poison(bad, ["x", "dt", "z", "B", "C", "dy"])
    a, b = gpu_scan(cuda(k)), gpu_scan(cuda(bad))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    p, q = gpu_scan_bwd(cuda(k), dy.cuda(), df.cuda()), gpu_scan_bwd(cuda(bad), bad["dy"].cuda(), df.cuda())
    assert all(torch.equal(p[n], q[n]) for n in p)


def on_gpu(k):
    """The plain form's inputs, in 64 bits where the tensors are."""
    return {n: v.double() if isinstance(v, torch.Tensor) and n != "lengths" else v for n, v in k.items()}


def plain_scan(x, dt, A, B, C, D, z, dt_bias, h0):
    with torch.device("cuda"):  # where the plain form makes its own tensors
        return ref.scan(x, dt, A, B, C, D, z, dt_bias, h0)


# channel tiles for every SM and more, whole and odd ones; two groups
FULL = [(8, 40, 4096, 16, 1, BF16), (5, 33, 4098, 16, 2, BF16), (4, 24, 8192, 8, 1, F16), (8, 20, 1024, 64, 1, F32)]


@pytest.mark.parametrize("B,L,D,N,G,t", FULL)
def test_full_grid(B, L, D, N, G, t):
    k = cuda(make(B, L, D, N, G, t))
    f = on_gpu(k)
    y, fin = gpu_scan(k)
    ry, rfin = plain_scan(*(f[n] for n in GRADS))
    close(y, ry, "y")
    close(fin, rfin, "final state")


@pytest.mark.parametrize("B,L,D,N,G,t", FULL)
def test_full_grid_gradients(B, L, D, N, G, t):
    k = cuda(make(B, L, D, N, G, t))
    dy, df = (v.cuda() for v in grads_like(k))
    got = gpu_scan_bwd(k, dy, df)
    want = ref.gradients(plain_scan, {n: on_gpu(k)[n] for n in GRADS}, [dy.double(), df.double()])
    for n, r in want.items():
        close(got[GRADS[n]], r, GRADS[n])


@pytest.mark.parametrize("N", [12, 20, 32, 64, 128])
def test_step_of_many_sequences(N):
    """Four sequences per lane at every number of lanes, the last block of rows not full."""
    B, D = 22, 8192 if N < 32 else 4096
    k = cuda(make(B, 1, D, N, 2, BF16))
    pool, slots = torch.zeros((B + 3, D, N), device="cuda"), torch.randperm(B + 3)[:B].to(torch.int32).cuda()
    pool[slots.long()] = k["h0"]
    slots[4] = -1
    before = pool.clone()
    y = ssd().selective_scan_step(k["x"][:, 0], k["dt"][:, 0], k["A"], k["B"][:, 0], k["C"][:, 0], pool, True, slots=slots,
                                  D=k["D"], z=k["z"][:, 0], dt_bias=k["dt_bias"])
    f = on_gpu(k)
    ry, rfin = plain_scan(*(f[n] for n in GRADS))
    live = [b for b in range(B) if b != 4]
    close(y[live], ry[live, 0], "y")
    close(pool[slots[live].long()], rfin[live], "states")
    assert (y[4] == 0).all()
    rest = [s for s in range(B + 3) if s not in slots[live].tolist()]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("t", [F16, BF16])
def test_wide_steps_of_strided_inputs(t, offset):
    """dt in fp32 as a slice of its own projection, beside 16-bit slices; forward and backward."""
    k = cuda(make(2, 30, 48, 16, 1, t, dt32=True))
    wide = torch.randn((2, 30, 48 * 2 + 32 + 24 + offset), device="cuda").to(t)
    steps = torch.randn((2, 30, 48 + 7 + offset), device="cuda")
    cut, at = dict(k), offset
    for n, width in (("x", 48), ("z", 48), ("B", 16), ("C", 16)):
        part = wide[..., at:at + width]
        part.copy_(k[n].reshape(2, 30, width))
        cut[n] = part.unsqueeze(2) if n in "BC" else part
        at += width
    cut["dt"] = steps[..., offset:offset + 48]
    cut["dt"].copy_(k["dt"])
    ry, rfin = ref_scan({n: v.cpu() if isinstance(v, torch.Tensor) else v for n, v in k.items()})
    y, fin = gpu_scan(cut)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    dy, df = grads_like(k)
    got = gpu_scan_bwd(cut, dy.cuda(), df.cuda())
    for n, r in ref_scan_bwd(k, dy, df).items():
        close(got[n], r, n)


@pytest.mark.parametrize("shape", [(1, 700, 96), (2, 65, 33)])
@pytest.mark.parametrize("name", ["x", "dt", "z"])
@pytest.mark.parametrize("t", [F32, F16])
def test_scan_over_its_own_input_in_other_types(shape, name, t):
    gen = torch.Generator(device="cuda").manual_seed(3)
    B, L, D = shape
    k = {n: torch.randn(shape, generator=gen, device="cuda").to(t) for n in ("x", "dt", "z")}
    A = -torch.rand(D, 16, generator=gen, device="cuda")
    bc = [torch.randn(B, L, 1, 16, generator=gen, device="cuda").to(t) for _ in range(2)]
    want = ssd().selective_scan(k["x"], k["dt"], A, *bc, dt_softplus=True, z=k["z"])
    got = ssd().selective_scan(k["x"], k["dt"], A, *bc, dt_softplus=True, z=k["z"], out=k[name])
    assert got.data_ptr() == k[name].data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("name", ["x", "dt", "z"])
@pytest.mark.parametrize("B", [3, 130])
def test_steps_over_their_own_inputs(B, name):
    D = 41 if B == 3 else 2048
    k = cuda(make(B, 1, D, 16, 1, BF16))
    t = {n: k[n][:, 0].clone() for n in ("x", "dt", "z")}
    f = dict(D=k["D"], dt_bias=k["dt_bias"])
    want = ssd().selective_scan_step(t["x"], t["dt"], k["A"], k["B"][:, 0], k["C"][:, 0], k["h0"].clone(), True, z=t["z"], **f)
    got = ssd().selective_scan_step(t["x"], t["dt"], k["A"], k["B"][:, 0], k["C"][:, 0], k["h0"].clone(), True, z=t["z"], out=t[name], **f)
    assert got.data_ptr() == t[name].data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 2047, 2048])
@pytest.mark.parametrize("where", ["r", "o", "gate", "stream"])
def test_norm_over_its_own_inputs(D, where):
    """n or r' in the place of an input of its type, at rows of odd and of even width."""
    rows = 900
    o, r, g = (torch.randn(rows, D, device="cuda").to(BF16) for _ in range(3))
    w, s = 1 + 0.1 * torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    f = dict(w_post=w, scale=s)
    want = ssd().block_norm(o, r, w, gate=g, **f)
    kw = {"r": dict(r_out=r), "o": dict(out=o), "gate": dict(out=g), "stream": dict(out=r, r_out=o)}[where]
    got = ssd().block_norm(o, r, w, gate=g, **f, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_gradients_of_many_gates():
    """More gates of whole sequences than threads of a column in the sums."""
    from test_gpu_block_norm import check_bwd, make as make_norm
    check_bwd(make_norm((150, 3), 264, BF16, F32, "sequence"), BF16, F32)
    check_bwd(make_norm((70, 2), 33, F32, F32, "sequence"), F32, F32)


def test_norm_gradients_of_wide_rows():
    from test_gpu_block_norm import check_bwd, make as make_norm
    check_bwd(make_norm((40, 3), 10240, BF16, BF16, "token"), BF16, BF16)
    check_bwd(make_norm((9, 5), 12289, F16, F32, "sequence"), F16, F32)


def test_conv_gradients_on_a_full_grid():
    g = torch.Generator(device="cuda").manual_seed(6)
    B, L, C, W = 3, 500, 4100, 4
    x, dy = (torch.randn((B, L, C), generator=g, device="cuda").to(BF16) for _ in range(2))
    w, bias = torch.randn((C, W), generator=g, device="cuda") * 0.5, torch.randn(C, generator=g, device="cuda")
    got = ssd().causal_conv1d_bwd(x, w, dy, bias)

    def plain(x, w, bias):
        v = torch.nn.functional.pad(x, (0, 0, W - 1, 0))
        a = bias + sum(w[:, k] * v[:, k:k + L] for k in range(W))
        return (a * torch.sigmoid(a),)
    want = ref.gradients(plain, {"x": x.double(), "w": w.double(), "bias": bias.double()}, [dy.double()])
    for n, r in want.items():
        close(got["d" + n], r, "d" + n)


@pytest.mark.parametrize("t", [F32, BF16])
def test_one_token_for_every_sequence(t):
    """Rows of one token, shared by the batch: the batch stride is 0 and there is no other token."""
    k = cuda(make(3, 1, 40, 16, 2, t))
    for n in ("x", "dt", "z", "B", "C"):
        k[n] = k[n][:1].expand(k[n].shape)
    dense = {n: v.contiguous() if isinstance(v, torch.Tensor) else v for n, v in k.items()}
    a, b = gpu_scan(k), gpu_scan(dense)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dy, df = (v.cuda() for v in grads_like(dense))
    p, q = gpu_scan_bwd(k, dy, df), gpu_scan_bwd(dense, dy, df)
    assert all(torch.equal(p[n], q[n]) for n in p)
    w = torch.randn(40, 4, device="cuda")
    assert torch.equal(ssd().causal_conv1d_carry(k["x"], w), ssd().causal_conv1d_carry(dense["x"], w))
    sa = ssd().make_scan_args(k["x"], k["dt"], k["A"], k["B"], k["C"])
    assert sa.x_stride[0] == 0 and sa.x_stride[1] > 0 and math.isinf(sa.dt_max)
