"""The delta rule, the norm of queries and keys, the carried convolution and the block norm run together,
as a layer runs them: prompts, single tokens, gradients.  And their refusals of CUDA tensors."""
import os
import sys

import pytest
import torch

import _delta_ref as dref
import _selective_ref as sref
from _selective_ref import of
from test_gpu_delta import BF16, F16, F32, NAMES, cuda, make, ssd

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_runs():
    import delta_block
    drift, losses = delta_block.main(prompt=70, tokens=3)
    # bf16 layers: each rounding is off by at most 2^-8 of its value, and a dozen of them follow one another per layer
    assert drift < 24 * 2.0 ** -8
    assert all(v == v and v < float("inf") for v in losses)


def plain_stack(m, p_all, e):
    """The stack in 64 bits on the CPU, from its parameters."""
    d_model, heads, key_heads, d_key, d_value, _ = m.sizes
    n, r = sref.norm(None, e, of(m.norm))
    for p in p_all:
        x, _ = sref.conv(n @ p["in_proj"].t(), p["conv_w"], p["conv_b"])
        q, k, v = x.split([key_heads * d_key, key_heads * d_key, heads * d_value], -1)
        q, k = dref.qk_norm(q.unflatten(-1, (key_heads, d_key)), k.unflatten(-1, (key_heads, d_key)), norm="l2", freqs=of(m.freqs))
        ab = n @ p["gate_proj"].t()
        g = -torch.exp(p["A_log"]) * torch.nn.functional.softplus(ab[..., :heads] + p["dt_bias"], threshold=100)
        y, _ = dref.delta(q, k, v.unflatten(-1, (heads, d_value)), g, torch.sigmoid(ab[..., heads:]))
        n, r = sref.norm(y.flatten(-2) @ p["out_proj"].t(), r, p["w_pre"], p["w_post"], None, p["scale"])
    return n


def test_gradients_of_a_stack():
    """Every parameter's gradient in fp32 against the differentiated 64-bit form.  Projections are torch's fp32 products: a
    sum of n terms is off by n 2^-24 of their size at most, 128 terms here, and a dozen stages follow one another."""
    import delta_block
    m = delta_block.Stack(2, 32, 4, 2, 16, 24, rotated=8, dtype=F32, seed=3)
    gen = torch.Generator().manual_seed(2)
    e, target = torch.randn((2, 75, 32), generator=gen), torch.randn((2, 75, 32), generator=gen)
    loss, grads = m.loss_and_gradients(e.cuda(), target.cuda())
    leaves = [{k: of(v).requires_grad_(True) for k, v in p.items()} for p in m.layers]
    out = plain_stack(m, leaves, of(e))
    want_loss = ((out - of(target)) ** 2).mean()
    flat = [(i, k) for i, p in enumerate(leaves) for k in p]
    want = dict(zip(flat, torch.autograd.grad(want_loss, [leaves[i][k] for i, k in flat])))
    assert abs(loss.item() - want_loss.item()) <= 12 * 128 * 2.0 ** -24 * want_loss.item()
    for (i, k), w in want.items():
        d = (grads[i][k].double().cpu() - w).norm() / w.norm()
        assert d <= 12 * 128 * 2.0 ** -24, (i, k, d.item())


def test_prompt_in_parts_with_positions():
    """A prompt in two parts, the second from the first one's states at its own positions."""
    import delta_block
    m = delta_block.Stack(1, 32, 4, 2, 16, 24, rotated=8, dtype=F32, seed=3)
    e = torch.randn((2, 90, 32), generator=torch.Generator().manual_seed(5)).cuda()
    whole, _ = m.forward(e)
    _, states = m.forward(e[:, :50].contiguous())
    at = torch.arange(50, 90, dtype=torch.int32, device="cuda").expand(2, 40).contiguous()
    rest, _ = m.forward(e[:, 50:].contiguous(), states, positions=at)
    assert (rest - whole[:, 50:]).norm() <= 12 * 128 * 2.0 ** -24 * whole[:, 50:].norm()


# ---- refusals of CUDA tensors

def refused(fn, match, error=ValueError):
    with pytest.raises(error, match=match):
        fn()


def test_rule_refuses():
    k = cuda(make(2, 8, 4, 2, 32, 16, BF16))
    a = [k[n] for n in NAMES]
    call = ssd().delta_rule
    refused(lambda: call(a[0][0], *a[1:]), "dimensions")
    refused(lambda: call(a[0], a[1][:, :4], *a[2:]), "k: shape")
    refused(lambda: call(a[0], a[1].half(), *a[2:]), "k: dtype")
    refused(lambda: call(*a[:3], a[3].half(), a[4]), "g: dtype")
    refused(lambda: call(*a[:4], a[4][..., :3]), "beta: shape")
    refused(lambda: call(a[0].cpu(), *a[1:]), "CUDA")
    refused(lambda: call(*a[:2], a[2].cpu(), *a[3:]), "v: on")
    refused(lambda: call(a[0].double(), a[1].double(), a[2].double(), *a[3:]), "unsupported dtype")
    refused(lambda: call(a[0].transpose(2, 3).contiguous().transpose(2, 3), *a[1:]), "q: the values of a token")
    refused(lambda: call(a[0][:1, :1].expand(2, 8, 2, 32), *a[1:]), "broadcast")
    refused(lambda: call(*a, initial_states=k["h0"].bfloat16()), "initial_states: dtype")
    refused(lambda: call(*a, lengths=torch.zeros(2, device="cuda")), "lengths: dtype")
    refused(lambda: call(*a, out=torch.empty_like(a[2][:, :4])), "out: shape")
    error = type(ssd().SsdError(1, "", ""))
    refused(lambda: call(*a, out=a[2]), "overlap", error)
    refused(lambda: call(*a, scale=float("nan")), "scale", error)
    odd = torch.zeros((2, 8, 3, 32), device="cuda", dtype=BF16)
    refused(lambda: call(odd, odd, *a[2:]), "multiple", error)
    big = torch.zeros((1, 4, 1, 136), device="cuda")
    refused(lambda: call(big, big, big, big[..., 0], big[..., 0]), "N must be", error)
    empty = torch.zeros((0, 4, 1, 16), device="cuda")
    refused(lambda: call(empty, empty, empty, empty[..., 0], empty[..., 0]), "every dim", error)
    refused(lambda: ssd().delta_rule_bwd(*a, a[2][:, :, :2]), "dy: shape")
    refused(lambda: ssd().delta_rule_bwd(*a, a[2], dfinal=k["h0"][:1]), "dfinal: shape")


def test_step_refuses():
    k = cuda(make(2, 1, 4, 2, 32, 16, F16))
    a, state = [k[n][:, 0] for n in NAMES], k["h0"].clone()
    call = ssd().delta_rule_step
    error = type(ssd().SsdError(1, "", ""))
    refused(lambda: call(*a, state[:, :2]), "state: shape")
    refused(lambda: call(*a, state.half()), "state: dtype")
    refused(lambda: call(*a, state, slots=torch.zeros(2, dtype=torch.int64, device="cuda")), "slots: dtype")
    refused(lambda: call(*a, state[:1]), "nslots", error)
    refused(lambda: call(*a, state, state_out=state[:1]), "state_out: shape")
    refused(lambda: call(*a, state, out=a[2].contiguous()[:1]), "out: shape")


def test_norm_refuses():
    q, k = torch.zeros((2, 8, 4, 32), device="cuda"), torch.zeros((2, 8, 2, 32), device="cuda")
    f, w = torch.ones(8, device="cuda"), torch.ones(32, device="cuda")
    call = ssd().qk_norm
    error = type(ssd().SsdError(1, "", ""))
    refused(lambda: call(q, k[:, :4]), "k: shape")
    refused(lambda: call(q, k.half()), "k: dtype")
    refused(lambda: call(q, k, w_q=w[:16]), "w_q: shape")
    refused(lambda: call(q, k, w_k=w.half()), "w_k: dtype")
    refused(lambda: call(q, k, freqs=f.double()), "freqs: dtype")
    refused(lambda: call(q, k, freqs=f, positions=torch.zeros((2, 8), device="cuda")), "positions: dtype")
    refused(lambda: call(q, k, freqs=f, positions=torch.zeros((2, 4), dtype=torch.int32, device="cuda")), "positions: shape")
    refused(lambda: call(q, k, freqs=torch.ones(17, device="cuda")), "frequencies", error)
    refused(lambda: call(q, k, eps=-1.0), "eps", error)
    refused(lambda: call(q, k, norm="sum"), "norm")
    refused(lambda: call(q[:, 0], k[:, 0], freqs=f), "positions are required")
    refused(lambda: call(q, k, out_q=q[:, :, :, :16]), "out_q: shape")
    refused(lambda: call(k, k, out_q=k, out_k=k), "overlap", error)
    refused(lambda: ssd().qk_norm_bwd(q, k[:, :4], q, k), "dk_out: shape")


def test_one_token_for_all_of_a_row():
    """Tensors whose tokens, or whose rows, share memory are read like any others."""
    k = cuda(make(2, 70, 4, 2, 32, 16, BF16))
    for over in ({"q": k["q"][:, :1].expand(2, 70, 2, 32)}, {"k": k["k"][:1].expand(2, 70, 2, 32)}, {"v": k["v"][:, :1].expand(2, 70, 4, 16)},
                 {"g": k["g"][:1].expand(2, 70, 4), "beta": k["beta"][:, :1].expand(2, 70, 4)}):
        a, b = [{**k, **over}[n] for n in NAMES], [{**k, **over}[n].contiguous() for n in NAMES]
        assert torch.equal(ssd().delta_rule(*a), ssd().delta_rule(*b)), over.keys()
        x, y = ssd().delta_rule_bwd(*a, k["v"]), ssd().delta_rule_bwd(*b, k["v"])
        assert all(torch.equal(x[n], y[n]) for n in y), over.keys()
