"""A stack of selective state-space blocks over the library's operators.

Each layer is: norm -> in-projection -> short causal convolution -> selective
scan (gated) -> out-projection -> gated residual.  The end of one layer and the
norm before the next are one ``block_norm``; x, z, dt, B and C are slices of
the projections, read in place.  The three uses:

    prompts     Stack.forward(embeddings) -> (hidden states, carried states)
    tokens      Stack.step(embedding, carried states), in place
    training    Stack.loss_and_gradients(embeddings, target)

Run it on a GPU:  python examples/selective_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_ssd_chunked_fwd_gb300 as ssd  # noqa: E402


class Stack:
    def __init__(self, layers, d_model, d_inner, d_state, dt_rank, width=4, dtype=torch.bfloat16, seed=0):
        self.sizes = (d_model, d_inner, d_state, dt_rank, width)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0, dt=torch.float32):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

        def matrix(rows, cols):
            return normal(rows, cols, scale=cols ** -0.5, dt=dtype)

        self.norm = torch.ones(d_model, device="cuda")
        self.layers = []
        for _ in range(layers):
            d = torch.exp(torch.rand(d_inner, generator=g, device="cuda") * 4.6 - 6.9)  # steps of 0.001 to 0.1
            self.layers.append({
                "in_proj": matrix(2 * d_inner, d_model), "conv_w": normal(d_inner, width, scale=width ** -0.5),
                "conv_b": normal(d_inner, scale=0.1), "x_proj": matrix(dt_rank + 2 * d_state, d_inner),
                "dt_proj": matrix(d_inner, dt_rank), "dt_bias": d + torch.log(-torch.expm1(-d)),
                "A": -torch.arange(1, d_state + 1, device="cuda").float().repeat(d_inner, 1),
                "D": torch.ones(d_inner, device="cuda"), "out_proj": matrix(d_model, d_inner),
                "w_post": torch.ones(d_model, device="cuda"), "scale": torch.full((d_model,), 0.5, device="cuda"),
                "w_pre": torch.ones(d_model, device="cuda")})  # the norm after this layer

    def _split(self, p, xc):
        """dt, B and C (views) from the convolved x."""
        _, _, n, r, _ = self.sizes
        proj = xc @ p["x_proj"].t()
        return proj, proj[..., :r] @ p["dt_proj"].t(), proj[..., r:r + n].unsqueeze(-2), proj[..., r + n:].unsqueeze(-2)

    def forward(self, e, states=None, lengths=None, keep=None):
        """e [B,L,d_model]; states: the second result of an earlier call on the
        same sequences; lengths (int32 [B]): tokens per row.  keep: a list that
        gets what the backward needs."""
        d_inner = self.sizes[1]
        n, r = ssd.block_norm(None, e, self.norm)
        carried = []
        for i, p in enumerate(self.layers):
            conv0, h0 = states[i] if states else (None, None)
            xz = n @ p["in_proj"].t()
            x, z = xz[..., :d_inner], xz[..., d_inner:]
            xc, conv1 = ssd.causal_conv1d_carry(x, p["conv_w"], p["conv_b"], initial_state=conv0, lengths=lengths,
                                                return_final_state=True)
            proj, dt, B, C = self._split(p, xc)
            y, h1 = ssd.selective_scan(xc, dt, p["A"], B, C, dt_softplus=True, return_final_state=True, D=p["D"], z=z,
                                       dt_bias=p["dt_bias"], initial_states=h0, lengths=lengths)
            o = y @ p["out_proj"].t()
            n_in = n
            n, r = ssd.block_norm(o, r, p["w_pre"], w_post=p["w_post"], scale=p["scale"])
            carried.append((conv1, h1))
            if keep is not None:
                keep.append((n_in, x, z, xc, proj, dt, B, C, y, o, r))
        return n, carried

    def step(self, e, states, slots=None):
        """One token per row, e [B,d_model]: advances the states in place."""
        d_inner = self.sizes[1]
        n, r = ssd.block_norm(None, e, self.norm)
        for p, (conv, h) in zip(self.layers, states):
            xz = n @ p["in_proj"].t()
            xc = ssd.causal_conv1d_step(xz[..., :d_inner], conv, p["conv_w"], p["conv_b"], slots=slots)
            _, dt, B, C = self._split(p, xc)
            y = ssd.selective_scan_step(xc, dt, p["A"], B, C, h, dt_softplus=True, slots=slots, D=p["D"],
                                        z=xz[..., d_inner:], dt_bias=p["dt_bias"])
            n, r = ssd.block_norm(y @ p["out_proj"].t(), r, p["w_pre"], w_post=p["w_post"], scale=p["scale"])
        return n

    def loss_and_gradients(self, e, target):
        """Mean squared error of the hidden states, and the gradients of every layer's parameters."""
        kept = []
        out, _ = self.forward(e, keep=kept)
        diff = out.float() - target.float()
        loss = (diff * diff).mean()
        dn = (diff * (2.0 / diff.numel())).to(out.dtype)
        dr, grads = None, []

        def outer(a, b):  # the gradient of a projection's matrix
            return a.reshape(-1, a.shape[-1]).t() @ b.reshape(-1, b.shape[-1])

        for p, (n_in, x, z, xc, proj, dt, B, C, y, o, r) in zip(reversed(self.layers), reversed(kept)):
            rank = self.sizes[3]
            g = {}
            k = ssd.block_norm_bwd(dn, dr, o, r, p["w_pre"], w_post=p["w_post"], scale=p["scale"])
            g["w_pre"], g["w_post"], g["scale"], dr = k["dw_pre"], k["dw_post"], k["dscale"], k["dr"]
            g["out_proj"] = outer(k["do"], y)
            s = ssd.selective_scan_bwd(xc, dt, p["A"], B, C, k["do"] @ p["out_proj"], dt_softplus=True, D=p["D"], z=z,
                                       dt_bias=p["dt_bias"])
            g["A"], g["D"], g["dt_bias"] = s["dA"], s["dD"], s["ddt_bias"]
            g["dt_proj"] = outer(s["ddt"], proj[..., :rank])
            dproj = torch.cat([s["ddt"] @ p["dt_proj"], s["dB"].squeeze(-2), s["dC"].squeeze(-2)], -1)
            g["x_proj"] = outer(dproj, xc)
            c = ssd.causal_conv1d_bwd(x, p["conv_w"], s["dx"] + dproj @ p["x_proj"], p["conv_b"])
            g["conv_w"], g["conv_b"] = c["dw"], c["dbias"]
            dxz = torch.cat([c["dx"], s["dz"]], -1)
            g["in_proj"] = outer(dxz, n_in)
            dn = dxz @ p["in_proj"]
            grads.append(g)
        return loss, grads[::-1]


def main(layers=2, d_model=256, d_inner=512, d_state=16, dt_rank=16, batch=2, prompt=96, tokens=8):
    m = Stack(layers, d_model, d_inner, d_state, dt_rank)
    g = torch.Generator(device="cuda").manual_seed(1)
    e = torch.randn((batch, prompt + tokens, d_model), generator=g, device="cuda").bfloat16()
    whole, _ = m.forward(e)
    out, states = m.forward(e[:, :prompt].contiguous())
    steps = [m.step(e[:, prompt + t].contiguous(), states) for t in range(tokens)]
    drift = (torch.stack(steps, 1).float() - whole[:, prompt:].float()).norm() / whole[:, prompt:].float().norm()
    print(f"prompt of {prompt} then {tokens} single tokens against one prompt: relative difference {drift.item():.2e}")
    target = torch.randn(whole.shape, generator=g, device="cuda").bfloat16()
    losses = []
    for _ in range(5):
        loss, grads = m.loss_and_gradients(e, target)
        losses.append(loss.item())
        for p, gr in zip(m.layers, grads):
            for k in p:
                if k == "A":  # through its logarithm, so that it stays negative
                    slope = gr[k] * p[k]
                    p[k] = p[k] * torch.exp(-0.05 * slope / (slope.abs().max() + 1e-12))
                    continue
                step = 0.05 * gr[k].float() / (gr[k].float().norm() + 1e-12) * p[k].float().norm()
                p[k] = (p[k].float() - step).to(p[k].dtype)
    print("training losses:", " ".join(f"{v:.4f}" for v in losses))
    return drift.item(), losses


if __name__ == "__main__":
    main()
