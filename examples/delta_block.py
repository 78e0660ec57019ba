"""A stack of gated delta-rule blocks over the library's operators.

Each layer is: norm -> projection -> short causal convolution of queries, keys and
values -> norm of queries and keys with their rotation -> gated delta rule ->
out-projection -> residual.  The end of one layer and the norm before the next
are one ``block_norm``; q, k and v are slices of the convolved projection, read in place.
The three uses:

    prompts     Stack.forward(embeddings) -> (hidden states, carried states)
    tokens      Stack.step(embedding, carried states, positions), in place
    training    Stack.loss_and_gradients(embeddings, target)

Run it on a GPU:  python examples/delta_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_ssd_chunked_fwd_gb300 as ssd  # noqa: E402


class Stack:
    def __init__(self, layers, d_model, heads, key_heads, d_key, d_value, rotated=0, width=4, dtype=torch.bfloat16, seed=0):
        self.sizes = (d_model, heads, key_heads, d_key, d_value, width)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0, dt=torch.float32):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

        def matrix(rows, cols):
            return normal(rows, cols, scale=cols ** -0.5, dt=dtype)

        inner = 2 * key_heads * d_key + heads * d_value
        self.freqs = 10000.0 ** (-torch.arange(rotated // 2, device="cuda") / max(rotated // 2, 1)) if rotated else None
        self.norm = torch.ones(d_model, device="cuda")
        self.layers = []
        for _ in range(layers):
            d = torch.exp(torch.rand(heads, generator=g, device="cuda") * 4.6 - 6.9)  # steps of 0.001 to 0.1
            self.layers.append({
                "in_proj": matrix(inner, d_model), "gate_proj": matrix(2 * heads, d_model), "conv_w": normal(inner, width, scale=width ** -0.5),
                "conv_b": normal(inner, scale=0.1), "A_log": torch.log(1 + 15 * torch.rand(heads, generator=g, device="cuda")),
                "dt_bias": d + torch.log(-torch.expm1(-d)), "out_proj": matrix(d_model, heads * d_value),
                "w_post": torch.ones(d_model, device="cuda"), "scale": torch.full((d_model,), 0.5, device="cuda"),
                "w_pre": torch.ones(d_model, device="cuda")})  # the norm after this layer

    def _gates(self, p, n):
        """The decay's logarithm g (32 bits) and beta, with what their gradients need."""
        heads = self.sizes[1]
        ab = n @ p["gate_proj"].t()
        raw = ab[..., :heads].float() + p["dt_bias"]
        return -torch.exp(p["A_log"]) * torch.nn.functional.softplus(raw), torch.sigmoid(ab[..., heads:]), raw

    def _split(self, x):
        _, heads, key_heads, d_key, d_value, _ = self.sizes
        q, k, v = x.split([key_heads * d_key, key_heads * d_key, heads * d_value], -1)
        return q.unflatten(-1, (key_heads, d_key)), k.unflatten(-1, (key_heads, d_key)), v.unflatten(-1, (heads, d_value))

    def forward(self, e, states=None, lengths=None, positions=None, keep=None):
        """e [B,L,d_model]; states: the second result of an earlier call on the same
        sequences, positions (int32 [B,L], default 0 .. L-1) then their places; lengths
        (int32 [B]): tokens per row.  keep: a list that gets what the backward needs."""
        n, r = ssd.block_norm(None, e, self.norm)
        carried = []
        for i, p in enumerate(self.layers):
            conv0, h0 = states[i] if states else (None, None)
            x = n @ p["in_proj"].t()
            xc, conv1 = ssd.causal_conv1d_carry(x, p["conv_w"], p["conv_b"], initial_state=conv0, lengths=lengths, return_final_state=True)
            q, k, v = self._split(xc)
            g, beta, raw = self._gates(p, n)
            qn, kn = ssd.qk_norm(q, k, norm="l2", freqs=self.freqs, positions=positions)
            y, h1 = ssd.delta_rule(qn, kn, v, g, beta, initial_states=h0, lengths=lengths, return_final_state=True)
            o = y.flatten(-2) @ p["out_proj"].t()
            n_in = n
            n, r = ssd.block_norm(o, r, p["w_pre"], w_post=p["w_post"], scale=p["scale"])
            carried.append((conv1, h1))
            if keep is not None:
                keep.append((n_in, x, q, k, v, g, beta, raw, qn, kn, y, o, r))
        return n, carried

    def step(self, e, states, positions, slots=None):
        """One token per row, e [B,d_model] at positions [B]: advances the states in place."""
        n, r = ssd.block_norm(None, e, self.norm)
        for p, (conv, h) in zip(self.layers, states):
            xc = ssd.causal_conv1d_step(n @ p["in_proj"].t(), conv, p["conv_w"], p["conv_b"], slots=slots)
            q, k, v = self._split(xc)
            g, beta, _ = self._gates(p, n)
            qn, kn = ssd.qk_norm(q, k, norm="l2", freqs=self.freqs, positions=positions)
            y = ssd.delta_rule_step(qn, kn, v, g, beta, h, slots=slots)
            n, r = ssd.block_norm(y.flatten(-2) @ p["out_proj"].t(), r, p["w_pre"], w_post=p["w_post"], scale=p["scale"])
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

        for p, (n_in, x, q, k, v, g, beta, raw, qn, kn, y, o, r) in zip(reversed(self.layers), reversed(kept)):
            d = {}
            b = ssd.block_norm_bwd(dn, dr, o, r, p["w_pre"], w_post=p["w_post"], scale=p["scale"])
            d["w_pre"], d["w_post"], d["scale"], dr = b["dw_pre"], b["dw_post"], b["dscale"], b["dr"]
            d["out_proj"] = outer(b["do"], y.flatten(-2))
            s = ssd.delta_rule_bwd(qn, kn, v, g, beta, (b["do"] @ p["out_proj"]).reshape(y.shape))
            t = ssd.qk_norm_bwd(s["dq"], s["dk"], q, k, norm="l2", freqs=self.freqs)
            c = ssd.causal_conv1d_bwd(x, p["conv_w"], torch.cat([t["dq"].flatten(-2), t["dk"].flatten(-2), s["dv"].flatten(-2)], -1), p["conv_b"])
            d["conv_w"], d["conv_b"], d["in_proj"] = c["dw"], c["dbias"], outer(c["dx"], n_in)
            d["A_log"] = (s["dg"] * g).sum((0, 1))
            draw = -s["dg"] * torch.exp(p["A_log"]) * torch.sigmoid(raw)
            d["dt_bias"] = draw.sum((0, 1))
            dab = torch.cat([draw.to(beta.dtype), s["dbeta"] * beta * (1 - beta)], -1)
            d["gate_proj"] = outer(dab, n_in)
            dn = c["dx"] @ p["in_proj"] + dab @ p["gate_proj"]
            grads.append(d)
        return loss, grads[::-1]


def main(layers=2, d_model=256, heads=4, key_heads=2, d_key=64, d_value=64, rotated=32, batch=2, prompt=150, tokens=8):
    m = Stack(layers, d_model, heads, key_heads, d_key, d_value, rotated)
    g = torch.Generator(device="cuda").manual_seed(1)
    e = torch.randn((batch, prompt + tokens, d_model), generator=g, device="cuda").bfloat16()
    whole, _ = m.forward(e)
    _, states = m.forward(e[:, :prompt].contiguous())
    steps = [m.step(e[:, prompt + t].contiguous(), states, torch.full((batch,), prompt + t, dtype=torch.int32, device="cuda"))
             for t in range(tokens)]
    drift = (torch.stack(steps, 1).float() - whole[:, prompt:].float()).norm() / whole[:, prompt:].float().norm()
    print(f"prompt of {prompt} then {tokens} single tokens against one prompt: relative difference {drift.item():.2e}")
    target = torch.randn(whole.shape, generator=g, device="cuda").bfloat16()
    losses = []
    for _ in range(5):
        loss, grads = m.loss_and_gradients(e, target)
        losses.append(loss.item())
        for p, gr in zip(m.layers, grads):
            for k in p:
                step = 0.05 * gr[k].float() / (gr[k].float().norm() + 1e-12) * p[k].float().norm()
                p[k] = (p[k].float() - step).to(p[k].dtype)
    print("training losses:", " ".join(f"{v:.4f}" for v in losses))
    return drift.item(), losses


if __name__ == "__main__":
    main()
