"""A linear-attention layer from the package's operators: prompt, decode, training.

    python examples/linear_attention_layer.py

One fused projection gives queries, keys and values; qk_norm normalises and
rotates the first two (in place in the projection's buffer), linear_attention
mixes along the sequence with a decay for each head, a second projection leaves
the layer.  The same weights then serve

* prefill: a prompt of T tokens, which returns the state;
* decode: one token a call from that state (linear_attention_step);
* a training step: gradients of the weights through linear_attention_backward
  and qk_norm_backward.

The script checks that decoding token by token equals the whole prompt and that
a few steps of gradient descent lower the loss, and shows the same normalised
queries and keys in the delta-rule layer (prism.forward with L = 0).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_recurrent_sequence_shortconv_amd import prism as P  # noqa: E402


class Layer:
    """H query heads over Hk key / value heads of d values, model width D."""

    def __init__(self, D, H, Hk, d, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=device)
        self.H, self.Hk, self.d, self.scale = H, Hk, d, d ** -0.5
        self.w_in = (normal(D, (H + 2 * Hk) * d) * D ** -0.5).to(dtype)
        self.w_out = (normal(H * d, D) * (H * d) ** -0.5).to(dtype)
        self.wq, self.wk = (torch.ones(d, dtype=dtype, device=device) for _ in range(2))
        # decays of 1 - 2^-5 .. 1 - 2^-8 over the heads, as logs
        self.g = torch.log1p(-torch.exp2(-torch.linspace(5.0, 8.0, H, device=device)))
        self.turns = P.rope_turns(d, device=device)

    def _project(self, x):
        row = x @ self.w_in
        cut = lambda a, n: row[..., a * self.d:(a + n) * self.d].unflatten(-1, (n, self.d))
        return row, cut(0, self.H), cut(self.H, self.Hk), cut(self.H + self.Hk, self.Hk)

    def _norm(self):
        return {"wq": self.wq, "wk": self.wk, "turns": self.turns, "norm": "rms"}

    def prefill(self, x, positions, S0=None):
        """x [B, T, D], positions [B, T] int32 -> y [B, T, D], state [B, H, d, d]."""
        _, q, k, v = self._project(x)
        P.qk_norm(q, k, positions=positions, q_out=q, k_out=k, **self._norm())
        o, S = P.linear_attention(q, k, v, self.g, S0=S0, scale=self.scale)
        return o.flatten(-2) @ self.w_out, S

    def decode(self, x, positions, S):
        """One token of each sequence, x [B, 1, D]; the state is updated in place."""
        _, q, k, v = self._project(x)
        P.qk_norm(q, k, positions=positions, q_out=q, k_out=k, **self._norm())
        o = P.linear_attention_step(q, k, v, self.g, S=S, scale=self.scale)
        return o.flatten(-2) @ self.w_out

    def train_step(self, x, positions, target, lr):
        """One step of gradient descent on mean (y - target)^2.  Returns the loss."""
        _, q, k, v = self._project(x)
        qn, kn = P.qk_norm(q, k, positions=positions, **self._norm())
        o, _ = P.linear_attention(qn, kn, v, self.g, scale=self.scale, need_state=False)
        y = (o.flatten(-2) @ self.w_out).float()
        dy = (2.0 / y.numel()) * (y - target)
        dyh = dy.to(x.dtype)
        dw_out = o.flatten(-2).flatten(0, -2).t().contiguous() @ dyh.flatten(0, -2)
        dO = (dyh @ self.w_out.t().contiguous()).unflatten(-1, (self.H, self.d))
        m = P.linear_attention_backward(qn, kn, v, self.g, dO, scale=self.scale)
        # the gradients of q and k go straight into the fused projection's gradient
        drow = torch.empty(*x.shape[:-1], (self.H + 2 * self.Hk) * self.d, dtype=x.dtype, device=x.device)
        cut = lambda a, n: drow[..., a * self.d:(a + n) * self.d].unflatten(-1, (n, self.d))
        w = P.qk_norm_backward(q, k, m["dq"], m["dk"], positions=positions, dq=cut(0, self.H),
                               dk=cut(self.H, self.Hk), **self._norm())
        cut(self.H + self.Hk, self.Hk).copy_(m["dv"])
        dw_in = x.flatten(0, -2).t().contiguous() @ drow.flatten(0, -2)
        for p, g in ((self.w_in, dw_in), (self.w_out, dw_out), (self.wq, w["dwq"]), (self.wk, w["dwk"])):
            p.sub_((lr * g.float()).to(p.dtype))
        return float((y - target).square().mean())


def main(B=2, T=200, D=256, H=4, Hk=2, d=64, new=8):
    layer = Layer(D, H, Hk, d)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, T + new, D, generator=gen, device="cuda").bfloat16()
    pos = torch.arange(T + new, dtype=torch.int32, device="cuda").expand(B, T + new).contiguous()

    whole, S_whole = layer.prefill(x, pos)
    y, S = layer.prefill(x[:, :T].contiguous(), pos[:, :T].contiguous())
    for t in range(T, T + new):
        step = layer.decode(x[:, t:t + 1].contiguous(), pos[:, t:t + 1].contiguous(), S)
        y = torch.cat([y, step], 1)
    off = float((y.float() - whole.float()).norm() / whole.float().norm())
    off_S = float((S - S_whole).norm() / S_whole.norm())
    print(f"prompt of {T} and {new} steps against {T + new} at once: outputs {off:.1e}, state {off_S:.1e}")

    target = torch.randn(B, T + new, D, generator=gen, device="cuda") * 0.1
    losses = [layer.train_step(x, pos, target, lr=0.1) for _ in range(5)]
    print("loss " + " ".join(f"{v:.4f}" for v in losses))

    # the delta-rule layer takes the same normalised queries and keys
    _, q, k, v = layer._project(x)
    q, k = P.qk_norm(q[:, :, :Hk], k, positions=pos, turns=layer.turns)
    alpha = layer.g[:Hk].exp().expand(B, T + new, Hk).contiguous()
    o, _ = P.forward(q, k, v.contiguous(), alpha, torch.full_like(alpha, 0.5))
    print(f"delta-rule layer on them: output norm {float(o.float().norm()):.2f}")
    return off, off_S, losses, o


if __name__ == "__main__":
    main()
