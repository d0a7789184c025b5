"""A recurrent block from the package's operators: prompt, decode, training.

    python examples/recurrent_block.py

The residual stream enters with the sum of the block before it: layer_norm forms
stream + x and its norm in one pass.  One projection gives values, forget gates
and input gates; short_conv mixes the values over the last four tokens and
gated_recurrence along the whole sequence; a second projection leaves the block.
The same weights then serve

* prefill: a prompt of T tokens, which returns the convolution's last tokens and
  the recurrence's state;
* decode: one token a call from these (short_conv with its history in place,
  gated_recurrence_step);
* a training step: gradients of all weights through gated_recurrence_backward,
  short_conv_backward and layer_norm_backward.

The script checks that decoding token by token equals the whole prompt, takes a
few steps of gradient descent, and runs the delta-rule layer with short_conv in
front of queries, keys and values and layer_norm on each head's output.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_recurrent_sequence_shortconv_amd import prism as P  # noqa: E402


class Block:
    """Model width D, recurrence over R channels."""

    K = 4

    def __init__(self, D, R, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=device)
        self.R = R
        self.w_in = (normal(D, 3 * R) * D ** -0.5).to(dtype)
        self.w_out = (normal(R, D) * R ** -0.5).to(dtype)
        self.w_norm, self.b_norm = torch.ones(D, dtype=dtype, device=device), torch.zeros(D, dtype=dtype, device=device)
        self.w_conv = (normal(R, self.K) * self.K ** -0.5).to(dtype)
        self.b_conv = torch.zeros(R, dtype=dtype, device=device)
        # an open gate keeps 0.9 .. 0.999 of the state
        self.lam = -torch.log(torch.linspace(0.9, 0.999, R, device=device))

    def _project(self, y):
        row = y @ self.w_in
        return row[..., :self.R], row[..., self.R:2 * self.R], row[..., 2 * self.R:]

    def prefill(self, x, stream, hist=None, state=None):
        """x, stream [B, T, D] -> block output, the new stream, history, state."""
        y, stream = P.layer_norm(x, self.w_norm, self.b_norm, residual=stream)
        v, f, i = self._project(y)
        last = x.new_empty(x.shape[0], self.K - 1, self.R)
        u = P.short_conv(v, self.w_conv, b=self.b_conv, hist=hist, activation="silu", hist_out=last)
        h, state = P.gated_recurrence(u, f, i=i, lam=self.lam, h0=state, gate="power")
        return h @ self.w_out, stream, last, state

    def decode(self, x, stream, hist, state):
        """One token of each sequence; history and state are updated in place."""
        y, stream = P.layer_norm(x, self.w_norm, self.b_norm, residual=stream, h=stream)
        v, f, i = self._project(y)
        u = P.short_conv(v, self.w_conv, b=self.b_conv, hist=hist, activation="silu", hist_out=hist)
        h = P.gated_recurrence_step(u, f, state, i=i, lam=self.lam, gate="power")
        return h @ self.w_out, stream

    def gradients(self, x, stream, target):
        """Loss and gradients of mean (stream + block output - target)^2."""
        y, s = P.layer_norm(x, self.w_norm, self.b_norm, residual=stream)
        v, f, i = self._project(y)
        u = P.short_conv(v, self.w_conv, b=self.b_conv, activation="silu")
        h, _ = P.gated_recurrence(u, f, i=i, lam=self.lam, gate="power", need_state=False)
        off = s.float() + (h @ self.w_out).float() - target
        d = (2.0 / off.numel()) * off
        dh_stream = d.to(x.dtype)                       # reaches the stream and the block's output alike
        flat = lambda t: t.flatten(0, -2)
        g = {"w_out": flat(h).t().contiguous() @ flat(dh_stream)}
        # the gradients of the projection's three parts go into one buffer
        drow = x.new_empty(*x.shape[:-1], 3 * self.R)
        part = lambda k: drow[..., k * self.R:(k + 1) * self.R]
        r = P.gated_recurrence_backward(u, f, h, dh_stream @ self.w_out.t().contiguous(), i=i, lam=self.lam,
                                        gate="power", df=part(1), di=part(2))
        c = P.short_conv_backward(v, self.w_conv, r["dx"], b=self.b_conv, activation="silu", dx=part(0))
        g.update(lam=r["dlam"], w_conv=c["dw"], b_conv=c["db"])
        g["w_in"] = flat(y).t().contiguous() @ flat(drow)
        n = P.layer_norm_backward(s, drow @ self.w_in.t().contiguous(), self.w_norm, dh=dh_stream, need_db=True)
        g.update(w_norm=n["dw"], b_norm=n["db"], x=n["dx"])
        return float(off.square().mean()), g

    def train_step(self, x, stream, target, lr):
        loss, g = self.gradients(x, stream, target)
        for n in ("w_in", "w_out", "w_norm", "b_norm", "w_conv", "b_conv", "lam"):
            p = getattr(self, n)
            p.sub_((lr * g[n].float()).to(p.dtype))
        self.lam.clamp_(min=1e-4)
        return loss


def delta_rule_layer(x, B, T, H, d, seed=2):
    """The delta-rule layer on queries, keys and values that short_conv mixed, its
    output normalised for each head."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    D = x.shape[-1]
    row = x @ (normal(D, 3 * H * d) * D ** -0.5).to(x.dtype)
    taps = (0.5 * normal(3 * H * d, 4)).to(x.dtype)
    q, k, v = (t.unflatten(-1, (H, d)) for t in P.short_conv(row, taps, activation="silu").chunk(3, -1))
    q, k = P.qk_norm(q, k)
    alpha, beta = torch.full((B, T, H), 0.95, device="cuda"), torch.full((B, T, H), 0.5, device="cuda")
    o, _ = P.forward(q, k, v.contiguous(), alpha, beta)
    return o, P.layer_norm(o, torch.ones(d, dtype=x.dtype, device="cuda"), norm="rms")[0]


def main(B=2, T=300, D=256, R=320, new=8):
    block = Block(D, R)
    gen = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda: torch.randn(B, T + new, D, generator=gen, device="cuda").bfloat16()
    x, stream = draw(), draw()
    whole, sum_whole, last_whole, state_whole = block.prefill(x, stream)
    part = lambda t, a, b: t[:, a:b].contiguous()
    y, s, hist, state = block.prefill(part(x, 0, T), part(stream, 0, T))
    for t in range(T, T + new):
        step, s1 = block.decode(part(x, t, t + 1), part(stream, t, t + 1), hist, state)
        y, s = torch.cat([y, step], 1), torch.cat([s, s1], 1)
    off = float((y.float() - whole.float()).norm() / whole.float().norm())
    off_state = float((state - state_whole).norm() / state_whole.norm())
    same = torch.equal(s, sum_whole) and hist.shape == last_whole.shape
    print(f"prompt of {T} and {new} steps against {T + new} at once: outputs {off:.1e}, state {off_state:.1e}")

    target = torch.randn(B, T + new, D, generator=gen, device="cuda")
    losses = [block.train_step(x, stream, target, lr=1.0) for _ in range(5)]
    print("loss " + " ".join(f"{v:.4f}" for v in losses))

    o, n = delta_rule_layer(x, B, T + new, 4, 64)
    print(f"delta-rule layer behind short convolutions: {float(o.float().norm()):.2f}, its heads normalised "
          f"{float(n.float().norm()):.2f}")
    return off, off_state, same, losses, n


if __name__ == "__main__":
    main()
