"""The recurrent-block example runs, decodes as it reads a prompt, and its
gradients equal those of a plain fp32 form under autograd and differences.

Bounds.  Decoding: the two projections of a prompt and of a token are products of
other shapes, whose bf16 results may be rounded the other way, 2^-8 of a value
each: v, f and i enter the state with three of these, 1.2e-2; the output adds h's
own and the second projection's: 2e-2.  Gradients in fp32: products and sums of up
to a few hundred terms at 2^-24 each, 1e-5; a difference of losses at a step of 2^-6
keeps the third derivative's part, 2^-12 of it, and the losses' own 1e-6 / 2^-6."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
NAMES = ("w_in", "w_out", "w_norm", "b_norm", "w_conv", "b_conv", "lam")


def test_example_runs():
    from examples import recurrent_block as E
    off, off_state, same, losses, n = E.main()
    assert off < 2e-2 and off_state < 1.2e-2 and same
    assert all(math.isfinite(v) for v in losses) and bool(torch.isfinite(n.float()).all())


def _plain(b, w, x, stream, target):
    """The block's loss in plain operations."""
    s = x + stream
    y = (s - s.mean(-1, keepdim=True)) * torch.rsqrt(s.var(-1, unbiased=False, keepdim=True) + 1e-5)
    row = (y * w["w_norm"] + w["b_norm"]) @ w["w_in"]
    v, f, i = row.split(b.R, -1)
    T = x.shape[1]
    full = torch.cat([v.new_zeros(v.shape[0], b.K - 1, b.R), v], 1)
    z = w["b_conv"] + sum(w["w_conv"][:, j] * full[:, b.K - 1 - j:b.K - 1 - j + T] for j in range(b.K))
    u = z * torch.sigmoid(z)
    e = -w["lam"] * torch.sigmoid(f)
    a, u = e.exp(), (-torch.expm1(2 * e)).sqrt() * torch.sigmoid(i) * u
    h, out = torch.zeros_like(u[:, 0]), []
    for t in range(T):
        h = a[:, t] * h + u[:, t]
        out.append(h)
    return (s + torch.stack(out, 1) @ w["w_out"] - target).square().mean()


def test_gradients_against_autograd_and_differences():
    from examples import recurrent_block as E
    B, T, D, R = 2, 150, 64, 80
    b = E.Block(D, R, dtype=torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, stream, target = (torch.randn(B, T, D, generator=gen, device="cuda") for _ in range(3))
    w = {n: getattr(b, n).clone().requires_grad_() for n in NAMES}
    xg = x.clone().requires_grad_()
    loss = _plain(b, w, xg, stream, target)
    loss.backward()
    got, g = b.gradients(x, stream, target)
    assert abs(got - float(loss.detach())) < 1e-5 * abs(got)
    for n, want in [*((n, w[n].grad) for n in NAMES), ("x", xg.grad)]:
        assert float((g[n] - want).norm()) < 1e-5 * float(want.norm()), n
    # along each gradient, the losses on either side (lam starts at -ln 0.999 = 1.0005e-3:
    # a step of 2^-6 along its gradient leaves lam >= 0; its differences are the oracle's)
    for n in NAMES[:-1]:
        p, keep = getattr(b, n), getattr(b, n).clone()
        step = 2.0 ** -6 * g[n] / g[n].norm()
        side = []
        for sign in (1, -1):
            p.copy_(keep + sign * step)
            side.append(b.gradients(x, stream, target)[0])
        p.copy_(keep)
        slope = (side[0] - side[1]) * 2.0 ** 5
        want = float(g[n].norm())
        assert abs(slope - want) < 5e-3 * want + 1e-4, n
