"""The linear-attention example runs: decode equals the prompt, the loss falls,
and its weight gradients equal those of an fp32 recurrence under autograd.

Bounds: outputs pass a bf16 projection behind bf16 operators (each within 5e-3 of
exact, both sides); states are fp32 over the same bf16 inputs.  Gradients in fp32:
products and sums of a few hundred terms at 2^-24 each, 1e-5."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_linear_attention_layer_example():
    from examples import linear_attention_layer as E
    off, off_S, losses, o = E.main()
    assert off < 1.5e-2 and off_S < 1e-2
    assert all(b < a for a, b in zip(losses, losses[1:])) and math.isfinite(losses[-1])
    assert bool(torch.isfinite(o.float()).all())


def test_weight_gradients_against_autograd():
    from examples import linear_attention_layer as E
    B, T, D, H, Hk, d = 2, 40, 128, 4, 2, 32
    L = E.Layer(D, H, Hk, d, dtype=torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, target = (torch.randn(B, T, D, generator=gen, device="cuda") for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    w = {n: getattr(L, n).clone().requires_grad_() for n in ("w_in", "w_out", "wq", "wk")}
    row = x @ w["w_in"]
    cut = lambda a, n: row[..., a * d:(a + n) * d].unflatten(-1, (n, d))

    def norm(y, weight):
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight
        angle = (pos.long()[..., None] * L.turns).double() * (2.0 ** -64 * 2 * math.pi)
        c, s = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    wide = lambda y: y.repeat_interleave(H // Hk, 2)
    q, k, v = norm(cut(0, H), w["wq"]), wide(norm(cut(H, Hk), w["wk"])), wide(cut(H + Hk, Hk))
    S, o = torch.zeros(B, H, d, d, device="cuda"), []
    for t in range(T):
        S = S * L.g.exp()[None, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
        o.append((S * q[:, t, :, None, :]).sum(-1) * L.scale)
    loss = (torch.stack(o, 1).flatten(-2) @ w["w_out"] - target).square().mean()
    loss.backward()
    before = {n: getattr(L, n).clone() for n in w}
    got = L.train_step(x, pos, target, 1.0)
    assert abs(got - float(loss.detach())) < 1e-5 * abs(got)
    for n in w:
        g = before[n] - getattr(L, n)
        # (a weight of size 1 less a gradient keeps 2^-24 of the weight)
        room = 1e-5 * float(w[n].grad.norm()) + 2.0 ** -23 * float(before[n].norm())
        assert float((g - w[n].grad).norm()) < room, n
