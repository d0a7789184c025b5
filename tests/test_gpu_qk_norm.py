"""qk_norm and its backward pass on the GPU against the float64 oracle.

Tolerances (2-norm of the error over 2-norm of the result):
* fp32 results (fp32 storage, and weight gradients always): a row's sum, root,
  angle and products each round at 2^-24; a dozen such steps give < 1e-6, and
  1e-5 leaves room for sums over rows that partly cancel.
* bf16 results: one rounding, of at most 2^-9 of a value: < 2^-9 = 1.96e-3,
  plus nothing else of note: 2.1e-3.
"""
import numpy as np
import pytest
import torch

from tests import operators_oracle as O

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
TOL = {BF: 2.1e-3, F: 1e-5}


def P():
    from linear_recurrent_sequence_shortconv_amd import prism
    return prism


def _np(t):
    return t.double().cpu().numpy()


def _draw(dt, B, T, Hq, Hk, d, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)
    x = {"q": r(B, T, Hq, d), "k": r(B, T, Hk, d) if Hk else None, "wq": 1 + 0.2 * r(d), "wk": 1 + 0.2 * r(d),
         "dqo": r(B, T, Hq, d), "dko": r(B, T, Hk, d) if Hk else None}
    pos = torch.randint(-1000, 1 << 20, (B, T), generator=gen, device="cuda", dtype=torch.int32)
    return x, pos


# dtype, B, T, Hq, Hk, d, rot, norm, wq, wk, interleaved
CASES = [
    (BF, 2, 5, 4, 4, 128, 128, "l2", False, False, False),
    (BF, 1, 1, 1, 0, 64, 64, "rms", True, False, False),
    (BF, 3, 7, 16, 4, 128, 64, "rms", True, True, False),
    (BF, 2, 9, 5, 3, 80, 40, "rms", True, True, False),     # 8-byte vectors: rot / 2 = 20
    (BF, 2, 9, 5, 3, 80, 40, "l2", False, True, True),
    (BF, 1, 3, 2, 2, 8, 8, "rms", True, True, False),
    (BF, 2, 33, 3, 1, 256, 256, "l2", True, False, True),
    (BF, 2, 4, 3, 3, 24, 0, "rms", True, True, False),      # no rotation
    (BF, 1, 4100, 3, 2, 48, 16, "rms", True, True, False),  # a wave a token
    (BF, 5, 1, 40, 8, 96, 96, "rms", True, True, True),
    (F, 2, 5, 4, 4, 128, 128, "l2", False, False, False),
    (F, 3, 11, 5, 5, 48, 32, "rms", True, True, True),
    (F, 1, 4133, 1, 1, 16, 8, "rms", True, True, False),
    (F, 2, 3, 7, 2, 256, 128, "rms", True, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_forward_and_backward(case):
    dt, B, T, Hq, Hk, d, rot, norm, uq, uk, il = case
    x, pos = _draw(dt, B, T, Hq, Hk, d, seed=B * 1000 + d)
    turns = P().rope_turns(rot) if rot else None
    tl = turns.tolist() if rot else []
    kw = dict(wq=x["wq"] if uq else None, wk=x["wk"] if uk else None, positions=pos if rot else None,
              turns=turns, norm=norm, interleaved=il)
    print(f"\n[qk_norm {case}]", flush=True)
    qo, ko = P().qk_norm(x["q"], x["k"], **kw)
    g = P().qk_norm_backward(x["q"], x["k"], x["dqo"], x["dko"], **kw)
    torch.cuda.synchronize()
    p = pos.cpu().numpy()
    for n, use, out, dout in (("q", uq, qo, x["dqo"]), ("k", uk, ko, x["dko"])):
        if x[n] is None:
            assert out is None
            continue
        w = _np(x["w" + n]) if use else None
        want = O.norm_forward(_np(x[n]), w, p, tl, norm, 1e-6, il)
        assert out.dtype == dt and O.rel2(_np(out), want) < TOL[dt]
        dx, dw = O.norm_backward(_np(x[n]), w, _np(dout), p, tl, norm, 1e-6, il)
        assert O.rel2(_np(g["d" + n]), dx) < TOL[dt]
        assert ("dw" + n in g) == use
        if use:
            assert O.rel2(_np(g["dw" + n]), dw) < TOL[F]


def test_strided_in_place_and_heads_first():
    """Views of a fused projection (in place as well) and heads-first tensors
    give bitwise what contiguous ones give; values between the views stay."""
    B, T, Hq, Hk, d = 2, 6, 4, 2, 64
    x, pos = _draw(BF, B, T, Hq, Hk, d, seed=1)
    turns = P().rope_turns(d)
    want = P().qk_norm(x["q"], x["k"], positions=pos, turns=turns)
    row = torch.cat([x["q"], x["k"], torch.full((B, T, Hk, d), 7.0, device="cuda", dtype=BF)], 2)
    q, k = row[:, :, :Hq], row[:, :, Hq:Hq + Hk]
    got = P().qk_norm(q, k, positions=pos, turns=turns)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    hf = x["q"].transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(P().qk_norm(hf, x["k"], positions=pos, turns=turns)[0], want[0])
    P().qk_norm(q, k, positions=pos, turns=turns, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and bool((row[:, :, Hq + Hk:] == 7).all())
    # gradients into the slices of one buffer; steps of 4 elements take 8-byte vectors
    g = P().qk_norm_backward(x["q"], x["k"], x["dqo"], x["dko"], wq=x["wq"], positions=pos, turns=turns)
    buf = torch.zeros(B, T, (Hq + Hk) * d + 4, device="cuda", dtype=BF)
    dq = buf[..., :Hq * d].unflatten(-1, (Hq, d))
    dk = buf[..., Hq * d:-4].unflatten(-1, (Hk, d))
    h = P().qk_norm_backward(x["q"], x["k"], x["dqo"], x["dko"], wq=x["wq"], positions=pos, turns=turns, dq=dq, dk=dk)
    assert O.rel2(_np(dq), _np(g["dq"])) < 1e-3 and O.rel2(_np(dk), _np(g["dk"])) < 1e-3
    assert O.rel2(_np(h["dwq"]), _np(g["dwq"])) < 1e-5 and bool((buf[..., -4:] == 0).all())


def test_packed_rows_equal_the_dense_batch():
    x, pos = _draw(F, 2, 5, 3, 3, 32, seed=2)
    turns = P().rope_turns(32)
    a = P().qk_norm(x["q"], x["k"], positions=pos, turns=turns)
    b = P().qk_norm(x["q"].flatten(0, 1), x["k"].flatten(0, 1), positions=pos.flatten(), turns=turns)
    assert torch.equal(a[0].flatten(0, 1), b[0]) and torch.equal(a[1].flatten(0, 1), b[1])


def test_no_tokens_and_zero_rows():
    x, pos = _draw(BF, 0, 5, 2, 2, 32, seed=3)
    qo, ko = P().qk_norm(x["q"], x["k"])
    assert qo.shape == (0, 5, 2, 32)
    g = P().qk_norm_backward(x["q"], x["k"], x["dqo"], x["dko"], wq=x["wq"], wk=x["wk"])
    assert bool((g["dwq"] == 0).all()) and bool((g["dwk"] == 0).all())
    x, pos = _draw(F, 1, 3, 2, 2, 32, seed=4)
    x["q"][:, 1] = 0     # a row of zeros: zero out, gradient dz / sqrt(eps)
    qo, _ = P().qk_norm(x["q"], x["k"], eps=1e-4)
    g = P().qk_norm_backward(x["q"], x["k"], x["dqo"], x["dko"], eps=1e-4)
    assert bool((qo[:, 1] == 0).all())
    assert O.rel2(_np(g["dq"][:, 1]), _np(x["dqo"][:, 1]) * 100.0) < 1e-5


def test_far_positions():
    """Positions at the ends of int32 turn as exactly as near ones."""
    x, _ = _draw(F, 1, 4, 2, 1, 64, seed=5)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 123456789, -1]], dtype=torch.int32, device="cuda")
    turns = P().rope_turns(64, base=500000.0)
    qo, _ = P().qk_norm(x["q"], x["k"], positions=pos, turns=turns)
    want = O.norm_forward(_np(x["q"]), None, pos.cpu().numpy(), turns.tolist(), "l2", 1e-6, False)
    assert O.rel2(_np(qo), want) < TOL[F]


def test_same_bits_each_time_and_on_another_stream():
    x, pos = _draw(BF, 1, 3000, 4, 2, 64, seed=6)
    turns = P().rope_turns(64)
    run = lambda: P().qk_norm_backward(x["q"], x["k"], x["dqo"], x["dko"], wq=x["wq"], wk=x["wk"], positions=pos,
                                       turns=turns)
    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_gradient_against_differences():
    """The kernel's fp32 gradient along a random direction against a central
    difference of the float64 forward."""
    x, pos = _draw(F, 1, 3, 2, 1, 32, seed=7)
    turns = P().rope_turns(32)
    kw = dict(wq=x["wq"], wk=x["wk"], positions=pos, turns=turns, norm="rms")
    g = P().qk_norm_backward(x["q"], x["k"], x["dqo"], x["dko"], **kw)
    rng = np.random.default_rng(8)
    p, tl = pos.cpu().numpy(), turns.tolist()
    u, uw = rng.standard_normal(x["q"].shape), rng.standard_normal(32)

    def f(h):
        return np.sum(_np(x["dqo"]) * O.norm_forward(_np(x["q"]) + h * u, _np(x["wq"]) + h * uw, p, tl, "rms", 1e-6, False))

    got = np.sum(_np(g["dq"]) * u) + np.sum(_np(g["dwq"]) * uw)
    want = (f(1e-5) - f(-1e-5)) / 2e-5
    size = np.linalg.norm(_np(g["dq"])) * np.linalg.norm(u)
    assert abs(got - want) < 1e-5 * size
