"""linear_attention, its backward pass and its step on the GPU against the
float64 oracle (token by token).

Tolerances (2-norm of the error over 2-norm of the result):
* fp32 results (states always; everything in fp32 storage): products and sums
  round at 2^-24 and a sum of T terms of random sign keeps that relative size;
  decays exp(G_t - G_i) are good to |G_t - G_i| 2^-24, largest where they are
  no longer seen: 1e-5.
* bf16 results: the last rounding (2^-9 of a value at most) and two roundings
  of intermediate operands of the same size: sqrt(3) 2^-9 = 3.4e-3; 5e-3.
* dg: a suffix sum of differences whose terms are good to a few 2^-24: over T
  tokens sqrt(T) of those against a result of at least a term or so; with T <=
  600 that is 25 * 4 * 6e-8 = 6e-6; 3e-5.
"""
import numpy as np
import pytest
import torch

from tests import operators_oracle as O

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
TOL = {BF: 5e-3, F: 1e-5}
TOL_DG = 3e-5


def P():
    from linear_recurrent_sequence_shortconv_amd import prism
    return prism


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _draw(dt, lead, B, H, Hk, dk, dv, decay, seed, states=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)
    x = {"q": unit(r(*lead, H, dk)), "k": unit(r(*lead, Hk, dk)), "v": r(*lead, Hk, dv).to(dt),
         "dO": r(*lead, H, dv).to(dt)}
    if decay == "head":
        x["g"] = torch.log1p(-torch.exp2(-3 - torch.arange(H, device="cuda").float()))
    else:
        x["g"] = torch.nn.functional.logsigmoid(2 + r(*lead, H))
    x["S0"] = r(B, H, dv, dk) if states else None
    x["dST"] = r(B, H, dv, dk) if states else None
    return x


def _oracle(x, spans, scale):
    """The oracle over the sequences `spans` (lists of index pairs into the
    token tensors flattened to [N, ..])."""
    flat = {n: _np(x[n]) for n in x}
    lead = x["q"].dim() - 2
    for n in ("q", "k", "v", "dO"):
        flat[n] = flat[n].reshape((-1,) + flat[n].shape[lead:])
    if x["g"].dim() > 1:
        flat["g"] = flat["g"].reshape(-1, x["g"].shape[-1])
    out = {n: np.zeros(flat[m].shape) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("o", "dO"))}
    out["dg"] = np.zeros(flat["g"].shape)
    H, dv, dk = x["q"].shape[-2], x["v"].shape[-1], x["q"].shape[-1]
    out["ST"], out["dS0"] = np.zeros((len(spans), H, dv, dk)), np.zeros((len(spans), H, dv, dk))
    for i, (a, b) in enumerate(spans):
        g = flat["g"][a:b] if flat["g"].ndim == 2 else flat["g"]
        args = [flat[n][a:b] for n in ("q", "k", "v")] + [g]
        S0 = None if flat["S0"] is None else flat["S0"][i]
        dST = None if flat["dST"] is None else flat["dST"][i]
        out["o"][a:b], out["ST"][i] = O.attend(*args, S0, scale)
        r = O.attend_backward(*args, flat["dO"][a:b], S0, dST, scale)
        for n in ("dq", "dk", "dv"):
            out[n][a:b] = r[n]
        out["dS0"][i] = r["dS0"]
        if flat["g"].ndim == 2:
            out["dg"][a:b] = r["dg"]
        else:
            out["dg"] += r["dg"]
    return out


def _check(got, want, dt, names):
    errs = {n: O.rel2(_np(got[n]).reshape(want[n].shape), want[n]) for n in names}
    print("  " + ", ".join(f"{n} {e:.1e}" for n, e in errs.items()), flush=True)
    for n, e in errs.items():
        tol = TOL_DG if n == "dg" else TOL[F] if n in ("ST", "dS0") else TOL[dt]
        assert e < tol, (n, e)


def _run(x, scale, **packed):
    o, ST = P().linear_attention(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], scale=scale, **packed)
    got = P().linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], S0=x["S0"], dST=x["dST"],
                                        scale=scale, need_dS0=True, need_dg=True, **packed)
    plain = P().linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], S0=x["S0"], dST=x["dST"],
                                          scale=scale, need_dS0=True, **packed)
    return {"o": o, "ST": ST, **got}, plain


ALL = ("o", "ST", "dq", "dk", "dv", "dg", "dS0")
# dtype, B, T, H, Hk, dk, dv, decay, states
CASES = [
    (BF, 2, 1, 2, 2, 64, 64, "head", True),
    (BF, 1, 2, 1, 1, 16, 16, "token", False),
    (BF, 2, 63, 3, 3, 128, 128, "token", True),
    (BF, 1, 64, 2, 1, 128, 128, "head", True),
    (BF, 1, 65, 4, 2, 32, 32, "token", True),
    (BF, 2, 200, 4, 4, 64, 64, "head", False),
    (BF, 1, 577, 2, 2, 128, 128, "token", True),     # several segments
    (BF, 1, 520, 4, 1, 128, 64, "token", True),
    (BF, 2, 130, 2, 2, 48, 112, "head", True),
    (BF, 1, 300, 3, 1, 80, 16, "token", True),
    (F, 2, 1, 2, 2, 64, 64, "token", True),
    (F, 1, 33, 2, 2, 128, 128, "token", True),
    (F, 1, 577, 2, 2, 64, 64, "token", True),
    (F, 2, 333, 3, 3, 64, 48, "token", True),
    (F, 1, 270, 4, 2, 128, 96, "head", True),
    (F, 1, 65, 2, 1, 16, 32, "head", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_whole_sequences(case):
    dt, B, T, H, Hk, dk, dv, decay, states = case
    print(f"\n[linear_attention {case}]", flush=True)
    x = _draw(dt, (B, T), B, H, Hk, dk, dv, decay, seed=T + dk, states=states)
    got, plain = _run(x, 0.5)
    want = _oracle(x, [(b * T, (b + 1) * T) for b in range(B)], 0.5)
    _check(got, want, dt, ALL)
    _check(plain, want, dt, ("dq", "dk", "dv", "dS0"))


@pytest.mark.parametrize("dt,dk,dv,decay", [(BF, 64, 64, "token"), (F, 32, 64, "token"), (BF, 128, 128, "head")])
def test_packed(dt, dk, dv, decay):
    lens = [0, 1, 64, 65, 130, 0, 7, 300]
    cu = np.concatenate([[0], np.cumsum(lens)])
    H = 2
    x = _draw(dt, (int(cu[-1]),), len(lens), H, 1, dk, dv, decay, seed=11)
    print(f"\n[packed {dt} {dk} {dv} {decay}]", flush=True)
    got, plain = _run(x, 1.0, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen=300)
    want = _oracle(x, [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])], 1.0)
    _check(got, want, dt, ALL)
    _check(plain, want, dt, ("dq", "dk", "dv", "dS0"))


def test_packed_offsets_out_of_order_are_clamped():
    """Offsets that fall back or pass the end give the sequences of the
    clamped, running-maximum offsets, and write no other row."""
    x = _draw(F, (40,), 3, 2, 2, 32, 32, "head", seed=12)
    x["S0"] = x["dST"] = None
    cu = torch.tensor([0, 30, 20, 90], dtype=torch.int32, device="cuda")
    o, ST = P().linear_attention(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, max_seqlen=64)
    want = _oracle(x, [(0, 30), (30, 30), (30, 40)], 1.0)
    _check({"o": o, "ST": ST}, want, F, ("o", "ST"))


@pytest.mark.parametrize("dt", [BF, F])
def test_resets_and_no_decay(dt):
    """-inf, the type's lowest value and zero as log decays, at the first token,
    inside a chunk, at its edge and twice in a row."""
    x = _draw(dt, (1, 150), 1, 2, 2, 64, 64, "token", seed=13)
    x["g"][:, 0, 0] = -float("inf")
    x["g"][:, 40, 0] = -float("inf")
    x["g"][:, 41, 0] = torch.finfo(F).min
    x["g"][:, 64, 0] = -200.0
    x["g"][:, :, 1] = 0.0
    x["g"][:, 100, 1] = -float("inf")
    print(f"\n[resets {dt}]", flush=True)
    got, plain = _run(x, 1.0)
    want = _oracle(x, [(0, 150)], 1.0)
    _check(got, want, dt, ALL)
    assert bool((got["dg"][0, [0, 40, 41, 64], 0] == 0).all()) and float(got["dg"][0, 100, 1]) == 0.0


def test_long_memory_and_strong_decay():
    x = _draw(F, (1, 512), 1, 2, 2, 64, 64, "token", seed=14)
    x["g"][:, :, 0] = -1e-5 * torch.rand(512, device="cuda")
    x["g"][:, :, 1] = -3.0 - 20.0 * torch.rand(512, device="cuda")
    got, _ = _run(x, 1.0)
    _check(got, _oracle(x, [(0, 512)], 1.0), F, ALL)


def test_no_tokens():
    x = _draw(BF, (2, 0), 2, 2, 1, 32, 32, "head", seed=15)
    got, _ = _run(x, 1.0)
    torch.cuda.synchronize()
    assert torch.equal(got["ST"], x["S0"]) and torch.equal(got["dS0"], x["dST"])
    assert bool((got["dg"] == 0).all()) and got["o"].shape == (2, 0, 2, 32)
    x["S0"] = None
    o, ST = P().linear_attention(x["q"], x["k"], x["v"], x["g"])
    assert bool((ST == 0).all())


def test_strides_and_in_place_state():
    """Views of a fused projection, heads-first tensors and a state updated in
    place give bitwise what contiguous operands give."""
    B, T, H, Hk, d = 2, 100, 4, 2, 64
    x = _draw(BF, (B, T), B, H, Hk, d, d, "token", seed=16)
    run = lambda q, k, v, **kw: P().linear_attention(q, k, v, x["g"], S0=x["S0"], **kw)
    want = run(x["q"], x["k"], x["v"])
    row = torch.cat([t.flatten(-2) for t in (x["q"], x["k"], x["v"])], -1)
    cut = lambda a, n: row[..., a * d:(a + n) * d].unflatten(-1, (n, d))
    got = run(cut(0, H), cut(H, Hk), cut(H + Hk, Hk))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    hf = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)
    o = torch.zeros(B, H, T, d, device="cuda", dtype=BF).transpose(1, 2)
    got = run(hf(x["q"]), hf(x["k"]), hf(x["v"]), o=o)
    assert torch.equal(o, want[0]) and torch.equal(got[1], want[1])
    S = x["S0"].clone()
    P().linear_attention(x["q"], x["k"], x["v"], x["g"], S0=S, ST=S)
    assert torch.equal(S, want[1])
    # the same over several segments (one sequence, few heads)
    y = _draw(BF, (1, 700), 1, 1, 1, d, d, "token", seed=17)
    o1, S1 = P().linear_attention(y["q"], y["k"], y["v"], y["g"], S0=y["S0"])
    S = y["S0"].clone()
    o2, _ = P().linear_attention(y["q"], y["k"], y["v"], y["g"], S0=S, ST=S)
    assert torch.equal(S, S1) and torch.equal(o1, o2)


@pytest.mark.parametrize("dt,B,T,H,Hk,dk,dv", [
    (BF, 3, 1, 4, 2, 128, 128), (BF, 1, 1, 1, 1, 16, 16), (BF, 2, 5, 2, 2, 48, 80), (F, 2, 3, 2, 1, 64, 48),
    (F, 70, 1, 16, 16, 32, 128)])
def test_step(dt, B, T, H, Hk, dk, dv):
    x = _draw(dt, (B, T), B, H, Hk, dk, dv, "token", seed=18)
    keep = x["S0"].clone()
    out = torch.empty_like(keep)
    print(f"\n[step {dt} {B} {T} {H} {Hk} {dk} {dv}]", flush=True)
    o = P().linear_attention_step(x["q"], x["k"], x["v"], x["g"], S=x["S0"], S_out=out, scale=0.3)
    assert torch.equal(x["S0"], keep)
    want = _oracle(x, [(b * T, (b + 1) * T) for b in range(B)], 0.3)
    _check({"o": o, "ST": out}, want, dt, ("o", "ST"))
    o2 = P().linear_attention_step(x["q"], x["k"], x["v"], x["g"], S=keep, scale=0.3)
    assert torch.equal(o, o2) and torch.equal(keep, out)


def test_prompt_then_steps_equals_the_whole():
    x = _draw(F, (2, 90), 2, 3, 3, 64, 64, "token", seed=19)
    part = lambda a, b: [x[n][:, a:b].contiguous() for n in ("q", "k", "v", "g")]
    o, ST = P().linear_attention(*part(0, 90), S0=x["S0"])
    o1, S = P().linear_attention(*part(0, 70), S0=x["S0"])
    outs = [o1]
    for t in range(70, 90):
        outs.append(P().linear_attention_step(*part(t, t + 1), S=S))
    assert O.rel2(_np(torch.cat(outs, 1)), _np(o)) < 1e-5 and O.rel2(_np(S), _np(ST)) < 1e-5


def test_same_bits_each_time_on_another_stream_and_in_a_graph():
    x = _draw(BF, (1, 700), 1, 2, 1, 128, 128, "token", seed=20)
    a, _ = _run(x, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, _ = _run(x, 1.0)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c, _ = _run(x, 1.0)
    for i in range(3):
        for n in c:
            c[n].zero_()
        x["v"].mul_(1.0 if i == 0 else 1.5)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = _run(x, 1.0)
        assert all(torch.equal(c[n], want[n]) for n in c), i


def test_non_finite_tokens_stay_in_their_sequence():
    """Rows behind the end of a packed sequence are another's: NaN there must
    not reach it."""
    cu = torch.tensor([0, 70, 100], dtype=torch.int32, device="cuda")
    x = _draw(BF, (100,), 2, 2, 2, 64, 64, "token", seed=21)
    clean, _ = _run(x, 1.0, cu_seqlens=cu, max_seqlen=70)
    for n in ("q", "k", "v", "dO", "g"):
        x[n][70:] = float("nan")
    got, _ = _run(x, 1.0, cu_seqlens=cu, max_seqlen=70)
    for n in ("o", "dq", "dk", "dv", "dg"):
        assert torch.equal(got[n][:70], clean[n][:70]), n
    assert torch.equal(got["ST"][0], clean["ST"][0]) and torch.equal(got["dS0"][0], clean["dS0"][0])


def test_gradient_against_differences():
    """The kernel's fp32 gradients along a random direction against a central
    difference of the float64 forward."""
    x = _draw(F, (1, 40), 1, 2, 1, 16, 32, "token", seed=22)
    g = P().linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], S0=x["S0"], dST=x["dST"], scale=0.4,
                                      need_dS0=True, need_dg=True)
    rng = np.random.default_rng(23)
    names = (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("S0", "dS0"))
    u = {n: rng.standard_normal(x[n].shape) for n, _ in names}

    def f(h):
        a = [(_np(x[n]) + h * u[n])[0] for n, _ in names]
        o, S = O.attend(*a, 0.4)
        return np.sum(_np(x["dO"])[0] * o) + np.sum(_np(x["dST"])[0] * S)

    got = sum(np.sum(_np(g[d]) * u[n]) for n, d in names)
    want = (f(1e-5) - f(-1e-5)) / 2e-5
    size = np.sqrt(sum(np.sum(_np(g[d]) ** 2) * np.sum(u[n] ** 2) for n, d in names))
    assert abs(got - want) < 1e-5 * size
