"""Linear attention and the norm where paths, magnitudes and workspaces meet
their limits, on the GPU against the float64 oracle.  Tolerances are those of
test_gpu_linear_attention.py and test_gpu_qk_norm.py, derived there."""
import ctypes

import numpy as np
import pytest
import torch

from tests import operators_oracle as O
from tests import test_gpu_linear_attention as LA

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def P():
    from linear_recurrent_sequence_shortconv_amd import prism
    return prism


# ------------------------------------------------------------ empty batches
@pytest.mark.parametrize("packed", [False, True])
def test_dg_of_one_decay_a_head_without_sequences(packed):
    """No sequence adds to it: zeros, written without a workspace."""
    L = P().lib()
    desc = P().LinearAttentionDesc(B=0, T=5, H=4, Hk=2, dk=32, dv=32, dtype=P().PRISM_BF16, scale=1.0)
    for n, H in (("q", 4), ("k", 2), ("v", 2), ("o", 4)):
        setattr(desc, n, P().Strides(5 * H * 32, H * 32, 32))
    desc.g = P().Strides(0, 0, 1)
    g = torch.full((4,), -0.1, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    dg = torch.full((4,), float("nan"), device="cuda")
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    st = L.prism_linear_attention_backward(
        ctypes.byref(desc), None, None, None, ptr(g), None, ptr(cu) if packed else None, None, None, None, None,
        None, ptr(dg), None, None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and dg.tolist() == [0.0] * 4


# --------------------------------------------------------------- magnitudes
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("decay", ["slow", "token", "fast", "growth"])
def test_large_magnitudes(dt, decay):
    """Keys and values of 2^36: every product of the formulas is below 2^80, and
    so far from the end of fp32 that no result overflows."""
    print(f"\n[large {dt} {decay}]", flush=True)
    x = LA._draw(dt, (1, 300), 1, 2, 2, 64, 64, "token", seed=31)
    x["k"], x["v"] = x["k"] * 2.0 ** 36, x["v"] * 2.0 ** 36
    x["S0"], x["dST"] = x["S0"] * 2.0 ** 72, x["dST"]
    if decay != "token":
        lo, hi = {"slow": (-0.2, -0.2), "fast": (-1.6, -0.8), "growth": (-0.02, 0.06)}[decay]
        x["g"] = lo + (hi - lo) * torch.rand(1, 300, 2, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    got, plain = LA._run(x, 1.0)
    want = LA._oracle(x, [(0, 300)], 1.0)
    LA._check(got, want, dt, LA.ALL)
    LA._check(plain, want, dt, ("dq", "dk", "dv", "dS0"))


@pytest.mark.parametrize("dt", [BF, F])
def test_growth(dt):
    """Positive log decays: the state grows by 2^70 over a batch of decays, and
    decay and growth alternate."""
    print(f"\n[growth {dt}]", flush=True)
    x = LA._draw(dt, (1, 300), 1, 2, 2, 64, 64, "token", seed=32)
    u = torch.rand(1, 300, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    x["g"][:, :, 0] = 0.1 + 0.2 * u
    x["g"][:, :, 1] = 4.0 * (u - 0.5)
    got, plain = LA._run(x, 1.0)
    want = LA._oracle(x, [(0, 300)], 1.0)
    LA._check(got, want, dt, LA.ALL)
    LA._check(plain, want, dt, ("dq", "dk", "dv", "dS0"))


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_infinite_tokens_stay_in_their_sequence(value):
    cu = torch.tensor([0, 70, 100], dtype=torch.int32, device="cuda")
    x = LA._draw(BF, (100,), 2, 2, 2, 64, 64, "token", seed=21)
    clean, _ = LA._run(x, 1.0, cu_seqlens=cu, max_seqlen=70)
    for n in ("q", "k", "v", "dO"):
        x[n][70:] = value
    got, _ = LA._run(x, 1.0, cu_seqlens=cu, max_seqlen=70)
    for n in ("o", "dq", "dk", "dv", "dg"):
        assert torch.equal(got[n][:70], clean[n][:70]), n
    assert torch.equal(got["ST"][0], clean["ST"][0]) and torch.equal(got["dS0"][0], clean["dS0"][0])


# -------------------------------------------------------------------- paths
def _launches(f):
    """What f launches: name -> count."""
    with P().KernelTimer() as t:
        f()
    return {n: c for n, (_, c) in t.result.items()}


@pytest.mark.parametrize("dt,B,T,H,Hk,nseg", [(BF, 1, 1100, 128, 128, 2), (F, 1, 1100, 128, 64, 2),
                                              (BF, 2, 1100, 128, 128, 1), (F, 1, 1100, 256, 256, 1)])
def test_many_heads_with_dg(dt, B, T, H, Hk, nseg):
    """As many heads as a training batch has in flight: dv in a launch of its
    own, two segments whose entering states every pass (and the decay gradient)
    forms by itself, or one segment longer than 1024 tokens, of which the last
    chunk is cut."""
    print(f"\n[many heads {dt} {B} {T} {H} {Hk}]", flush=True)
    x = LA._draw(dt, (B, T), B, H, Hk, 16, 16, "token", seed=33)
    run = lambda: P().linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], S0=x["S0"], dST=x["dST"],
                                                scale=0.5, need_dS0=True, need_dg=True)
    did = _launches(run)
    assert "la_bwd_v" in did and "la_join" not in did and ("la_states" in did) == (nseg > 1), did
    want = LA._oracle(x, [(b * T, (b + 1) * T) for b in range(B)], 0.5)
    LA._check(run(), want, dt, ("dq", "dk", "dv", "dg", "dS0"))


@pytest.mark.parametrize("T,H,join", [(577, 2, False), (700, 1, True)])
def test_state_in_place_over_segments(T, H, join):
    """A state updated in place is written while other segments still start from
    it: they then start from joined copies, also where few segments would
    otherwise form their entering states from it by themselves."""
    x = LA._draw(BF, (1, T), 1, H, H, 64, 64, "token", seed=34)
    want = LA._oracle(x, [(0, T)], 1.0)
    run = lambda S, ST: P().linear_attention(x["q"], x["k"], x["v"], x["g"], S0=S, ST=ST)
    out, S = torch.empty_like(x["S0"]), x["S0"].clone()
    did = _launches(lambda: run(x["S0"], out))
    assert "la_states" in did and ("la_join" in did) == join, did
    o, _ = run(x["S0"], out)
    LA._check({"o": o, "ST": out}, want, BF, ("o", "ST"))
    did = _launches(lambda: run(S, S))
    assert "la_join" in did, did
    S = x["S0"].clone()
    o, _ = run(S, S)
    LA._check({"o": o, "ST": S}, want, BF, ("o", "ST"))


@pytest.mark.parametrize("dt,Hk", [(BF, 1), (F, 2)])
def test_packed_over_segments(dt, Hk):
    """One long sequence (several segments) between short and empty ones."""
    lens = [3, 700, 0, 33, 1]
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = LA._draw(dt, (int(cu[-1]),), len(lens), 2, Hk, 64, 48, "token", seed=35)
    packed = {"cu_seqlens": torch.tensor(cu, dtype=torch.int32, device="cuda"), "max_seqlen": 700}
    print(f"\n[packed over segments {dt}]", flush=True)
    assert "la_states" in _launches(lambda: LA._run(x, 1.0, **packed))
    got, plain = LA._run(x, 1.0, **packed)
    want = LA._oracle(x, [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])], 1.0)
    LA._check(got, want, dt, LA.ALL)
    LA._check(plain, want, dt, ("dq", "dk", "dv", "dS0"))


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("T,H", [(90, 2), (577, 2), (1100, 2)])
def test_without_states_in_or_out(dt, T, H):
    """No final state and no state gradient wanted: in one, four and more segments."""
    x = LA._draw(dt, (1, T), 1, H, H, 64, 64, "token", seed=36, states=False)
    want = LA._oracle(x, [(0, T)], 0.7)
    print(f"\n[no states {dt} {T}]", flush=True)
    o, ST = P().linear_attention(x["q"], x["k"], x["v"], x["g"], scale=0.7, need_state=False)
    assert ST is None
    g = P().linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], scale=0.7)
    assert set(g) == {"dq", "dk", "dv"}
    LA._check({"o": o, **g}, want, dt, ("o", "dq", "dk", "dv"))


def test_packed_workspace_follows_the_rows():
    """Backward of a packed batch with one long and many short sequences takes
    memory for its rows, not for as many rows as the longest has in every
    sequence."""
    lens = [8192] + [64] * 63
    N, H, Hk, d = sum(lens), 8, 2, 64
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = LA._draw(BF, (N,), len(lens), H, Hk, d, d, "token", seed=37, states=False)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    P().linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], cu_seqlens=cu, max_seqlen=8192, need_dg=True)
    torch.cuda.synchronize()
    used = torch.cuda.max_memory_allocated() - before
    # gradients (bf16 and dg), fp32 partials of dk and dv, nine floats a row and
    # head, states of the segments (at most 64 each way) and ST
    rows = N * H * (2 * 2 * d + 4 + 2 * 4 * d + 4 * 9)
    states = len(lens) * H * d * d * 4
    assert used < 1.1 * rows + 5 * states, (used, rows, states)


# --------------------------------------------------------------------- norm
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("size", [2.0 ** -50, 2.0 ** 50])
def test_norm_backward_of_small_and_large_rows(dt, size):
    """Without eps, rows of any length whose squares fp32 holds: the gradient is
    that of the unit row over the length."""
    gen = torch.Generator(device="cuda").manual_seed(38)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    q, k, dq, dk = (r(2, 5, 3, 64) for _ in range(4))
    q, k, dq, dk = (q * size).to(dt), (k * size).to(dt), dq.to(dt), dk.to(dt)
    pos = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    turns = P().rope_turns(64)
    w = (1 + 0.2 * r(64)).to(dt)
    g = P().qk_norm_backward(q, k, dq, dk, wq=w, positions=pos, turns=turns, eps=0.0)
    n = lambda t: t.double().cpu().numpy()
    for x, dz, ww, name in ((q, dq, w, "q"), (k, dk, None, "k")):
        dx, dw = O.norm_backward(n(x), None if ww is None else n(ww), n(dz), pos.cpu().numpy(), turns.tolist(), "l2", 0.0, False)
        assert O.rel2(n(g["d" + name]), dx) < {BF: 2.1e-3, F: 1e-5}[dt]
        if ww is not None:
            assert O.rel2(n(g["dwq"]), dw) < 1e-5
