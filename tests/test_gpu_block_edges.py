"""What the other tests of layer_norm, short_conv and gated_recurrence leave out:
other streams, calls at the same time, captured graphs, workspaces, tensors at odd
addresses and beyond 2^31 elements, states in place behind shut gates, very many
and very long sequences, and that neighbours of results stay as they are.
Tolerances as in those tests."""
import pytest
import torch

from tests import block_oracle as O
from tests.test_gpu_gated_recurrence import both, compare, draw

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def P():
    from linear_recurrent_sequence_shortconv_amd import prism
    return prism


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _block(dt, B, T, D, seed):
    """Inputs of all operators, and a function that runs them into new tensors."""
    gen = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    t = {n: r(B, T, D).to(dt) for n in ("x", "res", "dy", "dh", "f", "i")}
    t.update(w=(1 + 0.1 * r(D)).to(dt), b=r(D).to(dt), taps=r(D, 4).to(dt), hist=r(B, 3, D).to(dt),
             lam=-torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda")), h0=r(B, D), dhT=r(B, D))

    def run():
        out = {}
        y, h = P().layer_norm(t["x"], t["w"], t["b"], residual=t["res"])
        out["y"], out["h"] = y, h
        out.update({"n" + k: v for k, v in P().layer_norm_backward(h, t["dy"], t["w"], dh=t["dh"], need_db=True).items()})
        out["last"] = torch.empty_like(t["hist"])
        u = P().short_conv(y, t["taps"], b=t["b"], hist=t["hist"], activation="silu", hist_out=out["last"])
        out["u"] = u
        out.update({"c" + k: v for k, v in P().short_conv_backward(
            y, t["taps"], t["dy"], b=t["b"], hist=t["hist"], activation="silu", need_dhist=True).items()})
        for gate in ("log", "sigmoid", "power"):
            lam = t["lam"] if gate == "power" else None
            f = t["f"] if gate != "log" else -t["f"].abs()
            s, sT = P().gated_recurrence(u, f, i=t["i"], lam=lam, h0=t["h0"], gate=gate)
            out[gate + "s"], out[gate + "T"] = s, sT
            out.update({gate + k: v for k, v in P().gated_recurrence_backward(
                u, f, s, t["dh"], i=t["i"], lam=lam, h0=t["h0"], dhT=t["dhT"], gate=gate, need_dh0=True).items()})
        return out

    return t, run


def _same(a, b):
    assert a.keys() == b.keys()
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dt,B,T,D", [(BF, 2, 700, 256), (F, 3, 301, 65), (BF, 1, 3, 128)])
def test_captured_and_replayed(dt, B, T, D):
    """A graph of all operators, replayed with other inputs and eager work of the
    same kinds in between: every replay is the eager result, bitwise."""
    t, run = _block(dt, B, T, D, 1)
    run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            out = run()
    for k in range(4):
        gen = _gen(100 + k)
        for n in ("x", "res", "dy", "f"):
            t[n].copy_(torch.randn(B, T, D, generator=gen, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in out.items()}
        _same(got, run())
        torch.cuda.synchronize()


def test_streams_and_calls_at_the_same_time():
    """Two streams at work at once, each on its own inputs: the results of one
    after the other, bitwise."""
    pairs = [_block(BF, 1, 9000, 512, 3), _block(BF, 4, 2100, 384, 4)]
    want = [run() for _, run in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    got = [None, None]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = pairs[k][1]()
        torch.cuda.synchronize()
        for k in range(2):
            _same(got[k], want[k])


def test_workspace_of_the_caller():
    """One buffer for calls one after the other; one that is too small is refused."""
    B, T, D = 2, 900, 192
    x = draw(BF, (B, T), D, B, "power", True, True, 5)
    h, hT, g = both(x, "power")
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    args = dict(i=x["i"], lam=x["lam"], h0=x["h0"], gate="power", workspace=ws)
    for _ in range(2):
        h2, hT2 = P().gated_recurrence(x["x"], x["f"], **args)
        g2 = P().gated_recurrence_backward(x["x"], x["f"], h, x["dh"], dhT=x["dhT"], need_dh0=True, **args)
        assert torch.equal(h2, h) and torch.equal(hT2, hT) and all(torch.equal(g2[n], g[n]) for n in g)
    for call in (P().gated_recurrence, lambda *a, **k: P().gated_recurrence_backward(*a, h, x["dh"], **k)):
        with pytest.raises(RuntimeError, match="workspace"):
            call(x["x"], x["f"], **{**args, "workspace": ws[:512]})
    w = torch.ones(D, device="cuda", dtype=BF)
    n = P().layer_norm_backward(x["x"], x["dh"], w)
    assert torch.equal(P().layer_norm_backward(x["x"], x["dh"], w, workspace=ws)["dw"], n["dw"])
    with pytest.raises(RuntimeError, match="workspace"):
        P().layer_norm_backward(x["x"], x["dh"], w, workspace=ws[:256])
    taps = torch.ones(D, 4, device="cuda", dtype=BF)
    with pytest.raises(RuntimeError, match="workspace"):
        P().short_conv_backward(x["x"], taps, x["dh"], workspace=ws[:256])


@pytest.mark.parametrize("dt", [BF, F])
def test_odd_addresses(dt):
    """Tensors that start one element behind an aligned address give what aligned
    ones give (sums in another order: within a rounding)."""
    B, T, D = 2, 210, 64
    t, run = _block(dt, B, T, D, 6)
    want = run()
    for n, v in t.items():
        if v.dtype == dt:
            buf = torch.empty(v.numel() + 1, dtype=dt, device="cuda")
            t[n] = buf[1:].view(v.shape)
            t[n].copy_(v)
    got = run()
    for n in want:
        tol = 2.0 ** -7 if want[n].dtype == BF else 1e-4 if dt == BF else 1e-5
        assert O.rel2(got[n].double().cpu().numpy(), want[n].double().cpu().numpy()) < tol, n


def test_beyond_32_bits():
    """Batch entries more than 2^31 elements apart."""
    B, T, D = 2, 130, 128
    far = (1 << 31) + 128
    buf = torch.zeros(far + T * D, dtype=BF, device="cuda")
    out = torch.zeros(far + T * D, dtype=BF, device="cuda")
    view = lambda b: b.as_strided((B, T, D), (far, D, 1))
    gen = _gen(7)
    x = torch.randn(B, T, D, generator=gen, device="cuda").to(BF)
    view(buf).copy_(x)
    w, taps, h0 = torch.ones(D, device="cuda", dtype=BF), torch.randn(D, 4, generator=gen, device="cuda").to(BF), None
    P().layer_norm(view(buf), w, y=view(out))
    assert torch.equal(view(out), P().layer_norm(x, w)[0])
    P().layer_norm_backward(view(buf), x, w, dx=view(out))
    assert torch.equal(view(out), P().layer_norm_backward(x, x, w)["dx"])
    P().short_conv(view(buf), taps, y=view(out))
    assert torch.equal(view(out), P().short_conv(x, taps))
    P().short_conv_backward(view(buf), taps, x, dx=view(out))
    assert torch.equal(view(out), P().short_conv_backward(x, taps, x)["dx"])
    h, hT = P().gated_recurrence(view(buf), x, h0=h0, h=view(out))
    want, wT = P().gated_recurrence(x, x, h0=h0)
    assert torch.equal(h, want) and torch.equal(hT, wT)
    g = P().gated_recurrence_backward(view(buf), x, want, x, dx=view(out))
    assert torch.equal(g["dx"], P().gated_recurrence_backward(x, x, want, x)["dx"])
    between = buf[T * D:T * D + 4096]
    assert not bool(between.any()) and not bool(out[T * D:T * D + 4096].any())


def test_state_in_place_behind_shut_gates():
    """Tiles behind a shut gate do not wait for those before them, one of which
    still reads the state that the last one replaces."""
    B, T, D = 2, 2000, 64
    x = draw(F, (B, T), D, B, "log", False, True, 8)
    x["f"][:, 256:] = -float("inf")
    h, hT, g = both(x, "log")
    compare(x, list(range(B)), "log", h, hT, g, T, F)
    for _ in range(5):
        S = x["h0"].clone()
        h2, _ = P().gated_recurrence(x["x"], x["f"], h0=S, gate="log", hT=S)
        assert torch.equal(h2, h) and torch.equal(S, hT)


def test_many_sequences():
    """1500 packed sequences of 0 to 6 tokens, more than one look through their
    offsets; first and last rows outside."""
    lens = [(5 * k) % 7 for k in range(1500)]
    cu = [3]
    for n in lens:
        cu.append(cu[-1] + n)
    N, D = cu[-1] + 5, 40
    x = draw(F, (N,), D, len(lens), "sigmoid", True, True, 9)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h, hT, g = both(x, "sigmoid", off)
    compare(x, [slice(a, b) for a, b in zip(cu[:-1], cu[1:])], "sigmoid", h, hT, g, 6, F)
    taps = torch.randn(D, 4, generator=_gen(1), device="cuda")
    hist = torch.randn(len(lens), 3, D, generator=_gen(2), device="cuda")
    last = torch.empty_like(hist)
    y = P().short_conv(x["x"], taps, hist=hist, cu_seqlens=off, hist_out=last)
    for b in range(0, 1500, 37):
        at = slice(cu[b], cu[b + 1])
        one = lambda t: t.double().cpu().numpy()
        want, end = O.short_conv(one(x["x"][at]), one(taps), None, one(hist[b]))
        assert want.size == 0 or O.rel2(one(y[at]), want) < 1e-5
        assert O.rel2(one(last[b]), end) == 0.0


@pytest.mark.parametrize("dt,T,D,gate", [(BF, 70001, 6, "power"), (F, 33000, 2, "sigmoid"), (BF, 16384, 256, "log")])
def test_one_very_long_sequence(dt, T, D, gate):
    """Few tiles that look far: the oracle, and the same in two pieces."""
    x = draw(dt, (1, T), D, 1, gate, True, True, 10)
    h, hT, g = both(x, gate)
    if D < 100:
        compare(x, [0], gate, h, hT, g, T, dt)
    cut = T // 3
    kw = dict(lam=x["lam"], gate=gate)
    at = lambda n, a, b: x[n][:, a:b]
    _, S = P().gated_recurrence(at("x", 0, cut), at("f", 0, cut), i=at("i", 0, cut), h0=x["h0"], **kw)
    h2, S = P().gated_recurrence(at("x", cut, T), at("f", cut, T), i=at("i", cut, T), h0=S, **kw)
    tol = 2.0 ** -7 if dt == BF else 1e-5
    assert O.rel2(h2.double().cpu().numpy(), h[:, cut:].double().cpu().numpy()) < tol
    assert O.rel2(S.cpu().numpy(), hT.cpu().numpy()) < 1e-4


def test_rates_of_zero_and_growth():
    """lam = 0 keeps the state and lets nothing in; log gates somewhat above 0 grow."""
    B, T, D = 2, 300, 48
    x = draw(F, (B, T), D, B, "power", True, True, 11)
    x["lam"].zero_()
    h, hT, g = both(x, "power")
    assert torch.equal(h, x["h0"][:, None].expand(B, T, D)) and torch.equal(hT, x["h0"])
    assert not bool(g["dx"].any()) and bool(torch.isfinite(g["df"]).all()) and bool(torch.isfinite(g["dlam"]).all())
    x = draw(F, (B, T), D, B, "log", False, True, 12)
    x["f"].fill_(0.02)
    h, hT, _ = both(x, "log")
    want, last = O.recur(x["x"][0].double().cpu().numpy(), x["f"][0].double().cpu().numpy(), None, None,
                         x["h0"][0].double().cpu().numpy(), "log")
    # 300 decays of a rounding and an exponent's each, all alike
    assert O.rel2(hT[0].cpu().numpy(), last) < 300 * 3 * 2.0 ** -24


@pytest.mark.parametrize("D", [48, 333, 2048])
def test_neighbours_of_results_stay(D):
    """Results into the middle of larger buffers: nothing around them changes."""
    B, T = 2, 37
    t, _ = _block(BF, B, T, D, 13)

    def framed(shape, dtype=BF):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 2 * 1024,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[1024:1024 + n].view(shape)

    def check(buf):
        assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all())

    bufs = [framed((B, T, D)) for _ in range(6)]
    v = [b[1] for b in bufs]
    P().layer_norm(t["x"], t["w"], t["b"], residual=t["res"], y=v[0], h=v[1])
    P().layer_norm_backward(v[1], t["dy"], t["w"], dx=v[2])
    hist = framed((B, 3, D))
    P().short_conv(v[0], t["taps"], hist=t["hist"], y=v[3], hist_out=hist[1])
    P().short_conv_backward(v[0], t["taps"], t["dy"], dx=v[2])
    state = framed((B, D), F)
    P().gated_recurrence(t["x"], t["f"], i=t["i"], h=v[4], hT=state[1])
    P().gated_recurrence_backward(t["x"], t["f"], v[4], t["dh"], i=t["i"], dx=v[0], df=v[1], di=v[5])
    P().gated_recurrence_step(t["x"][:, :1].contiguous(), t["f"][:, :1].contiguous(), state[1])
    torch.cuda.synchronize()
    for b, _ in bufs + [hist, state]:
        check(b)


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dt,D", [(BF, 2), (BF, 9), (BF, 15), (BF, 515), (BF, 2051), (F, 3), (F, 7), (F, 257), (F, 4099)])
def test_last_values_of_odd_rows(dt, D):
    """Rows that no whole number of vectors makes, whose last lane may be another
    wave's than the one before it (515 of eights, 257 of fours): against the oracle,
    and in place bitwise as into new tensors."""
    gen = _gen(D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    B, T, tol = 3, 70, 2.0 ** -8 + 1e-5 if dt == BF else 1e-5
    x, res, dy, dh = (r(B, T, D).to(dt) for _ in range(4))
    w, b = (1 + 0.2 * r(D)).to(dt), r(D).to(dt)
    y, h = P().layer_norm(x, w, b, residual=res)
    g = P().layer_norm_backward(h, dy, w, dh=dh, need_db=True)
    want, s = O.layer_norm(_np(x), _np(w), _np(b), _np(res))
    assert O.rel2(_np(h), s) < tol
    if D > 3:          # (of two or three values the deviation may be far below the values)
        assert O.rel2(_np(y), want) < tol
    x2, res2 = x.clone(), res.clone()
    P().layer_norm(x2, w, b, residual=res2, y=x2, h=res2)
    assert torch.equal(x2, y) and torch.equal(res2, h)
    for into in range(3):
        args = [h.clone(), dy.clone(), dh.clone()]
        gi = P().layer_norm_backward(args[0], args[1], w, dh=args[2], need_db=True, dx=args[into])
        assert torch.equal(args[into], g["dx"]) and torch.equal(gi["dw"], g["dw"]) and torch.equal(gi["db"], g["db"])
    taps, hist = r(D, 4).to(dt), r(B, 3, D).to(dt)
    u = P().short_conv(x, taps, hist=hist, activation="silu", hist_out=(last := torch.empty_like(hist)))
    gc = P().short_conv_backward(x, taps, dy, hist=hist, activation="silu", need_dhist=True)
    for k in range(B):
        want, tail = O.short_conv(_np(x[k]), _np(taps), None, _np(hist[k]), "silu")
        wc = O.short_conv_backward(_np(x[k]), _np(taps), _np(dy[k]), None, _np(hist[k]), "silu")
        assert O.rel2(_np(u[k]), want) < tol and O.rel2(_np(last[k]), tail) == 0.0
        assert O.rel2(_np(gc["dx"][k]), wc["dx"]) < tol and O.rel2(_np(gc["dhist"][k]), wc["dhist"]) < 1e-5
    hist2 = hist.clone()
    assert torch.equal(P().short_conv(x, taps, hist=hist2, activation="silu", hist_out=hist2), u)
    assert torch.equal(hist2, last)
    one = hist.clone()          # a token a call
    steps = [P().short_conv(x[:, t:t + 1], taps, hist=one, activation="silu", hist_out=one) for t in range(5)]
    assert torch.equal(torch.cat(steps, 1), u[:, :5])


def test_tensors_of_another_device_than_the_current(monkeypatch):
    """The tensors' device is current around the launch, and the other one after it
    (with one device here: the current one is said to be another)."""
    entered = []

    class device(torch.cuda.device):
        def __init__(self, index):
            entered.append(index)
            super().__init__(index)

    _, run = _block(BF, 2, 20, 64, 5)
    want = run()
    assert not entered
    monkeypatch.setattr(P(), "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", device)
    _same(run(), want)
    assert entered == [0] * 10          # (norm, convolution, three gates, forward and backward)
