"""The selective state space scan (forward, packed forward, gradients, single
tokens on a pool of states) against its definition in fp64.

Tolerances.  Roundings are at most u = 2^-24 of what is rounded.  The step size
d is computed with at most 10 of them (of its relative size), a decay a = e^{dA}
has an exponent with 12 roundings of |dA| and is rounded twice more; where a
segment's state is carried on, the exponent is a sum of up to 64 steps here
(another 64).  So the state's error E obeys, with H the state that the sizes of
all terms would give,
    E <- a E + u ((78 |dA| + 4) a H' + 13 |d x B|),
and s = <C, h> + D x is off by <|C|, E> + u (N / 4 + 6) (<|C|, H> + |D x|), the
output y = s silu(z) by that times |silu(z)| and 10 u |y|.
Gradients are sums over paths: to each contributes a chain of at most T tokens
with some 6 roundings each, which are independent and grow as the root of their
number: for T <= 700 at most 65 u of the sum of the terms' sizes; three times
that, 200 u, is asked, plus 80 u |dA| e^{-|dA|} <= 30 u for the exponents, and
for sums over tokens and channels, whose order the kernels fix, no more: 256 u.
Outputs in bf16 are rounded once more, by at most half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_rnn_gdn_amd as g

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()
    return g


def _draw(lens, C, N, G, dtype, seed, full=True, h0=True, packed=False, rate=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    n = len(lens)
    x = dict(x=r(*lead, C), dt=0.7 * r(*lead, C), B=r(*lead, G, N), C=r(*lead, G, N), z=r(*lead, C) if full else None, dy=r(*lead, C))
    x = {k: None if t is None else t.to(DT[dtype]) for k, t in x.items()}
    x["A"] = -rate * torch.exp(r(C, N))
    x["D"], x["dt_bias"] = (r(C), r(C) - 2.0) if full else (None, None)
    x["h0"] = r(n, C, N) if h0 else None
    x["dh_T"] = r(n, C, N)
    return x


NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")


def _args(x, keys=NAMES):
    return {k: x[k] for k in keys if x[k] is not None}


def _double(x):
    return {k: None if t is None else t.detach().double().cpu() for k, t in x.items()}


def _silu(v):
    return v * torch.sigmoid(v)


def _spans(lens, packed):
    ends = np.cumsum(lens)
    return [(0, int(e - n), int(e)) if packed else (i, 0, n) for i, (n, e) in enumerate(zip(lens, ends))]


def _forward(v, lens, packed=False, softplus=True):
    """y, h_T and the errors allowed of them; fp64."""
    C, N = v["A"].shape
    rep = C // v["B"].shape[2]
    y, ey = torch.zeros_like(v["x"]), torch.zeros_like(v["x"])
    hT, eT = torch.zeros(len(lens), C, N, dtype=torch.float64), torch.zeros(len(lens), C, N, dtype=torch.float64)
    step = v["dt"] if v["dt_bias"] is None else v["dt"] + v["dt_bias"]
    step = torch.nn.functional.softplus(step, threshold=200.0) if softplus else step
    for i, (b, lo, hi) in enumerate(_spans(lens, packed)):
        h = v["h0"][i].clone() if v["h0"] is not None else torch.zeros(C, N, dtype=torch.float64)
        H, E = h.abs(), torch.zeros_like(h)
        for t in range(lo, hi):
            d, x = step[b, t, :, None], v["x"][b, t, :, None]
            B, Cc = (v[k][b, t].repeat_interleave(rep, 0) for k in ("B", "C"))
            a, add = torch.exp(d * v["A"]), d * x * B
            E = a * E + U * ((78 * (d * v["A"]).abs() + 4) * a * H + 13 * add.abs())
            h, H = a * h + add, a * H + add.abs()
            s, es = (Cc * h).sum(-1), (Cc.abs() * E).sum(-1)
            size = (Cc.abs() * H).sum(-1)
            if v["D"] is not None:
                s = s + v["D"] * v["x"][b, t]
                size = size + (v["D"] * v["x"][b, t]).abs()
            es = es + U * (N / 4 + 6) * size
            if v["z"] is not None:
                g = _silu(v["z"][b, t])
                s, es = s * g, es * g.abs()
            y[b, t], ey[b, t] = s, es + 10 * U * s.abs()
        hT[i], eT[i] = h, E
    return dict(y=y, h_T=hT), dict(y=ey, h_T=eT)


def _gradients(v, lens, softplus=True, sizes=False):
    """The gradients by their formulas; ``sizes``: every term by its size."""
    size = torch.abs if sizes else (lambda t: t)
    C, N = v["A"].shape
    G = v["B"].shape[2]
    rep = C // G
    T = v["x"].shape[1]
    raw = v["dt"] if v["dt_bias"] is None else v["dt"] + v["dt_bias"]
    step = torch.nn.functional.softplus(raw, threshold=200.0) if softplus else raw
    dstep = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    D = torch.zeros(C, dtype=torch.float64) if v["D"] is None else size(v["D"])
    zeros = lambda t: torch.zeros_like(t)
    g = dict(dx=zeros(v["x"]), ddt=zeros(v["x"]), dz=zeros(v["x"]), dB=zeros(v["B"]), dC=zeros(v["C"]), dA=zeros(v["A"]),
             dD=torch.zeros(C, dtype=torch.float64), ddt_bias=torch.zeros(C, dtype=torch.float64),
             dh0=torch.zeros(len(lens), C, N, dtype=torch.float64))
    A = size(v["A"])
    for b in range(len(lens)):
        h = [size(v["h0"][b]) if v["h0"] is not None else torch.zeros(C, N, dtype=torch.float64)]
        decay = []
        for t in range(T):
            d = step[b, t, :, None]
            decay.append(torch.exp(d * v["A"]))
            h.append(decay[t] * h[t] + size(d * v["x"][b, t, :, None]) * size(v["B"][b, t]).repeat_interleave(rep, 0))
        dh = size(v["dh_T"][b]).clone()
        for t in reversed(range(T)):
            d, x, dy = size(step[b, t]), size(v["x"][b, t]), size(v["dy"][b, t])
            B, Cc = (size(v[k][b, t]).repeat_interleave(rep, 0) for k in ("B", "C"))
            if v["z"] is not None:
                z = v["z"][b, t]
                sg = torch.sigmoid(z)
                s = (Cc * h[t + 1]).sum(-1) + D * x
                # silu' = sg + z sg (1 - sg): two terms, whose difference near z = -1.278 is far smaller than both, while each
                # is rounded relative to itself: its error goes by the sum of their sizes
                g["dz"][b, t] = dy * s * (sg + size(z * sg * (1 - sg)))
                dy = dy * size(_silu(z))
            dh = dh + Cc * dy[:, None]
            g["dC"][b, t] = (dy[:, None] * h[t + 1]).view(G, rep, N).sum(1)
            g["dB"][b, t] = ((d * x)[:, None] * dh).view(G, rep, N).sum(1)
            du = (B * dh).sum(-1)
            dh = decay[t] * dh
            q = h[t] * dh
            dv = (x * du + (A * q).sum(-1)) * dstep[b, t]
            g["dx"][b, t], g["ddt"][b, t] = d * du + D * dy, dv
            g["dA"] += d[:, None] * q
            g["dD"] += dy * x
            g["ddt_bias"] += dv
        g["dh0"][b] = dh
    for name, key in (("dz", "z"), ("dD", "D"), ("ddt_bias", "dt_bias")):
        if v[key] is None:
            del g[name]
    return g


def _close(name, got, ref, err):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, name
    assert got.isfinite().all(), name
    off, bound = (got - ref).abs(), err + half * (ref.abs() + err) + 1e-30
    if off.numel():
        print(f"  {name}: worst {float((off / bound).max()):.3f} of its bound", flush=True)
    assert (off <= bound).all(), name


def _cuda(x):
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def test_reference_gradients_are_derivatives():
    for full, softplus in ((True, True), (False, False)):
        v = _double(_draw([6, 6], 4, 3, 2, "f32", 1, full))
        if not softplus:
            v["dt"] = v["dt"].abs() * 0.3
        for t in v.values():
            if t is not None:
                t.requires_grad_(True)

        def loss(w):
            step = w["dt"] + (0 if w["dt_bias"] is None else w["dt_bias"])
            step = torch.log1p(torch.exp(step)) if softplus else step
            total = 0
            for b in range(2):
                h = w["h0"][b]
                for t in range(6):
                    d = step[b, t, :, None]
                    h = torch.exp(d * w["A"]) * h + d * w["x"][b, t, :, None] * w["B"][b, t].repeat_interleave(2, 0)
                    s = (w["C"][b, t].repeat_interleave(2, 0) * h).sum(-1) + (0 if w["D"] is None else w["D"] * w["x"][b, t])
                    s = s if w["z"] is None else s * w["z"][b, t] * torch.sigmoid(w["z"][b, t])
                    total = total + (s * w["dy"][b, t]).sum()
                total = total + (h * w["dh_T"][b]).sum()
            return total

        loss(v).backward()
        with torch.no_grad():
            plain = {k: None if t is None else t.detach() for k, t in v.items()}
            g = _gradients(plain, [6, 6], softplus)
            y, _ = _forward(plain, [6, 6], softplus=softplus)
            assert abs((y["y"] * plain["dy"]).sum() + (y["h_T"] * plain["dh_T"]).sum() - loss(plain)) < 1e-9
        for name, grad in g.items():
            assert torch.allclose(grad, v[name[1:]].grad, rtol=1e-9, atol=1e-9), name
            way = torch.randn(grad.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
            with torch.no_grad():
                up, down = dict(plain), dict(plain)
                up[name[1:]], down[name[1:]] = plain[name[1:]] + 1e-5 * way, plain[name[1:]] - 1e-5 * way
                assert abs((loss(up) - loss(down)) / 2e-5 - (grad * way).sum()) < 1e-6 * (1 + (grad * way).abs().sum()), name


SIZES = [(1, 1, 1, 1), (1, 7, 5, 1), (2, 9, 64, 1), (1, 31, 65, 1), (1, 33, 130, 2), (3, 100, 48, 4), (1, 257, 192, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("B,T,C,G", SIZES)
def test_forward(gdn, B, T, C, G, N, dtype):
    for full, h0, o in ((True, True, "f32"), (False, False, dtype)):
        x = _draw([T] * B, C, N, G, dtype, T + N, full, h0)
        ref, err = _forward(_double(x), [T] * B)
        d = _cuda(x)
        y, hT = gdn.ssm_fwd(**_args(d), h0=d["h0"], o_dtype=DT[o])
        assert y.dtype == DT[o]
        _close("y", y, ref["y"], err["y"])
        _close("h_T", hT, ref["h_T"], err["h_T"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 5], [3, 0, 1, 2, 0, 40, 1, 1, 0], [32, 32, 64], [150, 1, 33, 200, 2], [1] * 70])
def test_packed(gdn, lens, N, dtype):
    for C, G, full, h0 in ((40, 2, True, True), (67, 1, False, False)):
        x = _draw(lens, C, N, G, dtype, 3 + len(lens), full, h0, packed=True)
        ref, err = _forward(_double(x), lens, True)
        d = _cuda(x)
        cu = [0] + np.cumsum(lens).tolist()
        y, hT = gdn.ssm_fwd_varlen(**_args(d), cu_seqlens=cu, h0=d["h0"], o_dtype=DT[dtype])
        _close("y", y, ref["y"], err["y"])
        _close("h_T", hT, ref["h_T"], err["h_T"])
        y2, none = gdn.ssm_fwd_varlen(**_args(d), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), h0=d["h0"],
                                      o_dtype=DT[dtype], output_final_state=False)
        assert none is None and torch.equal(y, y2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("B,T,C,G", SIZES)
def test_gradients(gdn, B, T, C, G, N, dtype):
    for full, h0 in ((True, True), (False, False)):
        x = _draw([T] * B, C, N, G, dtype, T + 2 * N, full, h0)
        v = _double(x)
        ref, sizes = _gradients(v, [T] * B), _gradients(v, [T] * B, sizes=True)
        d = _cuda(x)
        got = gdn.ssm_bwd(**_args(d), dy=d["dy"], h0=d["h0"], dh_T=d["dh_T"])
        assert set(got) == set(ref)
        for k, t in got.items():
            assert t.dtype == (DT[dtype] if k in ("dx", "ddt", "dz", "dB", "dC") else torch.float32)
            _close(k, t, ref[k], 256 * U * sizes[k])
        if not full:
            v["dh_T"] = torch.zeros_like(v["dh_T"])
            none, small = _gradients(v, [T] * B), _gradients(v, [T] * B, sizes=True)
            got = gdn.ssm_bwd(**_args(d), dy=d["dy"], h0=d["h0"])
            for k, t in got.items():
                _close(k + " without dh_T", t, none[k], 256 * U * small[k])


@pytest.mark.gpu
def test_steps_given_as_they_are(gdn):
    # no softplus, growing states (positive rates), and resets (a step so long that nothing is left)
    x = _draw([90], 70, 16, 1, "f32", 21)
    x["dt"] = x["dt"].abs() * 0.1
    x["dt"][0, 40] = 1e6
    x["x"][0, 40] *= 1e-6
    x["dt_bias"] = None
    x["A"][:5] *= -0.2
    x["dt"][0, 40, :5] = 0.1
    v = _double(x)
    ref, err = _forward(v, [90], softplus=False)
    d = _cuda(x)
    y, hT = gdn.ssm_fwd(**_args(d), h0=d["h0"], softplus=False)
    _close("y", y, ref["y"], err["y"])
    _close("h_T", hT, ref["h_T"], err["h_T"])
    g, sizes = _gradients(v, [90], False), _gradients(v, [90], False, sizes=True)
    got = gdn.ssm_bwd(**_args(d), dy=d["dy"], h0=d["h0"], dh_T=d["dh_T"], softplus=False)
    for k, t in got.items():
        _close(k, t, g[k], 256 * U * sizes[k])


@pytest.mark.gpu
def test_step_sizes_over_their_range(gdn):
    # softplus, and through it y = d x of a state without a past, to relative accuracy: 10 roundings of d, 6 of the rest
    dt = torch.cat([torch.linspace(-100, 100, 4001), torch.tensor([-0.0, 0.0, 1e-30, -1e-30, 300.0, 3e38])])
    n = dt.numel()
    one = torch.ones(1, 1, n, device="cuda")
    B = torch.zeros(1, 1, 1, 8, device="cuda")
    B[..., 0] = 1
    y, _ = gdn.ssm_fwd(one, dt.cuda().view(1, 1, n), -torch.ones(n, 8, device="cuda"), B, B)
    want = dt.double().clamp(min=0) + torch.log1p(torch.exp(-dt.double().abs()))
    off = (y.cpu().double().view(-1) - want).abs()
    assert (off <= 16 * U * want + 2.0 ** -126).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("B,C,G", [(1, 1, 1), (1, 512, 1), (5, 130, 2), (40, 2056, 4), (300, 24, 3)])
def test_step(gdn, B, C, G, N, dtype):
    gen = torch.Generator().manual_seed(B + C)
    n = B + 7
    pool = torch.randn(n, C, N, generator=gen)
    slots = torch.randperm(n, generator=gen)[:B].to(torch.int32)
    if B >= 5:
        slots[1], slots[3], slots[4] = -1, n, slots[0]      # padded, outside, an earlier row's
    for full, o in ((True, dtype), (False, "f32")):
        x = _draw([1] * B, C, N, G, dtype, B, full, False)
        v = _double(x)
        v["h0"] = torch.stack([pool[s].double() if 0 <= s < n else torch.zeros(C, N, dtype=torch.float64) for s in slots.tolist()])
        ref, err = _forward(v, [1] * B)
        want, slack, used = pool.double(), torch.zeros(n, C, N, dtype=torch.float64), set()
        for b, s in enumerate(slots.tolist()):
            if 0 <= s < n and s not in used:
                used.add(s)
                want[s], slack[s] = ref["h_T"][b], err["h_T"][b]
            else:
                ref["y"][b] = err["y"][b] = 0
        d = {k: t[:, 0] if t is not None and k in ("x", "dt", "B", "C", "z") else t for k, t in _cuda(x).items()}
        state = pool.cuda()
        y = gdn.ssm_step(**_args(d), state=state, slots=slots.cuda(), o_dtype=DT[o])
        _close("y", y, ref["y"][:, 0], err["y"][:, 0])
        _close("state", state, want, slack)
        others = [s for s in range(n) if s not in used]
        assert torch.equal(state[others].cpu(), pool[others])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(gdn, dtype):
    x = _draw([70, 70], 96, 16, 2, dtype, 31)
    ref, err = _forward(_double(x), [70, 70])
    d = _cuda(x)
    part = lambda lo, hi: {k: t[:, lo:hi].contiguous() if k in ("x", "dt", "B", "C", "z") else t for k, t in _args(d).items()}
    y, state = gdn.ssm_fwd(**part(0, 61), h0=d["h0"])
    steps = []
    for t in range(61, 70):
        one = {k: v[:, 0] if k in ("x", "dt", "B", "C", "z") else v for k, v in part(t, t + 1).items()}
        steps.append(gdn.ssm_step(**one, state=state))
    _close("y", torch.cat([y, torch.stack(steps, 1)], 1), ref["y"], err["y"])
    _close("state", state, ref["h_T"], err["h_T"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_columns_of_a_wider_tensor(gdn, dtype):
    x = _cuda(_draw([45, 45], 51, 8, 1, dtype, 41))
    wide = torch.randn(2, 45, 2 * 51 + 3, device="cuda").to(DT[dtype])
    wide[..., 1:52], wide[..., 52:103] = x["x"], x["z"]
    proj = torch.randn(2, 45, 48, device="cuda").to(DT[dtype])
    proj[..., 8:16], proj[..., 32:40] = x["B"][:, :, 0], x["C"][:, :, 0]
    view = dict(x, x=wide[..., 1:52], z=wide[..., 52:103], B=proj[..., 8:16].unsqueeze(2), C=proj[..., 32:40].unsqueeze(2))
    assert all(torch.equal(p, q) for p, q in zip(gdn.ssm_fwd(**_args(view)), gdn.ssm_fwd(**_args(x))))
    a, b = (gdn.ssm_bwd(**_args(t), dy=x["dy"]) for t in (view, x))
    assert all(torch.equal(a[k], b[k]) for k in b)


@pytest.mark.gpu
def test_bad_values_stay_in_their_channel_and_sequence(gdn):
    x = _cuda(_draw([50, 60], 70, 16, 1, "f32", 51, packed=True))
    args = _args(x)
    clean, hT = gdn.ssm_fwd_varlen(**args, cu_seqlens=[0, 50, 110], h0=x["h0"])
    bad = dict(args, x=x["x"].clone())
    bad["x"][0, 20, 3] = float("nan")
    y, h2 = gdn.ssm_fwd_varlen(**bad, cu_seqlens=[0, 50, 110], h0=x["h0"])
    touched = torch.zeros_like(y, dtype=torch.bool)
    touched[0, 20:50, 3] = True
    assert torch.equal(y[~touched], clean[~touched]) and y[0, 20:50, 3].isnan().all()
    assert torch.equal(h2[1], hT[1]) and h2[0, 3].isnan().all() and torch.equal(h2[0, :3], hT[0, :3])


@pytest.mark.gpu
def test_offsets_that_are_no_partition_stay_inside(gdn):
    x = _cuda(_draw([80], 24, 8, 1, "f32", 61, packed=True))
    h0 = torch.randn(3, 24, 8, device="cuda")
    for cu in ([-5, 90, 10, 200], [60, 70, 80, 90], [80, 0, 80, 0], [10, 20, 30, 40], [2 ** 31 - 1, -2 ** 31, 7, 3]):
        room, states = torch.full((3, 80, 24), 7.0, device="cuda"), torch.full((5, 24, 8), 7.0, device="cuda")
        gdn.ssm_fwd_varlen(**_args(x), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), h0=h0, out=room[1:2],
                           final_state=states[1:4])
        torch.cuda.synchronize()
        assert (room[0] == 7).all() and (room[2] == 7).all() and (states[0] == 7).all() and (states[4] == 7).all()


@pytest.mark.gpu
def test_streams_graphs_and_repeats(gdn):
    x = _cuda(_draw([200, 200], 200, 16, 2, "bf16", 71))

    def everything(stream=None):
        y, hT = gdn.ssm_fwd(**_args(x), h0=x["h0"], stream=stream)
        g = gdn.ssm_bwd(**_args(x), dy=x["dy"], h0=x["h0"], dh_T=x["dh_T"], stream=stream)
        return [y, hT] + [g[k] for k in sorted(g)]

    ref = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(side)
    here = everything()          # two calls at once
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(ref, got, here))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = everything()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, held))
        for t in held:
            t.zero_()
        assert all(torch.equal(a, b) for a, b in zip(ref, everything()))


@pytest.mark.gpu
def test_convolution_and_scan_as_a_layer_runs_them(gdn):
    # the gradients of a prompt through both, against the two references in a row
    gen = torch.Generator().manual_seed(81)
    x = _draw([37], 24, 8, 1, "f32", 82)
    u, w = torch.randn(1, 37, 24, generator=gen), torch.randn(24, 4, generator=gen) * 0.5
    d = _cuda(x)
    d["x"], window = gdn.conv_fwd(u.cuda(), w.cuda())
    y, hT = gdn.ssm_fwd(**_args(d), h0=d["h0"])
    g = gdn.ssm_bwd(**_args(d), dy=d["dy"], h0=d["h0"], dh_T=d["dh_T"])
    back = gdn.conv_bwd(u.cuda(), w.cuda(), g["dx"])
    v = _double(x)
    u64, w64 = u.double().requires_grad_(True), w.double().requires_grad_(True)
    pre = sum(torch.nn.functional.pad(u64, (0, 0, 3 - k, 0))[:, :37] * w64[:, k] for k in range(4))
    act = _silu(pre)
    v["x"] = act.detach()
    ref, err = _forward(v, [37])
    grads, sizes = _gradients(v, [37]), _gradients(v, [37], sizes=True)
    act.backward(grads["dx"])
    # x itself is off by up to 20 u of its terms' sizes here: ten times the scan's own bound covers it
    _close("y", y, ref["y"], 10 * err["y"] + 1e-5)
    _close("h_T", hT, ref["h_T"], 10 * err["h_T"] + 1e-5)
    for name, got, want in (("du", back["dx"], u64.grad), ("dweight", back["dweight"], w64.grad)):
        assert (got.cpu().double() - want).abs().max() <= 1e-4 * want.abs().max(), name


@pytest.mark.gpu
def test_refusals(gdn):
    x = _cuda(_draw([6, 6], 16, 8, 2, "bf16", 91))
    a = _args(x)
    one = {k: v[:, 0] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    f = lambda **kw: gdn.ssm_fwd(**{**a, **kw})
    odd = torch.zeros(2, 6, 20, device="cuda", dtype=torch.bfloat16)   # (rows of B that are no whole 16 bytes apart)
    for error, call in (
            (TypeError, lambda: f(x=a["x"].half())), (TypeError, lambda: f(dt=a["dt"].float())), (TypeError, lambda: f(A=a["A"].bfloat16())),
            (ValueError, lambda: f(dt=a["dt"][:, :5])), (ValueError, lambda: f(A=a["A"][:8])), (ValueError, lambda: f(B=a["B"][:, :, :1])),
            (ValueError, lambda: f(C=a["C"].transpose(2, 3))), (ValueError, lambda: f(x=a["x"].cpu())), (ValueError, lambda: f(D=a["D"][:3])),
            (ValueError, lambda: f(x=a["x"].transpose(1, 2).contiguous().transpose(1, 2))), (ValueError, lambda: f(x=a["x"][:, :1].expand(2, 6, 16))),
            (ValueError, lambda: f(h0=x["h0"][:1])), (TypeError, lambda: f(h0=x["h0"].bfloat16())), (TypeError, lambda: f(A=None)),
            (gdn.GdnError, lambda: f(A=a["A"][:, :4].contiguous(), B=a["B"][..., :4].contiguous(), C=a["C"][..., :4].contiguous())),
            (gdn.GdnError, lambda: f(B=odd[..., :16].unflatten(-1, (2, 8)))),
            (gdn.GdnError, lambda: gdn.ssm_fwd(**{**a, "B": torch.cat([a["B"]] * 3, 2)[:, :, :3].contiguous(), "C": torch.cat([a["C"]] * 3, 2)[:, :, :3].contiguous()})),
            (ValueError, lambda: f(out=torch.empty(2, 6, 8, device="cuda"))), (ValueError, lambda: f(final_state=x["h0"], h0=x["h0"])),
            (ValueError, lambda: f(o_dtype=torch.bfloat16, out=a["z"])), (TypeError, lambda: f(o_dtype=torch.float16)),
            (ValueError, lambda: gdn.ssm_fwd_varlen(**a, cu_seqlens=[0, 6])),
            (ValueError, lambda: gdn.ssm_bwd(**a, dy=x["dy"][:1])), (TypeError, lambda: gdn.ssm_bwd(**a, dy=x["dy"].float())),
            (gdn.GdnError, lambda: gdn.ssm_bwd(**a, dy=x["dy"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
            (ValueError, lambda: gdn.ssm_step(**one, state=x["h0"][:, :8].contiguous())), (gdn.GdnError, lambda: gdn.ssm_step(**one, state=x["h0"][:1])),
            (TypeError, lambda: gdn.ssm_step(**one, state=x["h0"], slots=torch.zeros(2, device="cuda")))):
        with pytest.raises(error):
            call()
    g = gdn.ssm_bwd(**a, dy=x["dy"])
    with pytest.raises(ValueError, match="dx overlaps x"):
        gdn.ssm_bwd(**a, dy=x["dy"], out=dict(g, dx=a["x"]))
    with pytest.raises(ValueError, match="ddt overlaps dx"):
        gdn.ssm_bwd(**a, dy=x["dy"], out=dict(g, ddt=g["dx"]))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 16, 32])
def test_gates_far_below_zero_keep_their_precision_in_the_gradients(gdn, N):
    # dh0 through segments behind the first, without decay (A = 0): the sum over 17 tokens of C dy silu(z), one channel per z.
    # silu is good to 8 roundings; a term has 3 products more, a sum of 17 terms at most 17 + 3: 31 roundings of positive terms.
    # (An exponent z log2(e) that is only rounded is off by half a unit in the place of 64 to 128 times the slope ln 2: up to
    # 45 roundings of the result, and 20 more by the rounding of log2(e).)
    gates = (-40 - torch.arange(161) * 0.25).bfloat16().unique()
    n, T = gates.numel(), 25
    z = gates.expand(1, T, n).contiguous()
    dy = torch.ones(1, T, n).bfloat16()
    dy[:, :8] = 0
    rows = torch.ones(1, T, 1, N).bfloat16()
    x = dict(x=torch.ones(1, T, n).bfloat16(), dt=torch.ones(1, T, n).bfloat16(), A=torch.zeros(n, N), B=rows, C=rows, z=z)
    got = gdn.ssm_bwd(**_cuda(x), dy=dy.cuda())["dh0"].cpu().double()
    want = 17 * _silu(gates.double()).view(1, n, 1).expand(1, n, N)
    off = ((got - want) / want).abs().max() / U
    print(f"  dh0: {float(off):.1f} roundings", flush=True)
    assert off <= 31


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("T,C", [(1, 16), (6, 70), (43, 130), (64, 24)])
def test_a_bad_last_token_leaves_the_gradients_before_it(gdn, T, C, N, dtype):
    # x of the last token is in no other token's gradients, in neither those of A (which take the states in front of a token) nor h0's
    x = _cuda(_draw([T, T], C, N, 1, dtype, 23 + T))
    call = lambda v: gdn.ssm_bwd(**dict(_args(x), x=v), dy=x["dy"], h0=x["h0"], dh_T=x["dh_T"])
    clean = call(x["x"])
    bad = x["x"].clone()
    bad[0, -1, 3], bad[1, -1, 5], bad[1, -1, C - 1] = float("inf"), float("nan"), -float("inf")
    got = call(bad)
    for k in ("dA", "dh0", "dx"):
        assert torch.equal(got[k], clean[k]), k
    for k in ("ddt", "dz", "dB", "dC"):
        assert torch.equal(got[k][:, :-1], clean[k][:, :-1]), k
    others = [c for c in range(C) if c not in (3, 5, C - 1)]
    for k in ("ddt", "dz"):
        assert torch.equal(got[k][..., others], clean[k][..., others]), k
    for k in ("dD", "ddt_bias"):
        assert torch.equal(got[k][others], clean[k][others]) and not got[k][[3, 5, C - 1]].isfinite().any(), k


@pytest.mark.gpu
@pytest.mark.parametrize("T", [12000, 30000])
@pytest.mark.parametrize("N", [8, 16, 32])
def test_growing_states_that_are_zero_for_long_stay_zero(gdn, N, T):
    # Rates above zero, no input before the last 300 tokens, no cotangent behind the first 300: over the tokens between them a
    # state would grow by far more than fp32 holds, but there is none, forward and back.  What comes out is what calls on the 300
    # tokens alone give, whose segments begin elsewhere.  All terms are positive, so each call is off by its roundings, relative
    # to the value: of exponents that add up to 300 x 0.1 x 0.5 = 15 at most, 76 u of each (12 of the exponent and 64 of sums),
    # 1140 u; of 300 tokens, 4 u each, 1200 u; of the output fewer than 60 u.  Two calls: 4800 u.
    gen = torch.Generator().manual_seed(T + N)
    C = 5
    pos = lambda *s: 0.5 + torch.rand(*s, generator=gen)
    x, dy = torch.zeros(1, T, C), torch.zeros(1, T, C)
    x[:, -300:], dy[:, :300] = pos(1, 300, C), pos(1, 300, C)
    all_ = dict(x=x, dt=torch.full((1, T, C), 0.1), A=0.3 + 0.2 * torch.rand(C, N, generator=gen), B=pos(1, T, 1, N), C=pos(1, T, 1, N))
    cut = lambda lo, hi: {k: v if k == "A" else v[:, lo:hi].contiguous() for k, v in all_.items()}
    near = lambda a, b: bool(((a - b).abs() <= 4800 * U * b).all())
    y, h = gdn.ssm_fwd(**_cuda(all_), softplus=False)
    y1, h1 = gdn.ssm_fwd(**_cuda(cut(T - 300, T)), softplus=False)
    assert (y[:, :-300] == 0).all() and near(y[:, -300:], y1) and near(h, h1)
    g = gdn.ssm_bwd(**_cuda(all_), dy=dy.cuda(), softplus=False)
    g1 = gdn.ssm_bwd(**_cuda(cut(0, 300)), dy=dy[:, :300].contiguous().cuda(), softplus=False)
    for k in ("dx", "dh0"):
        assert near(g[k][:, :300] if k == "dx" else g[k], g1[k]), k
    assert (g["dx"][:, 300:] == 0).all() and all((g[k] == 0).all() for k in ("dA", "dB", "dC", "ddt"))
