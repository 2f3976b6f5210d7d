"""The short causal convolution (forward, packed forward, gradients, single
tokens on a pool of windows) against its definition in fp64.

Tolerances.  Roundings are at most 2^-24 of what is rounded.  A value before
the activation is a sum of W products and the bias: W + 2 of them, of the sum P
of the terms' sizes at most.  silu has slope at most 1.1 and is itself computed
with fewer than 8 roundings of its value; its derivative, with slope at most
0.5, likewise.  So |y| is off by at most 2^-24 (1.1 (W + 2) P + 8 |y|), d = dy
act' by |dy| 2^-24 (0.5 (W + 2) P + 10), a gradient by the sum of those errors
over its terms and (terms + 2) 2^-24 of the terms' sizes; a sum over tokens is
made of runs of at most 64, up to 64 of them where there are that many tokens,
and pieces in fp64: fewer than 300 roundings.  Outputs in bf16 are rounded once more, by at most half a step, 2^-8 of
the value.
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


def _draw(lens, C, W, dtype, seed, bias=True, h0=True, packed=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    return dict(x=r(*lead, C).to(DT[dtype]), weight=r(C, W) * 0.5, bias=r(C) if bias else None,
                h0=r(len(lens), W - 1, C).to(DT[dtype]) if h0 else None, dy=r(*lead, C).to(DT[dtype]),
                dh_T=r(len(lens), W - 1, C).to(DT[dtype]))


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def _sigmoid(v):
    return 1 / (1 + np.exp(-v))


def _spans(lens, packed):
    ends = np.cumsum(lens)
    return [(0, int(e - n), int(e)) if packed else (i, 0, n) for i, (n, e) in enumerate(zip(lens, ends))]


def _reference(x, lens, packed, silu):
    """Outputs, gradients and the errors allowed of each."""
    v = {k: _np(t) for k, t in x.items()}
    C, W = v["weight"].shape
    w = v["weight"]
    out = {k: np.zeros_like(v["x"]) for k in ("y", "dx")}
    err = {k: np.zeros_like(v["x"]) for k in ("y", "dx")}
    for k in ("h_T", "dh0"):
        out[k], err[k] = np.zeros((len(lens), W - 1, C)), np.zeros((len(lens), W - 1, C))
    out["dweight"], err["dweight"] = np.zeros((C, W)), np.zeros((C, W))
    out["dbias"], err["dbias"] = np.zeros(C), np.zeros(C)
    for i, (b, lo, hi) in enumerate(_spans(lens, packed)):
        n = hi - lo
        long = np.concatenate([v["h0"][i] if v["h0"] is not None else np.zeros((W - 1, C)), v["x"][b, lo:hi]])
        out["h_T"][i] = long[n:]
        dlong, elong = np.zeros_like(long), np.zeros_like(long)
        dlong[n:] += v["dh_T"][i]
        elong[n:] += 2 * U * np.abs(v["dh_T"][i])
        if n:
            terms = np.stack([long[k:k + n] * w[:, k] for k in range(W)])
            pre = terms.sum(0) + (0 if v["bias"] is None else v["bias"])
            P = np.abs(terms).sum(0) + (0 if v["bias"] is None else np.abs(v["bias"]))
            s = _sigmoid(pre)
            y = pre * s if silu else pre
            slope = s * (1 + pre * (1 - s)) if silu else np.ones_like(pre)
            out["y"][b, lo:hi] = y
            err["y"][b, lo:hi] = U * (1.1 * (W + 2) * P + 8 * np.abs(y))
            dy = v["dy"][b, lo:hi]
            d = dy * slope
            ed = np.abs(dy) * U * (0.5 * (W + 2) * P + 10)
            for k in range(W):
                dlong[k:k + n] += d * w[:, k]
                elong[k:k + n] += ed * np.abs(w[:, k]) + U * (W + 4) * np.abs(d * w[:, k])
                out["dweight"][:, k] += (d * long[k:k + n]).sum(0)
                err["dweight"][:, k] += (ed * np.abs(long[k:k + n])).sum(0) + 300 * U * np.abs(d * long[k:k + n]).sum(0)
            out["dbias"] += d.sum(0)
            err["dbias"] += ed.sum(0) + 300 * U * np.abs(d).sum(0)
        out["dx"][b, lo:hi], err["dx"][b, lo:hi] = dlong[W - 1:], elong[W - 1:]
        out["dh0"][i], err["dh0"][i] = dlong[:W - 1], elong[:W - 1]
    return out, err


def _close(name, got, ref, err):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    got = _np(got)
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), name
    off, bound = np.abs(got - ref), err + half * (np.abs(ref) + err) + 1e-30
    if off.size:
        print(f"  {name}: worst {float((off / bound).max()):.3f} of its bound", flush=True)
    assert (off <= bound).all(), name


def _cuda(x):
    return {k: None if t is None else t.cuda() for k, t in x.items()}


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("lens,packed", [([5, 5], False), ([1], False), ([2], False), ([3, 0, 4, 1], True)])
def test_reference_gradients_are_differences(lens, packed, silu):
    x = {k: None if t is None else t.double() for k, t in _draw(lens, 3, 4, "f32", 5, packed=packed).items()}
    ref, _ = _reference(x, lens, packed, silu)

    def loss(**change):
        out, _ = _reference({**x, **change}, lens, packed, silu)
        return (out["y"] * _np(x["dy"])).sum() + (out["h_T"] * _np(x["dh_T"])).sum()

    gen = torch.Generator().manual_seed(1)
    for name, grad in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("h0", "dh0")):
        way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        h = 2.0 ** -10   # exact in the fp32 that _np rounds to, but for the sum: 2^-24 / 2^-10 of the loss's size
        up, down = (x[name] + h * way).float().double(), (x[name] - h * way).float().double()
        step = _np(up) - _np(down)
        diff = loss(**{name: up}) - loss(**{name: down})
        want = (ref[grad] * step).sum()
        assert abs(diff - want) <= 1e-5 * np.abs(ref[grad] * step).sum() + 1e-8, name


SIZES = [(1, 1, 8), (1, 2, 64), (2, 3, 5), (1, 4, 1), (3, 77, 129), (2, 130, 512), (1, 513, 200), (2, 33, 2056), (1, 1000, 24)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", SIZES)
def test_forward_and_gradients(gdn, B, T, C, W, dtype):
    seed = 100 * W + T
    for silu, bias, h0 in ((True, True, True), (False, False, False)):
        x = _draw([T] * B, C, W, dtype, seed, bias, h0)
        ref, err = _reference(x, [T] * B, False, silu)
        d = _cuda(x)
        act = "silu" if silu else None
        y, hT = gdn.conv_fwd(d["x"], d["weight"], d["bias"], d["h0"], activation=act)
        _close("y", y, ref["y"], err["y"])
        assert hT.dtype == d["x"].dtype and np.array_equal(_np(hT), ref["h_T"])
        got = gdn.conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["h0"], d["dh_T"], activation=act)
        assert set(got) == {"dx", "dweight", "dh0"} | ({"dbias"} if bias else set())
        for k, t in got.items():
            _close(k, t, ref[k], err[k])
        none = gdn.conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["h0"], activation=act)
        x0 = dict(x, dh_T=torch.zeros_like(x["dh_T"]))
        ref0, err0 = _reference(x0, [T] * B, False, silu)
        _close("dx without dh_T", none["dx"], ref0["dx"], err0["dx"])
        _close("dh0 without dh_T", none["dh0"], ref0["dh0"], err0["dh0"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("lens", [[1], [7], [0, 0, 5], [3, 0, 1, 2, 0, 40, 1, 1, 0], [16, 16, 16], [500, 1, 33, 700, 2], [1] * 70, [0]])
def test_packed(gdn, lens, W, dtype):
    for C, h0 in ((40, True), (1027, False)):
        x = _draw(lens, C, W, dtype, 7 + len(lens), h0=h0, packed=True)
        ref, err = _reference(x, lens, True, True)
        d = _cuda(x)
        cu = [0] + np.cumsum(lens).tolist()
        y, hT = gdn.conv_fwd_varlen(d["x"], d["weight"], cu, d["bias"], d["h0"])
        _close("y", y, ref["y"], err["y"])
        assert np.array_equal(_np(hT), ref["h_T"])
        y2, none = gdn.conv_fwd_varlen(d["x"], d["weight"], torch.tensor(cu, dtype=torch.int32, device="cuda"), d["bias"], d["h0"],
                                       output_final_state=False)
        assert none is None and torch.equal(y, y2)


@pytest.mark.gpu
def test_offsets_that_are_no_partition_stay_inside(gdn):
    x = _cuda(_draw([50], 24, 4, "bf16", 3, packed=True))
    h0 = torch.randn(3, 3, 24, device="cuda").to(torch.bfloat16)
    for cu in ([-5, 90, 10, 200], [60, 70, 80, 90], [50, 0, 50, 0], [10, 20, 30, 40], [2 ** 31 - 1, -2 ** 31, 7, 3]):
        # (which values come out is not specified: only that the call ends and writes nothing but its outputs)
        room = torch.full((3, 50, 24), 7.0, device="cuda", dtype=torch.bfloat16)
        gdn.conv_fwd_varlen(x["x"], x["weight"], torch.tensor(cu, dtype=torch.int32, device="cuda"), x["bias"], h0, out=room[1:2])
        torch.cuda.synchronize()
        assert (room[0] == 7).all() and (room[2] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,C", [(1, 1), (1, 512), (5, 129), (64, 2056), (300, 40)])
def test_step(gdn, B, C, W, dtype):
    gen = torch.Generator().manual_seed(B + C)
    n = B + 7
    pool = torch.randn(n, W - 1, C, generator=gen).to(DT[dtype])
    slots = torch.randperm(n, generator=gen)[:B].to(torch.int32)
    if B >= 5:
        slots[1], slots[3], slots[4] = -1, n, slots[0]      # padded, outside, an earlier row's
    for silu, bias in ((True, True), (False, False)):
        x = _draw([1] * B, C, W, dtype, B, bias, False)
        x["h0"] = torch.stack([pool[s] if 0 <= s < n else torch.zeros(W - 1, C, dtype=pool.dtype) for s in slots.tolist()])
        ref, err = _reference(x, [1] * B, False, silu)
        want, used = _np(pool), set()
        for b, s in enumerate(slots.tolist()):
            if 0 <= s < n and s not in used:
                used.add(s)
                want[s] = ref["h_T"][b]
            else:
                ref["y"][b] = err["y"][b] = 0
        state = pool.cuda()
        y = gdn.conv_step(x["x"][:, 0].cuda(), x["weight"].cuda(), state, None if x["bias"] is None else x["bias"].cuda(), slots.cuda(),
                          activation="silu" if silu else None)
        _close("y", y, ref["y"][:, 0], err["y"][:, 0])
        assert np.array_equal(_np(state), want)
    if B == 1:   # without slots: row b has slot b
        state = pool.cuda()
        gdn.conv_step(x["x"][:, 0].cuda(), x["weight"].cuda(), state)
        assert torch.equal(state[1:].cpu(), pool[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(gdn, dtype):
    # a prompt in two parts and single tokens give what one call gives
    x = _cuda(_draw([60, 60], 136, 4, dtype, 11))
    whole, end = gdn.conv_fwd(x["x"], x["weight"], x["bias"], x["h0"])
    a, mid = gdn.conv_fwd(x["x"][:, :33].contiguous(), x["weight"], x["bias"], x["h0"])
    b, mid = gdn.conv_fwd(x["x"][:, 33:50].contiguous(), x["weight"], x["bias"], mid)
    steps = [gdn.conv_step(x["x"][:, t], x["weight"], mid, x["bias"]) for t in range(50, 60)]
    assert torch.equal(torch.cat([a, b, torch.stack(steps, 1)], 1), whole) and torch.equal(mid, end)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,wide,at", [(64, 192, 64), (64, 200, 7), (24, 25, 1)])
def test_columns_of_a_wider_tensor(gdn, dtype, C, wide, at):
    x = _cuda(_draw([21, 21], C, 4, dtype, 12))
    proj = torch.randn(2, 21, wide, device="cuda").to(DT[dtype])
    proj[..., at:at + C] = x["x"]
    view = proj[..., at:at + C]
    assert all(torch.equal(p, q) for p, q in zip(gdn.conv_fwd(view, x["weight"], x["bias"]), gdn.conv_fwd(x["x"], x["weight"], x["bias"])))
    a, b = (gdn.conv_bwd(t, x["weight"], x["dy"], x["bias"]) for t in (view, x["x"]))
    for k in a:   # (the layouts sum over tokens in other orders)
        assert torch.allclose(a[k].float(), b[k].float(), rtol=1e-4 if a[k].dtype == torch.float32 else 2 ** -7, atol=1e-4), k
    state = torch.randn(2, 3, C, device="cuda").to(DT[dtype])
    s2 = state.clone()
    assert torch.equal(gdn.conv_step(view[:, 3], x["weight"], state), gdn.conv_step(x["x"][:, 3], x["weight"], s2)) and torch.equal(state, s2)


@pytest.mark.gpu
def test_bad_values_stay_in_their_window(gdn):
    x = _cuda(_draw([40], 16, 4, "f32", 13))
    clean, _ = gdn.conv_fwd(x["x"], x["weight"], x["bias"])
    bad = x["x"].clone()
    bad[0, 20, 3], bad[0, 30, 5] = float("nan"), float("inf")
    y, _ = gdn.conv_fwd(bad, x["weight"], x["bias"])
    touched = torch.zeros_like(y, dtype=torch.bool)
    touched[0, 20:24, 3] = touched[0, 30:34, 5] = True
    assert torch.equal(y[~touched], clean[~touched]) and y[0, 20:24, 3].isnan().all()
    far = torch.full((1, 4, 8), -1e30, device="cuda")   # silu of what is far below zero
    one = torch.ones(8, 2, device="cuda")
    y, _ = gdn.conv_fwd(far, one)
    assert (y == 0).all()
    g = gdn.conv_bwd(far, one, torch.ones_like(far))
    assert (g["dx"] == 0).all() and (g["dweight"] == 0).all()
    y, _ = gdn.conv_fwd(-far, one)
    assert (y[:, 1:] == 2e30).all()


@pytest.mark.gpu
def test_streams_graphs_and_repeats(gdn):
    x = _cuda(_draw([300, 300], 264, 4, "bf16", 14))
    def everything(stream=None):
        y, hT = gdn.conv_fwd(x["x"], x["weight"], x["bias"], x["h0"], stream=stream)
        g = gdn.conv_bwd(x["x"], x["weight"], x["dy"], x["bias"], x["h0"], x["dh_T"], stream=stream)
        return [y, hT] + [g[k] for k in sorted(g)]
    ref = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
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
def test_refusals(gdn):
    x = _cuda(_draw([6, 6], 16, 4, "bf16", 15))
    X, w, b = x["x"], x["weight"], x["bias"]
    for error, call in (
            (TypeError, lambda: gdn.conv_fwd(X.half(), w)), (TypeError, lambda: gdn.conv_fwd(X, w.bfloat16())),
            (ValueError, lambda: gdn.conv_fwd(X, w[:8].contiguous())), (ValueError, lambda: gdn.conv_fwd(X, w, b[:8])),
            (ValueError, lambda: gdn.conv_fwd(X, w, b, x["h0"][:, :2].contiguous())), (TypeError, lambda: gdn.conv_fwd(X, w, b, x["h0"].float())),
            (ValueError, lambda: gdn.conv_fwd(X.transpose(0, 1), w)), (ValueError, lambda: gdn.conv_fwd(X[:, :1].expand(2, 6, 16), w)),
            (ValueError, lambda: gdn.conv_fwd(X.transpose(1, 2).contiguous().transpose(1, 2), w)),
            (ValueError, lambda: gdn.conv_fwd(X.cpu(), w)), (ValueError, lambda: gdn.conv_fwd(X, w.cpu())),
            (ValueError, lambda: gdn.conv_fwd(X, w, activation="relu")), (gdn.GdnError, lambda: gdn.conv_fwd(X, torch.ones(16, 5, device="cuda"))),
            (gdn.GdnError, lambda: gdn.conv_fwd(X, torch.ones(16, 1, device="cuda"))),
            (ValueError, lambda: gdn.conv_fwd(X, w, out=X)), (ValueError, lambda: gdn.conv_fwd(X, w, final_state=X.view(-1)[:96].view(2, 3, 16))),
            (ValueError, lambda: gdn.conv_fwd_varlen(X, w, [0, 6])), (ValueError, lambda: gdn.conv_fwd_varlen(X[:1], w, [0])),
            (ValueError, lambda: gdn.conv_bwd(X, w, x["dy"][:1])), (TypeError, lambda: gdn.conv_bwd(X, w, x["dy"].float())),
            (TypeError, lambda: gdn.conv_bwd(X, w, x["dy"], workspace=X)),
            (gdn.GdnError, lambda: gdn.conv_bwd(X, w, x["dy"], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
            (ValueError, lambda: gdn.conv_step(X[:, 0], w, x["h0"][:, :2].contiguous())),
            (gdn.GdnError, lambda: gdn.conv_step(X[:, 0], w, x["h0"][:1])),
            (ValueError, lambda: gdn.conv_step(X[:, 0], w, x["h0"], slots=torch.zeros(3, dtype=torch.int32, device="cuda"))),
            (TypeError, lambda: gdn.conv_step(X[:, 0], w, x["h0"], slots=torch.zeros(2, device="cuda")))):
        with pytest.raises(error):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [8192, 8191])
def test_steps_of_rows_far_apart(gdn, dtype, C):
    # one token of a batch of longer prompts: the rows lie more than 2^20 elements apart
    prompts = torch.randn(3, 130, C, device="cuda").to(DT[dtype])
    w, state = torch.randn(C, 4, device="cuda"), torch.randn(3, 3, C, device="cuda").to(DT[dtype])
    assert prompts[:, 77].stride(0) > 1 << 20
    s2 = state.clone()
    y = gdn.conv_step(prompts[:, 77], w, state)
    assert torch.equal(y, gdn.conv_step(prompts[:, 77].contiguous(), w, s2)) and torch.equal(state, s2)


@pytest.mark.gpu
def test_steps_of_rows_as_far_apart_as_they_may_be(gdn):
    apart, C = (1 << 31) - 1, 24
    room = torch.empty(apart + C, device="cuda", dtype=torch.bfloat16)
    x, small = room.as_strided((2, C), (apart, 1)), torch.randn(2, C, device="cuda").bfloat16()
    x.copy_(small)
    w, state = torch.randn(C, 3, device="cuda"), torch.randn(2, 2, C, device="cuda").bfloat16()
    s2 = state.clone()
    assert torch.equal(gdn.conv_step(x, w, state), gdn.conv_step(small, w, s2)) and torch.equal(state, s2)
    with pytest.raises(gdn.GdnError):   # (a prompt's tokens may not)
        gdn.conv_fwd(x.unsqueeze(0), w)
    with pytest.raises(gdn.GdnError):
        gdn.conv_bwd(x.unsqueeze(0), w, small.unsqueeze(0))


@pytest.mark.gpu
def test_steps_of_rows_far_apart_on_a_stream_and_in_a_graph(gdn):
    C = 8192
    prompts, w, first = torch.randn(3, 130, C, device="cuda").bfloat16(), torch.randn(C, 4, device="cuda"), torch.randn(4, 3, C, device="cuda").bfloat16()
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    eager, held, aside = first.clone(), first.clone(), first.clone()
    want = gdn.conv_step(prompts[:, 5].contiguous(), w, eager, slots=slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.conv_step(prompts[:, 5], w, aside, slots=slots, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(aside, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gdn.conv_step(prompts[:, 5], w, held, slots=slots)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(held, eager)
        prompts[:, 5] = torch.randn(3, C, device="cuda").bfloat16()
        want = gdn.conv_step(prompts[:, 5].contiguous(), w, eager, slots=slots)


@pytest.mark.gpu
def test_rows_too_far_apart_are_called_that(gdn):
    C = 16
    room = torch.empty((1 << 31) + C, device="cuda", dtype=torch.bfloat16)
    x, w, state = room.as_strided((2, C), (1 << 31, 1)), torch.randn(C, 4, device="cuda"), torch.zeros(2, 3, C, device="cuda", dtype=torch.bfloat16)
    for call in (lambda: gdn.conv_step(x, w, state), lambda: gdn.conv_fwd(x.unsqueeze(0), w)):
        with pytest.raises(ValueError, match="x: tokens must be fewer than 2\\^31 elements apart"):
            call()
    with pytest.raises(ValueError, match="x: tokens must not overlap"):
        gdn.conv_step(room.as_strided((2, C), (C - 1, 1)), w, state)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T,C", [(1, 16), (5, 8), (40, 16), (64, 24), (131, 17)])
def test_a_bad_last_token_stays_with_its_tap(gdn, T, C, W, dtype):
    # without an activation a gradient of the weights is a sum of d[t] x[t - (W - 1) + w]: the last token's x is in the last tap's alone
    x = _cuda(_draw([T, T], C, W, dtype, 17 + T, h0=False))
    call = lambda v: gdn.conv_bwd(v, x["weight"], x["dy"], x["bias"], dh_T=x["dh_T"], activation=None)
    clean = call(x["x"])
    bad = x["x"].clone()
    bad[0, -1, 3], bad[1, -1, 5], bad[1, -1, C - 1] = float("inf"), float("nan"), -float("inf")
    got = call(bad)
    for k in ("dx", "dbias", "dh0"):
        assert torch.equal(got[k], clean[k]), k
    touched = torch.zeros_like(got["dweight"], dtype=torch.bool)
    touched[[3, 5, C - 1], W - 1] = True
    assert torch.equal(got["dweight"][~touched], clean["dweight"][~touched]) and not got["dweight"][touched].isfinite().any()
