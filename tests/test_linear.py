"""Linear attention with a decay per head in chunks (forward, packed forward,
gradients) against its definition in fp64, every pair of tokens at a time.

Tolerances.  Sums are kept in fp32 (decay sums in fp64) and the matrix cores'
operands as bf16 planes: three planes hold all 24 bits of a value, so every
rounding is at most 2^-24 of the value rounded; two planes (the state and the
scores, where o is rounded to bf16 anyway) leave 2^-17.  An element is a sum
over at most one segment's walk: 2048 tokens at most / 32 per chunk = 64 state
updates of up to 128 products each plus the chunk's own, independent
roundings that add as the root of their number, at most
sqrt(64 x 128) = 91 x 2^-24 = 5.4e-6 of a term, whose size the RMS bounds to
within the peak factor of these draws, below 8: 4.3e-5.  What is asked of fp32
outputs is 5e-5 of the tensor's RMS; of bf16 ones half a step of bf16,
2^-8 |x|, and for the two planes 8 x 2^-17 = 6.1e-5 of the RMS, together
1.2e-4.  The decays' gradient is a difference of sums over up to 2048 tokens
of terms of its own size: sqrt(2048) = 45 x 2^-24 more relative to terms up to
the peak factor of its RMS, 2.2e-5: 1e-4 of the RMS is asked.  Summed over all tokens for a
decay that is shared by them, the terms add up with either sign: the bound is
1e-4 of the root of the sum of the squares of the tokens' gradients.
"""
import numpy as np
import pytest
import torch

D = 128
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_rnn_gdn_amd as g

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()
    return g


def _draw(B, T, Hqk, Hv, dtype, seed, fixed=False, rows=None, h0=0.1, strength=3.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    rows = B if rows is None else rows
    return dict(q=unit(r(B, T, Hqk, D)).to(DT[dtype]), k=unit(r(B, T, Hqk, D)).to(DT[dtype]), v=r(B, T, Hv, D).to(DT[dtype]),
                g=torch.nn.functional.logsigmoid(r(*((Hv,) if fixed else (B, T, Hv))) + strength),
                h0=h0 * r(rows, Hv, D, D) if h0 else None, dO=r(B, T, Hv, D).to(DT[dtype]), dh_T=0.1 * r(rows, Hv, D, D))


def _reference(x, spans, grads=False):
    """fp64 on the GPU (plain matrix products), one sequence and head at a time."""
    x = {n: None if t is None else t.cuda().double() for n, t in x.items()}
    q, k, v, h0 = x["q"], x["k"], x["v"], x["h0"]
    B, T, Hv = v.shape[:3]
    R = Hv // k.shape[2]
    g = x["g"].clamp(min=-200.0).expand(B, T, Hv)
    o, hT = torch.zeros_like(v), torch.zeros((len(spans), Hv, D, D), dtype=torch.float64, device="cuda")
    out = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v), dg=torch.zeros_like(v[..., 0]),
               dh0=torch.zeros_like(hT))
    for i, (b, lo, hi) in enumerate(spans):
        for h in range(Hv):
            S0 = torch.zeros(D, D, dtype=torch.float64, device="cuda") if h0 is None else h0[i, h]
            dS = x["dh_T"][i, h] if x["dh_T"] is not None else torch.zeros_like(S0)
            if hi == lo:
                hT[i, h], out["dh0"][i, h] = S0, dS
                continue
            qs, ks, vs, gs = q[b, lo:hi, h // R], k[b, lo:hi, h // R], v[b, lo:hi, h], g[b, lo:hi, h]
            n = hi - lo
            G = gs.cumsum(0)
            t = torch.arange(n, device="cuda")
            W = torch.where(t[:, None] >= t, (G[:, None] - G).clamp(max=0).exp(), 0.0) if float(gs.max()) <= 0 else \
                (G[:, None] - G).masked_fill(t[:, None] < t, -float("inf")).exp()
            head, tail = G.exp()[:, None], (G[-1] - G).exp()[:, None]
            A = (qs @ ks.T) * W
            o[b, lo:hi, h] = A @ vs + head * (qs @ S0)
            hT[i, h] = ks.T @ (tail * vs) + G[-1].exp() * S0
            if not grads:
                continue
            dO = x["dO"][b, lo:hi, h]
            dA = (dO @ vs.T) * W
            dq = dA @ ks + head * (dO @ S0.T)
            dk = dA.T @ qs + tail * (vs @ dS.T)
            out["dv"][b, lo:hi, h] = A.T @ dO + tail * (ks @ dS)
            out["dh0"][i, h] = qs.T @ (head * dO) + G[-1].exp() * dS
            d = (qs * dq).sum(1) - (ks * dk).sum(1)
            out["dg"][b, lo:hi, h] = d.flip(0).cumsum(0).flip(0) + (hT[i, h] * dS).sum()
            out["dq"][b, lo:hi, h // R] += dq
            out["dk"][b, lo:hi, h // R] += dk
    return o, hT, out


def _close(name, got, ref, tol, bf16=False, rms=None):
    got, ref = got.double().cpu().numpy(), ref.cpu().numpy()
    assert got.shape == ref.shape, name
    if not ref.size:
        return
    rms = max(float(np.sqrt(np.mean(ref ** 2))), 1e-30) if rms is None else rms
    bound = tol * rms + (np.abs(ref) * 2.0 ** -8 if bf16 else 0.0)
    off = np.abs(got - ref)
    print(f"  {name}: worst {float((off / bound).max()):.3f} of its bound, rms {rms:.3e}", flush=True)
    assert np.isfinite(got).all() and (off <= bound).all(), name


def _cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def _check_fwd(o, hT, o_ref, h_ref, o_dtype):
    _close("o", o, o_ref, 1.2e-4 if o_dtype == "bf16" else 5e-5, bf16=o_dtype == "bf16")
    if hT is not None:
        _close("h_T", hT, h_ref, 5e-5)


SHAPES = [
    # B, T, H_qk, H_v, fixed, h0
    (1, 1, 1, 1, False, 0.1),
    (2, 31, 1, 2, True, 0.0),
    (1, 32, 1, 1, False, 0.1),
    (1, 33, 2, 2, False, 0.0),
    (3, 64, 1, 3, False, 0.1),
    (2, 65, 2, 4, True, 0.1),
    (1, 257, 1, 2, False, 0.1),      # two segments, the second of one token
    (2, 700, 3, 9, False, 0.0),      # odd heads, three segments
    (1, 2500, 2, 4, False, 0.1),     # more segments than the scan takes at a time
    (5, 300, 16, 64, True, 0.1),     # 320 heads: whole states per workgroup, one segment
    (40, 70, 4, 16, False, 0.0),     # 640
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,o_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,T,Hqk,Hv,fixed,h0", SHAPES)
def test_forward(gdn, B, T, Hqk, Hv, fixed, h0, dtype, o_dtype):
    x = _draw(B, T, Hqk, Hv, dtype, seed=T + Hv, fixed=fixed, h0=h0)
    o_ref, h_ref, _ = _reference(x, [(b, 0, T) for b in range(B)])
    c = _cuda(x)
    o, hT = gdn.linear_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], o_dtype=DT[o_dtype])
    _check_fwd(o, hT, o_ref, h_ref, o_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,o_dtype,fixed", [("bf16", "bf16", False), ("bf16", "f32", True), ("f32", "f32", False)])
@pytest.mark.parametrize("lens", [
    [5], [0, 7, 0], [64, 1, 130, 63], [300, 0, 1000, 2, 511], [1] * 40, [17, 33] * 150, [3000, 1]])
def test_forward_packed(gdn, lens, dtype, o_dtype, fixed):
    Hqk, Hv = 1, 2
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = cu[-1]
    x = _draw(1, T, Hqk, Hv, dtype, seed=T, fixed=fixed, rows=len(lens))
    o_ref, h_ref, _ = _reference(x, [(0, cu[i], cu[i + 1]) for i in range(len(lens))])
    c = _cuda(x)
    o, hT = gdn.linear_chunk_fwd_varlen(c["q"], c["k"], c["v"], c["g"], cu, c["h0"], o_dtype=DT[o_dtype])
    _check_fwd(o, hT, o_ref, h_ref, o_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[900, 40, 300, 0, 1500, 700], [1, 199, 100, 0, 200] * 8])
def test_forward_packed_many_heads(gdn, lens):
    # few long walks (one workgroup per compute unit) and many short ones
    Hqk, Hv = 16, 32
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    x = _draw(1, cu[-1], Hqk, Hv, "bf16", seed=len(lens), rows=len(lens))
    o_ref, h_ref, _ = _reference(x, [(0, cu[i], cu[i + 1]) for i in range(len(lens))])
    c = _cuda(x)
    for turn in range(2):  # segments of one length start in any order: the results are the same
        o, hT = gdn.linear_chunk_fwd_varlen(c["q"], c["k"], c["v"], c["g"], cu, c["h0"])
        _check_fwd(o, hT, o_ref, h_ref, "bf16" if o.dtype == torch.bfloat16 else "f32")
        if turn == 0:
            first = o.clone(), hT.clone()
    assert torch.equal(first[0], o) and torch.equal(first[1], hT)


@pytest.mark.gpu
def test_packed_offsets_that_are_no_partition_touch_nothing_else(gdn):
    # results are unspecified, but only the outputs may change: the inputs and
    # guard rows around the outputs keep their values
    Hqk, Hv, T, n = 1, 2, 300, 5
    x = _cuda(_draw(1, T, Hqk, Hv, "bf16", seed=1, rows=n))
    keep = {a: t.clone() for a, t in x.items() if t is not None}
    for cu in ([-5, 100, 50, 2 ** 31 - 1, 7, 300], [0, 300, 0, 300, 0, 300], [300, 200, 100, 50, 20, 0],
               [0, 10, 20, 30, 40, 100]):
        buf = torch.full((T + 128, Hv, D), 7.0, device="cuda")
        st = torch.full((n + 2, Hv, D, D), 7.0, device="cuda")
        gdn.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["g"], cu, x["h0"], out=buf[64:-64].unsqueeze(0),
                                    final_state=st[1:-1])
        torch.cuda.synchronize()
        assert (buf[:64] == 7).all() and (buf[-64:] == 7).all() and (st[[0, -1]] == 7).all()
        # rows behind the last sequence are left as they were
        if cu[-1] == 100:
            assert (buf[64 + 100:] == 7).all()
        assert all(torch.equal(x[a], t) for a, t in keep.items())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hqk,Hv,fixed,h0", SHAPES[:9] + [(6, 300, 16, 64, True, 0.1), (1, 4200, 1, 1, False, 0.1)])
def test_gradients(gdn, B, T, Hqk, Hv, fixed, h0, dtype):
    x = _draw(B, T, Hqk, Hv, dtype, seed=2 * T + Hv, fixed=fixed, h0=h0)
    if h0 == 0.0:
        x["dh_T"] = None
    _, _, ref = _reference(x, [(b, 0, T) for b in range(B)], grads=True)
    c = _cuda(x)
    got = gdn.linear_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["dO"], h0=c["h0"], dh_T=c["dh_T"])
    assert all(got[n].dtype == DT[dtype] for n in ("dq", "dk", "dv"))
    for n in ("dq", "dk", "dv"):
        _close(n, got[n], ref[n], 5e-5, bf16=dtype == "bf16")
    _close("dh0", got["dh0"], ref["dh0"], 5e-5)
    if fixed:
        rms = float(ref["dg"].square().sum((0, 1)).max().sqrt())
        _close("dg", got["dg"], ref["dg"].sum((0, 1)), 1e-4, rms=rms)
    else:
        _close("dg", got["dg"], ref["dg"], 1e-4)


@pytest.mark.gpu
def test_gradients_against_differences(gdn):
    # the loss of the fp32 forward, moved along one random direction per input:
    # central differences in steps of 2^-4 (the loss is linear in v and h0 and
    # a polynomial of degree 2 in q, k together; in g its third derivative is
    # of the loss's own size, off by h^2 / 6 = 6.5e-4 of the slope) against the
    # gradients' inner products; the forward's own error (5e-5 of the outputs)
    # over the step: 16 x 5e-5 of the loss's spread.  2e-3 of the norms of
    # gradient and direction, over the root of their size, covers both.
    B, T, Hqk, Hv = 1, 150, 1, 2
    x = _cuda(_draw(B, T, Hqk, Hv, "f32", seed=6))
    got = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], h0=x["h0"], dh_T=x["dh_T"])

    def loss(**kw):
        a = dict(x, **kw)
        o, h = gdn.linear_chunk_fwd(a["q"], a["k"], a["v"], a["g"], a["h0"])
        return float((o.double() * x["dO"].double()).sum() + (h.double() * x["dh_T"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    step = 2.0 ** -4
    for name in ("q", "k", "v", "g", "h0"):
        d = torch.randn(x[name].shape, generator=gen, device="cuda")
        if name == "g":
            d = d * 0.1
        d = d / d.norm() * x[name].norm() * (0.1 if name == "g" else 1.0)
        slope = (loss(**{name: x[name] + step * d}) - loss(**{name: x[name] - step * d})) / (2 * step)
        grad = got["d" + name].double()
        want = float((grad * d.double()).sum())
        scale = float(grad.norm() * d.norm().double()) / grad.numel() ** 0.5
        print(f"  d{name}: {want:.6f} against {slope:.6f}, scale {scale:.4f}", flush=True)
        assert abs(want - slope) <= 2e-3 * max(scale, abs(want)) + 16 * 5e-5 * float(x["dO"].norm()) * 0.1


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["resets", "strong", "none", "growing"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_decays(gdn, case, dtype):
    # resets: g = -inf, the type's lowest value, and -1000 at some tokens (one of
    # them a segment's first); strong: -20 everywhere; none: 0; growing: g > 0
    B, T, Hqk, Hv = 1, 300, 1, 2
    x = _draw(B, T, Hqk, Hv, dtype, seed=3)
    if case == "resets":
        x["g"][0, 37, 0], x["g"][0, 256, 1], x["g"][0, 257, 0], x["g"][0, 70] = -float("inf"), torch.finfo(torch.float32).min, -1000.0, -500.0
    else:
        x["g"] = torch.full_like(x["g"], dict(strong=-20.0, none=0.0, growing=0.01)[case])
    o_ref, h_ref, ref = _reference(x, [(0, 0, T)], grads=True)
    c = _cuda(x)
    o, hT = gdn.linear_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"])
    _check_fwd(o, hT, o_ref, h_ref, "f32")
    got = gdn.linear_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["dO"], h0=c["h0"], dh_T=c["dh_T"])
    for n in ("dq", "dk", "dv", "dh0"):
        _close(n, got[n], ref[n], 5e-5, bf16=dtype == "bf16" and n != "dh0")
    # dg sums differences <q, dq> - <k, dk> in which a token's pair with itself
    # cancels.  With decays of e^-20 that pair is all there is: dg is 1e-9 of the
    # terms, and what is left is their rounding, 2^-24 of |q| |dq| + |k| |dk| each
    # (an inner product's rounding is relative to the product of the norms),
    # over at most 256 tokens of a segment: sqrt(256) 2^-24 = 9.6e-7 of the
    # terms, x 8 for the largest of them
    terms = None
    if case == "strong":
        norm = lambda a: x[a].double().norm(dim=-1).cuda() * ref["d" + a].norm(dim=-1)
        terms = float((norm("q") + norm("k")).max())
    _close("dg", got["dg"], ref["dg"], 1e-4 if terms is None else 8 * 9.6e-7, rms=terms)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_sequences(gdn, dtype):
    x = _cuda(_draw(3, 0, 1, 2, dtype, seed=3))
    o, hT = gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"])
    assert o.numel() == 0 and torch.equal(hT, x["h0"])
    _, hT = gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
    assert torch.count_nonzero(hT) == 0
    one = {a: x[a][:1].contiguous() for a in ("q", "k", "v", "g")}
    _, hT = gdn.linear_chunk_fwd_varlen(one["q"], one["k"], one["v"], one["g"], [0, 0, 0, 0], x["h0"])
    assert torch.equal(hT, x["h0"])
    got = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], h0=x["h0"], dh_T=x["dh_T"])
    assert torch.equal(got["dh0"], x["dh_T"]) and got["dq"].numel() == 0
    got = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], torch.zeros(2, device="cuda"), x["dO"])
    assert torch.count_nonzero(got["dg"]) == 0 and torch.count_nonzero(got["dh0"]) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(gdn, dtype):
    # a serving run: packed prompts into pool slots, then single tokens, against
    # the forward over the whole sequences
    lens, extra, Hqk, Hv = [70, 300, 1], 5, 1, 2
    n, Tm = len(lens), max(lens) + extra
    x = _cuda(_draw(n, Tm, Hqk, Hv, dtype, seed=8))
    pool = torch.zeros((6, Hv, D, D), device="cuda")
    slots = [4, 1, 3]
    pk = {a: torch.cat([x[a][i, :m] for i, m in enumerate(lens)]).unsqueeze(0).contiguous() for a in ("q", "k", "v", "g")}
    _, hT = gdn.linear_chunk_fwd_varlen(pk["q"], pk["k"], pk["v"], pk["g"], np.cumsum([0] + lens).tolist())
    pool[slots] = hT
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    outs = []
    for t in range(extra):
        a = {m: torch.stack([x[m][i, lens[i] + t] for i in range(n)]).contiguous() for m in ("q", "k", "v", "g")}
        outs.append(gdn.step(a["q"], a["k"], a["v"], a["g"], None, pool, slots=sl))
    for i, m in enumerate(lens):
        w = {a: x[a][i:i + 1, :m + extra].clone() for a in ("q", "k", "v", "g")}
        o, h = gdn.linear_chunk_fwd(w["q"], w["k"], w["v"], w["g"])
        rms = float(o.square().mean().sqrt())
        got = torch.stack([y[i] for y in outs])
        assert float((got - o[0, m:]).abs().max()) <= 1e-4 * rms
        assert float((pool[slots[i]] - h[0]).abs().max()) <= 1e-4 * float(h.square().mean().sqrt())


@pytest.mark.gpu
def test_training_step_in_a_graph(gdn):
    # forward and gradients recorded once and replayed with eager work between, bit for bit
    x = _cuda(_draw(2, 600, 2, 4, "bf16", seed=10))

    def work():
        o, h = gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], o_dtype=torch.bfloat16)
        return [o, h] + list(gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dh_T"]).values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(3):
        x["v"].copy_(torch.randn(x["v"].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)))
        ref = work()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.gpu
def test_workspace_holds_nothing_between_calls(gdn):
    # one workspace, filled with NaN, larger than needed, used by both calls in turn on a stream of the caller's
    x = _cuda(_draw(1, 900, 1, 2, "bf16", seed=11))
    ref = gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"])
    gref = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dh_T"])
    shape = gdn.GdnLinearShape(1, 900, 1, 2, 128, 128, 0, 1, 0)
    need = max(gdn.workspace_size_linear(shape, m) for m in (gdn.LINEAR_FWD, gdn.LINEAR_BWD))
    ws = torch.full(((need + 1023) // 1024 * 1024,), 255, dtype=torch.uint8, device="cuda")
    mine = torch.cuda.Stream()
    mine.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        got = gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], workspace=ws, stream=mine)
        grads = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dh_T"], workspace=ws, stream=mine)
    mine.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert all(torch.equal(grads[n], gref[n]) for n in gref)
    with pytest.raises(gdn.GdnError):
        gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], workspace=ws[:256])


@pytest.mark.gpu
def test_two_calls_at_once(gdn):
    # forward and gradients of two problems on two streams, started together,
    # against the same calls one after the other, bit for bit
    xs = [_cuda(_draw(1, 1500 + 300 * i, 2, 4, "bf16", seed=20 + i, fixed=bool(i))) for i in range(2)]

    def work(x, stream=None):
        o, h = gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], stream=stream)
        return [o, h] + list(gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dh_T"],
                                                  stream=stream).values())

    ref = [work(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = [work(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.gpu
def test_offsets_of_a_call_on_another_stream(gdn):
    # offsets given as a list belong to the call's stream: the current stream's
    # next allocations must not get their memory while that stream is busy
    lens = [300, 1, 700, 64]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    x = _cuda(_draw(1, cu[-1], 1, 2, "bf16", seed=41, rows=len(lens)))
    ref = gdn.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["g"], cu, x["h0"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = gdn.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["g"], cu, x["h0"], stream=s)
    fill = [torch.zeros(len(cu), dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert len(fill) == 8 and all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,C", [("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_sequence(gdn, dtype, C, bad):
    # tokens 210 .. of the middle sequence, and what lies behind the last one:
    # the other sequences, and the chunks before, keep their bits
    lens, at = [70, 401, 33], 210
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    x = _cuda(_draw(1, cu[-1] + 50, 1, 2, dtype, seed=51, rows=len(lens)))
    o, h = gdn.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["g"], cu, x["h0"], o_dtype=DT[dtype])
    y = {n: t.clone() for n, t in x.items()}
    for n in ("q", "k", "v"):
        y[n][0, cu[1] + at:cu[2]] = bad
        y[n][0, cu[3]:] = bad
    o2, h2 = gdn.linear_chunk_fwd_varlen(y["q"], y["k"], y["v"], y["g"], cu, x["h0"], o_dtype=DT[dtype])
    assert torch.equal(o2[0, :cu[1] + at // C * C], o[0, :cu[1] + at // C * C])
    assert torch.equal(o2[0, cu[2]:cu[3]], o[0, cu[2]:cu[3]])
    assert torch.equal(h2[[0, 2]], h[[0, 2]])
    assert not torch.isfinite(o2[0, cu[1] + at:cu[2]]).any() and not torch.isfinite(h2[1]).any()


@pytest.mark.gpu
def test_runs_agree_bit_for_bit(gdn):
    # no atomics: the same call gives the same bits, whatever else ran before
    x = _cuda(_draw(2, 777, 2, 6, "bf16", seed=31, fixed=True))
    first = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dh_T"])
    for _ in range(3):
        torch.randn(1 << 22, device="cuda").sum()
        again = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dh_T"])
        assert all(torch.equal(again[n], first[n]) for n in first)


# ---------------------------------------------------------------------------
# refusals (no GPU needed: everything is rejected before a launch)


@pytest.fixture(scope="module")
def abi():
    import os

    import linear_attention_rnn_gdn_amd as g

    if not os.path.exists(g.LIB_PATH):
        from linear_attention_rnn_gdn_amd import build

        build.build()
    g.lib()
    return g


def test_linear_calls_refuse_bad_arguments(abi):
    L = abi.lib()
    ok, odd, null, big = 1 << 20, (1 << 20) + 4, None, 1 << 40
    sizes = dict(B=2, T=4000, H_qk=2, H_v=4, d_k=128, d_v=128, g_fixed=0, dtype=1, o_dtype=0)

    def shape(**kw):
        return abi.GdnLinearShape(*{**sizes, **kw}.values())

    calls = {
        # entry point: pointers before the workspace, those that may be NULL
        abi.LINEAR_FWD: (L.gdn_linear_chunk_fwd, 7, {4, 6}),                      # q k v g h0 o h_T
        abi.LINEAR_VARLEN: (L.gdn_linear_chunk_fwd_varlen, 8, {5, 7}),            # cu q k v g h0 o h_T
        abi.LINEAR_BWD: (L.gdn_linear_chunk_bwd, 12, {4, 6, 11}),                 # q k v g h0 dO dh_T dq dk dv dg dh0
    }
    for kind, (f, count, optional) in calls.items():
        good = [ok] * count
        ws = abi.workspace_size_linear(shape(), kind)
        assert ws > 0
        for i in range(count):
            if i not in optional:
                assert f(shape(), *(good[:i] + [null] + good[i + 1:]), ok, ws, null) == -1, (kind, i)
            assert f(shape(), *(good[:i] + [odd] + good[i + 1:]), ok, ws, null) == -4, (kind, i)
        assert f(shape(), *good, null, ws, null) == -1
        assert f(shape(), *good, odd, ws, null) == -4
        assert f(shape(), *good, ok, ws - 1, null) == -5
        assert f(None, *good, ok, ws, null) == -1
        for bad, status in ((dict(B=0), -2), (dict(T=-1), -2), (dict(H_qk=0), -2), (dict(H_v=5), -2), (dict(d_k=64), -2),
                            (dict(d_v=256), -2), (dict(g_fixed=-1), -2), (dict(dtype=2), -3), (dict(o_dtype=7), -3),
                            (dict(H_qk=1, H_v=(1 << 14) + 1), -2), (dict(B=1 << 25, T=1), -2)):
            assert f(shape(**bad), *good, ok, big, null) == status, (kind, bad)
            with pytest.raises(abi.GdnError):
                abi.workspace_size_linear(shape(**bad), kind)
    assert L.gdn_linear_chunk_fwd(shape(B=2, T=1 << 30), *([ok] * 7), ok, big, null) == -2   # tokens past 32 bits
    with pytest.raises(abi.GdnError):
        abi.workspace_size_linear(shape(), 3)


def test_linear_workspace_sizes(abi):
    s = lambda **kw: abi.GdnLinearShape(*{**dict(B=1, T=60, H_qk=2, H_v=4, d_k=128, d_v=128, g_fixed=0, dtype=1, o_dtype=0),
                                          **kw}.values())
    assert abi.workspace_size_linear(s(), abi.LINEAR_FWD) == 0            # one segment: no workspace
    assert abi.workspace_size_linear(s(T=20000), abi.LINEAR_FWD) > 0
    assert abi.workspace_size_linear(s(), abi.LINEAR_VARLEN) > 0
    # the largest shapes do not overflow
    assert abi.workspace_size_linear(s(B=3000, T=700000, H_v=2), abi.LINEAR_BWD) > 1 << 38
    assert abi.workspace_size_linear(s(B=1, T=2 ** 31 - 1, H_v=2), abi.LINEAR_VARLEN) > 0


@pytest.mark.gpu
def test_linear_bindings_refuse_what_does_not_fit(gdn):
    x = _cuda(_draw(2, 40, 1, 2, "bf16", seed=1))
    args = dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"])
    bad = [("q", x["q"].float(), TypeError), ("q", x["q"][:, :20], ValueError), ("k", x["k"].half(), TypeError),
           ("v", x["v"][..., :64].contiguous(), ValueError), ("v", x["v"].transpose(1, 2), ValueError), ("g", x["g"].double(), TypeError),
           ("g", x["g"][:, :, :1].contiguous(), ValueError), ("g", x["g"].cpu(), ValueError), ("v", x["v"][0], ValueError)]
    for key, value, err in bad:
        with pytest.raises((err, gdn.GdnError) if key == "v" else err):
            gdn.linear_chunk_fwd(**dict(args, **{key: value}))
        with pytest.raises((err, gdn.GdnError) if key == "v" else err):
            gdn.linear_chunk_bwd(**dict(args, **{key: value}), dO=x["dO"])
    with pytest.raises(TypeError):
        gdn.linear_chunk_bwd(**args, dO=x["dO"].float())
    with pytest.raises(ValueError):
        gdn.linear_chunk_fwd(**args, h0=x["h0"][:1])
    with pytest.raises(ValueError):   # the final state written over the initial one
        gdn.linear_chunk_fwd(**args, h0=x["h0"], final_state=x["h0"])
    with pytest.raises(ValueError):
        gdn.linear_chunk_fwd_varlen(**args, cu_seqlens=[0, 40])
    one = {a: t[:1].contiguous() for a, t in args.items()}
    with pytest.raises(ValueError):
        gdn.linear_chunk_fwd_varlen(**one, cu_seqlens=[0])
    with pytest.raises(TypeError):
        gdn.linear_chunk_fwd_varlen(**one, cu_seqlens=torch.tensor([0, 40], device="cuda"))


def test_linear_sizes_that_no_launch_holds_are_refused(abi):
    # a launch holds fewer than 2^32 threads: 16 workgroups of 256 per state and
    # role in the scan, one of 512 per walk
    at = dict(B=1 << 16, T=1, H_qk=2, H_v=4, d_k=128, d_v=128, g_fixed=0, dtype=1, o_dtype=0)
    for kind in (abi.LINEAR_FWD, abi.LINEAR_VARLEN, abi.LINEAR_BWD):
        abi.workspace_size_linear(abi.GdnLinearShape(*at.values()), kind)
        with pytest.raises(abi.GdnError):
            abi.workspace_size_linear(abi.GdnLinearShape(*{**at, "B": (1 << 16) + 1}.values()), kind)
    long = dict(at, B=1, T=(1 << 29) - 1)   # B T H_v just below 2^31
    abi.workspace_size_linear(abi.GdnLinearShape(*long.values()), abi.LINEAR_BWD)
    with pytest.raises(abi.GdnError):
        abi.workspace_size_linear(abi.GdnLinearShape(*{**long, "H_v": 64}.values()), abi.LINEAR_BWD)
