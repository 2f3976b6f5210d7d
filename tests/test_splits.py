"""The convolution, the selective scan and the verification at sizes that take
every way of splitting the work (runs, segments, parts), at many sequences, at
addresses past 32 bits, and at no tokens at all.  The references and their
tolerances are those of test_conv.py, test_ssm.py and test_verify.py; where a
segment here is longer than the 64 steps that test_ssm.py's bound counts, or a
chain longer than its 700 tokens, the bound is scaled by arithmetic given
beside the test."""
import math

import numpy as np
import pytest
import torch

import test_conv as conv
import test_ssm as ssm
import test_verify as verify

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_rnn_gdn_amd as g

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()
    return g


# B, T, C, G: waves of one channel each (G = C), so that few tokens already make many waves
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("B,T,C,G", [
    (4, 70, 32, 32),      # 384 waves of 32 tokens (768 of 32 states): segments of 16
    (24, 40, 33, 33),     # 1584: of 32
    (43, 70, 64, 64),     # 8256: of 64
    (1, 1100, 8, 8),      # 280: of 16, 69 of them in a row
    (3, 4, 5, 1), (3, 8, 5, 1), (2, 5, 5, 1),   # a piece, one short of and one past it
])
def test_gradients_by_segments_of_every_length(gdn, B, T, C, G, N, dtype):
    x = ssm._draw([T] * B, C, N, G, dtype, T + N, True, True)
    v = ssm._double(x)
    ref, sizes = ssm._gradients(v, [T] * B), ssm._gradients(v, [T] * B, sizes=True)
    d = ssm._cuda(x)
    got = gdn.ssm_bwd(**ssm._args(d), dy=d["dy"], h0=d["h0"], dh_T=d["dh_T"])
    assert set(got) == set(ref)
    # three times the root of 6 T roundings, and 30 for the exponents: 274 for 1100 tokens; 256 at least, as at fewer
    factor = max(256, 3 * math.sqrt(6 * T) + 30)
    for k, t in got.items():
        ssm._close(k, t, ref[k], factor * U * sizes[k])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("B,T,C,G", [
    (8, 300, 64, 64),     # 512 walks: 8 segments of 40
    (17, 30, 256, 256),   # 4352: one segment each
    (16, 130, 70, 70),    # 1120: segments of 48
    (1, 1500, 3, 1),      # 94 segments of 16
])
def test_forward_by_segments_of_every_length(gdn, B, T, C, G, N):
    x = ssm._draw([T] * B, C, N, G, "f32", T + N, True, True)
    ref, err = ssm._forward(ssm._double(x), [T] * B)
    d = ssm._cuda(x)
    y, hT = gdn.ssm_fwd(**ssm._args(d), h0=d["h0"])
    # (segments of at most 64 tokens: the bound as it is)
    ssm._close("y", y, ref["y"], err["y"])
    ssm._close("h_T", hT, ref["h_T"], err["h_T"])
    room = torch.empty_like(y)
    again, none = gdn.ssm_fwd(**ssm._args(d), h0=d["h0"], output_final_state=False, out=room)
    assert none is None and again.data_ptr() == room.data_ptr() and torch.equal(room, y)


def _many(kind):
    if kind == "mixed":
        return [1, 0, 2, 7, 0, 0, 3] * 90            # 630 sequences
    if kind == "empty":
        return [0] * 4990 + [1, 0, 3] + [0] * 10     # 5003, most of them empty
    return [0] * 7 + [900] + [0] * 300 + [33]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["mixed", "empty", "long"])
def test_many_packed_sequences(gdn, kind):
    lens = _many(kind)
    cu = [0] + np.cumsum(lens).tolist()
    x = ssm._draw(lens, 3, 8, 1, "f32", 5, True, True, packed=True)
    ref, err = ssm._forward(ssm._double(x), lens, True)
    d = ssm._cuda(x)
    y, hT = gdn.ssm_fwd_varlen(**ssm._args(d), cu_seqlens=cu, h0=d["h0"])
    ssm._close("y", y, ref["y"], err["y"])
    ssm._close("h_T", hT, ref["h_T"], err["h_T"])
    for C in (9, 16):
        x = conv._draw(lens, C, 4, "f32", 6, packed=True)
        ref, err = conv._reference(x, lens, True, True)
        d = conv._cuda(x)
        y, hT = gdn.conv_fwd_varlen(d["x"], d["weight"], cu, d["bias"], d["h0"])
        conv._close("y", y, ref["y"], err["y"])
        assert np.array_equal(conv._np(hT), ref["h_T"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", [
    (20, 300, 2056),    # 16-byte pieces: 9 channel tiles, runs of 64
    (12, 140, 2052),    # (bf16: single elements) runs of 32 and 64
    (2, 700, 513),      # runs of 16
    (700, 3, 8),
])
def test_convolution_gradients_by_runs_of_every_length(gdn, B, T, C, W, dtype):
    x = conv._draw([T] * B, C, W, dtype, T + W)
    ref, err = conv._reference(x, [T] * B, False, True)
    d = conv._cuda(x)
    got = gdn.conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["h0"], d["dh_T"])
    for k, t in got.items():
        conv._close(k, t, ref[k], err[k])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,C", [(1025, 16), (1023, 24), (517, 257), (300, 2056)])
def test_convolution_steps_of_many_rows(gdn, B, C, W, dtype):
    # from 1024 workgroups on a thread may take two rows: odd numbers of them, and neighbours that share a slot
    gen = torch.Generator().manual_seed(B)
    n = B + 5
    pool = torch.randn(n, W - 1, C, generator=gen).to(DT[dtype])
    slots = torch.randperm(n, generator=gen)[:B].to(torch.int32)
    slots[1], slots[7], slots[10], slots[B - 1] = slots[0], -1, n, slots[B - 2]
    x = conv._draw([1] * B, C, W, dtype, B, True, False)
    x["h0"] = torch.stack([pool[s] if 0 <= s < n else torch.zeros(W - 1, C, dtype=pool.dtype) for s in slots.tolist()])
    ref, err = conv._reference(x, [1] * B, False, True)
    want, used = conv._np(pool), set()
    for b, s in enumerate(slots.tolist()):
        if 0 <= s < n and s not in used:
            used.add(s)
            want[s] = ref["h_T"][b]
        else:
            ref["y"][b] = err["y"][b] = 0
    state = pool.cuda()
    y = gdn.conv_step(x["x"][:, 0].cuda(), x["weight"].cuda(), state, x["bias"].cuda(), slots.cuda())
    conv._close("y", y, ref["y"][:, 0], err["y"][:, 0])
    assert np.array_equal(conv._np(state), want)


@pytest.mark.gpu
def test_no_tokens(gdn):
    x = ssm._cuda(ssm._draw([0, 0], 10, 8, 2, "bf16", 1))
    y, hT = gdn.ssm_fwd(**ssm._args(x), h0=x["h0"])
    assert y.shape == (2, 0, 10) and torch.equal(hT, x["h0"])
    g = gdn.ssm_bwd(**ssm._args(x), dy=x["dy"], h0=x["h0"], dh_T=x["dh_T"])
    assert torch.equal(g["dh0"], x["dh_T"]) and all((g[k] == 0).all() for k in ("dA", "dD", "ddt_bias"))
    c = conv._cuda(conv._draw([0, 0], 10, 4, "bf16", 1))
    y, hT = gdn.conv_fwd(c["x"], c["weight"], c["bias"], c["h0"])
    assert y.shape == (2, 0, 10) and torch.equal(hT, c["h0"])
    g = gdn.conv_bwd(c["x"], c["weight"], c["dy"], c["bias"], c["h0"], c["dh_T"])
    assert torch.equal(g["dh0"], c["dh_T"]) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


@pytest.mark.gpu
def test_tokens_far_apart(gdn):
    # columns of a tensor whose rows are 2^20 elements: the last tokens lie past 2^31 elements, and past 2^32 bytes
    T, C, wide = 2200, 64, 1 << 20
    far = torch.empty(1, T, wide, device="cuda", dtype=torch.bfloat16)
    x = ssm._cuda(ssm._draw([T], C, 8, 1, "bf16", 3))
    view = dict(x)
    for i, k in enumerate(("x", "dt", "z")):
        far[..., wide - (i + 1) * C:wide - i * C] = x[k]
        view[k] = far[..., wide - (i + 1) * C:wide - i * C]
    for i, k in enumerate(("B", "C")):
        far[..., 64 * i:64 * i + 8] = x[k][:, :, 0]
        view[k] = far[..., 64 * i:64 * i + 8].unsqueeze(2)
    for a, b in zip(gdn.ssm_fwd(**ssm._args(view)), gdn.ssm_fwd(**ssm._args(x))):
        assert torch.equal(a, b)
    a, b = (gdn.ssm_bwd(**ssm._args(t), dy=x["dy"], dh_T=x["dh_T"]) for t in (view, x))
    assert all(torch.equal(a[k], b[k]) for k in b)
    w, bias = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    assert all(torch.equal(p, q) for p, q in zip(gdn.conv_fwd(view["x"], w, bias), gdn.conv_fwd(x["x"], w, bias)))
    a, b = (gdn.conv_bwd(t["x"], w, x["dy"], bias) for t in (view, x))
    assert torch.equal(a["dx"], b["dx"])
    for k in ("dweight", "dbias"):   # (sums in another order: at most 2 x 300 roundings of the terms' sizes, here below 5 each)
        assert (a[k] - b[k]).abs().max() <= 600 * U * 5 * 5 * T, k


@pytest.mark.gpu
def test_long_prompts_past_32_bits(gdn):
    # 2^31 and some elements in every tensor of tokens.  Decays of e^-1 a token and more: what lies 200 tokens back counts below
    # e^-200, so the ends have to be what calls of the ends alone give, within both calls' errors (1e-4 of the largest: they are
    # some hundred roundings of fp32), rounded to bf16.
    T, C = (1 << 19) + 100, 4096
    gen = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)
    x = dict(x=r(1, T, C), dt=r(1, T, C).abs_(), B=r(1, T, 1, 8), C=r(1, T, 1, 8), A=-1 - torch.rand(C, 8, generator=gen, device="cuda"),
             D=torch.randn(C, generator=gen, device="cuda"), z=r(1, T, C), dt_bias=torch.ones(C, device="cuda"))
    dy = r(1, T, C)
    tokens = ("x", "dt", "z", "B", "C")
    near = lambda a, b: (a.float() - b.float()).abs().max() <= (1e-4 + 2 ** -7) * b.float().abs().max()
    cut = lambda lo, hi: {k: v[:, lo:hi] if k in tokens else v for k, v in x.items()}
    first, last = cut(0, 400), cut(T - 400, T)
    y, h = gdn.ssm_fwd(**x, o_dtype=torch.bfloat16)
    y1, _ = gdn.ssm_fwd(**first, o_dtype=torch.bfloat16)
    y2, h2 = gdn.ssm_fwd(**last, o_dtype=torch.bfloat16)
    assert near(y[:, :400], y1) and near(y[:, -200:], y2[:, -200:]) and near(h, h2)
    w, bias = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    u, window = gdn.conv_fwd(x["x"], w, bias)
    u2, window2 = gdn.conv_fwd(last["x"], w, bias)
    assert torch.equal(u[:, -300:], u2[:, -300:]) and torch.equal(window, window2)
    back, back2 = gdn.conv_bwd(x["x"], w, dy, bias), gdn.conv_bwd(last["x"], w, dy[:, -400:], bias)
    assert torch.equal(back["dx"][:, -300:], back2["dx"][:, -300:])
    del u, u2, back, back2, y, y1, y2
    g = gdn.ssm_bwd(**x, dy=dy)
    g1, g2 = gdn.ssm_bwd(**first, dy=dy[:, :400].contiguous()), gdn.ssm_bwd(**last, dy=dy[:, -400:].contiguous())
    for k in ("dx", "ddt", "dz", "dB", "dC"):
        assert near(g[k][:, :200], g1[k][:, :200]), k
        assert near(g[k][:, -200:], g2[k][:, -200:]), k


@pytest.mark.gpu
def test_pools_past_32_bits(gdn):
    C, n = 16384, 8300
    gen = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = dict(x=r(2, C), dt=r(2, C), A=-r(C, 16).abs(), B=r(2, 1, 16), C=r(2, 1, 16))
    slots, small = torch.tensor([n - 1, 8200], dtype=torch.int32, device="cuda"), r(2, C, 16)
    pool = torch.empty(n, C, 16, device="cuda")
    pool[slots.long()] = small
    y, y2 = gdn.ssm_step(**x, state=pool, slots=slots), gdn.ssm_step(**x, state=small)
    assert torch.equal(y, y2) and torch.equal(pool[slots.long()], small)
    del pool
    n = 50000
    pool, small, w = torch.empty(n, 3, C, device="cuda", dtype=torch.bfloat16), r(2, 3, C).bfloat16(), r(C, 4)
    slots = torch.tensor([n - 1, 45000], dtype=torch.int32, device="cuda")
    pool[slots.long()] = small
    u = r(2, C).bfloat16()
    y, y2 = gdn.conv_step(u, w, pool, slots=slots), gdn.conv_step(u, w, small)
    assert torch.equal(y, y2) and torch.equal(pool[slots.long()], small)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_large_vocabularies(gdn, draft):
    verify._same(gdn, verify._draw(2, 2, 1_100_003, 3, draft))       # 269 parts: more than one per thread that sums them
    x = verify._draw(3, 4, 9000, 4, draft)                            # no mass, over several parts; and all of it in the last
    x["target"][0] = 0.0
    x["target"][1] = 0.0
    x["target"][1, :, 8999] = 1.0
    verify._same(gdn, x)
    if draft:   # the residual of the last refusal has no mass: the sums are made again without it
        x = verify._draw(2, 3, 9000, 5, True, tree=False)
        x["target"][:, 0, 17] = 0
        x["tokens"][:, 0] = 17
        x["draft"] = x["target"][:, :3].contiguous()
        want = verify._same(gdn, x)
        assert (want[0] == -1).all() and (want[1] >= 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,V", [(2, 32768), (2, 32769), (32, 700), (33, 700)])
def test_verification_in_one_launch_and_in_several(gdn, B, V, draft):
    # on both sides of where the forms change: siblings refused in a row, absent nodes and rows, rows without mass
    x = verify._draw(B, 12, V, V + B, draft, near=0.0)
    verify._same(gdn, x)
    x["parents"][:] = -1
    x["tokens"][:, 1::2] = x["tokens"][:, ::2]
    x["uniform"][:, :12] = 1 - 2.0 ** -24
    verify._same(gdn, x)
    x["parents"][0], x["parents"][1, 3:] = -2, 2
    x["tokens"][1, 0], x["tokens"][1, 5] = -1, V
    x["target"][0] = 0.0
    x["target"][1, :, ::3] *= -1
    x["target"][1, 0, 5:9] = float("nan")
    for u in (0.0, 0.5, 1 - 2.0 ** -24):
        x["uniform"][:, 12] = u
        verify._same(gdn, x)
    if draft:   # the last refusal leaves no mass
        x["target"][:, 0] = x["draft"][:, 0]
        x["parents"][:], x["parents"][:, 0] = -2, -1
        x["target"][:, 0, 17], x["tokens"][:, 0] = 0, 17
        want = verify._same(gdn, x)
        assert (want[0] == -1).all() and (want[1] >= 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_verification_in_several_launches_on_streams_and_in_a_graph(gdn, draft):
    x = {k: None if t is None else t.cuda() for k, t in verify._draw(5, 12, 40001, 14, draft).items()}
    call = lambda **kw: gdn.tree_verify(x["tokens"], x["parents"], x["target"], x["uniform"], draft=x["draft"], **kw)
    ref = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, here = call(stream=side), call()
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(ref, got, here))
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(ref, call(workspace=ws)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, held))
        for t in held:
            t.fill_(-9)
        assert all(torch.equal(a, b) for a, b in zip(ref, call()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_in_a_graph(gdn, dtype):
    # a token's convolution and scan captured together: every replay moves the pools on by one token, as eager calls do
    B, C, N = 3, 72, 16
    x = ssm._cuda(ssm._draw([1] * B, C, N, 2, dtype, 15, True, True))
    one = {k: v[:, 0].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in ssm._args(x).items()}
    gen = torch.Generator().manual_seed(16)
    u, w = torch.randn(B, C, generator=gen).to(DT[dtype]).cuda(), torch.randn(C, 4, generator=gen).cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    states = torch.randn(6, C, N, generator=gen).cuda(), torch.randn(6, 3, C, generator=gen).to(DT[dtype]).cuda()

    def token(state, window):
        v = gdn.conv_step(u, w, window, slots=slots)
        return gdn.ssm_step(**{**one, "x": v}, state=state, slots=slots)

    eager, held = [t.clone() for t in states], [t.clone() for t in states]
    token(*[t.clone() for t in states])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token(*held)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = token(*eager)
        assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(held, eager))


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_probabilities_past_32_bits(gdn, draft):
    B, n, V = 9, 64, 3_800_001
    gen = torch.Generator(device="cuda").manual_seed(9)
    target = torch.rand(B, n + 1, V, generator=gen, device="cuda").div_(V / 2)
    q = torch.rand(B, n, V, generator=gen, device="cuda").div_(V / 2) if draft else None
    tokens = torch.randint(0, V, (B, n), generator=gen, device="cuda", dtype=torch.int32)
    parents = torch.arange(-1, n - 1, device="cuda", dtype=torch.int32).expand(B, n).contiguous()
    uniform = torch.full((B, n + 1), 0.0, device="cuda")
    uniform[:, n] = 0.75                                  # every drafted token accepted, the next one far behind
    last, token, path = gdn.tree_verify(tokens, parents, target, uniform, draft=q)
    assert (last == n - 1).all() and (path == torch.arange(n, device="cuda")).all()
    for b in (0, B - 1):
        p = target[b, n].double().cumsum(0)
        at = int(token[b])                               # (sums of up to V numbers in another order: 1e-9 of the whole)
        assert p[at] > (0.75 - 1e-9) * p[-1] and p[at - 1] <= (0.75 + 1e-9) * p[-1]
