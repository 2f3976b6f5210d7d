"""Operators on a pool of recurrent states (single-token step, drafted trees,
commit of an accepted path) against the rule applied token by token in fp64.

Tolerances.  The kernels keep sums and states in fp32 and split matrix-core
operands into planes that hold all 24 bits of an fp32 value, so each rounding
is at most 2^-24 of the value rounded.  An element here is reached through at
most 256 of them (a sum over 128 state rows, up to 64 dependent tree steps,
each of which contracts: |k| = 1, 0 < beta < 1, decays <= 1, and up to 64
added nodes); they are independent, so they grow as the root of their number,
16 x 2^-24, and a value is at most 16 times its tensor's RMS in these draws:
16 x 16 x 2^-24 = 1.5e-5.  2e-5 of the RMS is asked, and in addition half a
step of bf16, 2^-8 |o|, where o is rounded to bf16.
"""
import numpy as np
import pytest
import torch

DK = 128


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_rnn_gdn_amd as g

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()
    return g


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _draw(B, n, Hqk, Hv, n_slots, dtype, seed, fixed=False, delta=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    lead = (B,) if n is None else (B, n)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    x = dict(q=unit(r(*lead, Hqk, DK)).to(DT[dtype]), k=unit(r(*lead, Hqk, DK)).to(DT[dtype]),
             v=r(*lead, Hv, DK).to(DT[dtype]),
             g=torch.nn.functional.logsigmoid(r(*((Hv,) if fixed else lead + (Hv,))) + 3.0),
             beta=torch.sigmoid(r(*lead, Hv)) if delta else None, state=0.3 * r(n_slots, Hv, DK, DK))
    return x


def _token(S, q, k, v, g, beta):
    """One token's rule in fp64 on S [H, d_k, d_v]; returns (S', o, u)."""
    S = np.exp(g)[:, None, None] * S
    u = v if beta is None else beta[:, None] * (v - np.einsum("hkv,hk->hv", S, k))
    S = S + k[:, :, None] * u[:, None, :]
    return S, np.einsum("hkv,hk->hv", S, q), u


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def _heads(x, Hv):
    return None if x is None else np.repeat(x, Hv // x.shape[-2], axis=-2)


def _per_token(g, lead, Hv):
    return np.broadcast_to(g, lead + (Hv,))


def _close(name, got, ref, bf16=False):
    got, ref = _np(got), np.asarray(ref)
    assert got.shape == ref.shape
    rms = max(float(np.sqrt(np.mean(ref ** 2))), 1e-30)
    bound = 2e-5 * rms + (np.abs(ref) * 2.0 ** -8 if bf16 else 0.0)
    off = np.abs(got - ref)
    print(f"  {name}: worst {float((off / bound).max()):.3f} of its bound, rms {rms:.3e}", flush=True)
    assert np.isfinite(got).all() and (off <= bound).all(), name


def _cuda(x):
    return {k: (None if v is None else v.cuda()) for k, v in x.items()}


def _step_ref(x, slots):
    S = _np(x["state"])
    B, Hv = x["v"].shape[:2]
    q, k = _heads(_np(x["q"]), Hv), _heads(_np(x["k"]), Hv)
    v, g, beta = _np(x["v"]), _per_token(_np(x["g"]), (B,), Hv), _np(x["beta"])
    o, seen = np.zeros(v.shape), set()
    for b, s in enumerate(slots):
        if not 0 <= s < S.shape[0] or s in seen:
            continue
        seen.add(s)
        S[s], o[b], _ = _token(S[s], q[b], k[b], v[b], g[b], None if beta is None else beta[b])
    return o, S


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,o_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,Hqk,Hv,delta,fixed", [
    (1, 1, 1, True, False),       # the smallest call: 32 columns per workgroup
    (1, 16, 32, True, True),
    (5, 3, 9, False, False),      # odd heads, linear rule
    (7, 8, 32, True, False),      # 224 heads in all: 64 columns per workgroup
    (33, 8, 16, False, True),     # 528: whole states
])
def test_step(gdn, dtype, o_dtype, B, Hqk, Hv, delta, fixed):
    n_slots = B + 3
    x = _draw(B, None, Hqk, Hv, n_slots, dtype, seed=B + Hv, fixed=fixed, delta=delta)
    slots = np.random.RandomState(B).permutation(n_slots)[:B].tolist()
    o_ref, S_ref = _step_ref(x, slots)
    c = _cuda(x)
    o = gdn.step(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"],
                 slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), o_dtype=DT[o_dtype])
    _close("o", o, o_ref, o_dtype == "bf16")
    _close("state", c["state"], S_ref)
    untouched = [s for s in range(n_slots) if s not in slots]
    assert torch.equal(c["state"][untouched].cpu(), x["state"][untouched])


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hv", [(6, 2), (300, 2)])
def test_step_rows_without_a_state(gdn, B, Hv):
    # padded rows (-1), slots past the pool, and rows naming an earlier row's
    # slot: zero outputs, nothing written for them
    n_slots = 290
    x = _draw(B, None, 1, Hv, n_slots, "f32", seed=3)
    slots = np.random.RandomState(1).permutation(n_slots).tolist() + list(range(10))
    slots = slots[:B]
    slots[1], slots[2], slots[-1], slots[-2] = -1, n_slots, slots[0], 2 ** 31 - 1
    o_ref, S_ref = _step_ref(x, slots)
    c = _cuda(x)
    out = torch.full((B, Hv, DK), float("nan"), device="cuda")
    o = gdn.step(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"],
                 slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), out=out)
    assert o is out and torch.count_nonzero(o[[1, 2, B - 1, B - 2]]) == 0
    _close("o", o, o_ref)
    _close("state", c["state"], S_ref)


@pytest.mark.gpu
def test_steps_equal_the_chunked_forward(gdn):
    # 70 single-token steps without slots against the chunked forward of the
    # same tokens (its own bar for bf16 inputs: 2e-2 of the RMS)
    B, T, Hqk, Hv = 2, 70, 2, 4
    gen = torch.Generator().manual_seed(4)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q, k = (unit(torch.randn(B, T, Hqk, DK, generator=gen)).bfloat16().cuda() for _ in range(2))
    v = torch.randn(B, T, Hv, DK, generator=gen).bfloat16().cuda()
    g = torch.nn.functional.logsigmoid(torch.randn(B, T, Hv, generator=gen) + 3).cuda()
    beta = torch.sigmoid(torch.randn(B, T, Hv, generator=gen)).cuda()
    state = (0.1 * torch.randn(B, Hv, DK, DK, generator=gen)).cuda()
    o_ref, h_ref = gdn.chunk_fwd(q, k, v, g, beta, state.clone(), chunk=64)
    o = torch.stack([gdn.step(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(), g[:, t].contiguous(),
                              beta[:, t].contiguous(), state) for t in range(T)], 1)
    for a, b in ((o, o_ref), (state, h_ref)):
        assert float((a - b).abs().max()) <= 2e-2 * float(b.square().mean().sqrt())


@pytest.mark.gpu
@pytest.mark.parametrize("g", [float("-inf"), -3.0e38, -150.0, 0.0])
def test_step_extreme_decays(gdn, g):
    # a decay to nothing leaves k u^T alone, g = 0 keeps the state
    x = _draw(2, None, 1, 2, 2, "f32", seed=9)
    x["g"] = torch.full_like(x["g"], g)
    ref = dict(x, g=torch.full_like(x["g"], max(g, -200.0)))
    o_ref, S_ref = _step_ref(ref, [0, 1])
    c = _cuda(x)
    o = gdn.step(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"])
    _close("o", o, o_ref)
    _close("state", c["state"], S_ref)


# ---------------------------------------------------------------------------
# drafted trees


def _parents(kind, B, n, seed):
    rs = np.random.RandomState(seed)
    if kind == "chain":
        p = np.tile(np.arange(n) - 1, (B, 1))
    elif kind == "star":
        p = np.full((B, n), -1)
    elif kind == "random":
        p = np.array([[rs.randint(-1, r) if r else -1 for r in range(n)] for _ in range(B)])
    else:   # "broken": absent nodes among the others, their descendants absent too, a self and a forward reference
        p = np.array([[rs.randint(-1, r) if r else -1 for r in range(n)] for _ in range(B)])
        p[0, n // 2:] = -2
        p[-1, n // 3] = n // 3
        p[-1, n // 2] = n + 5
        p[-1, -1] = 2 ** 31 - 1
        p[0, 0] = -2 ** 31
    return p.astype(np.int32)


def _tree_ref(x, parents, slots):
    S0 = _np(x["state"])
    B, n, Hv = x["v"].shape[:3]
    q, k = _heads(_np(x["q"]), Hv), _heads(_np(x["k"]), Hv)
    v, g, beta = _np(x["v"]), _per_token(_np(x["g"]), (B, n), Hv), _np(x["beta"])
    o, u, states = np.zeros(v.shape), np.zeros(v.shape), []
    for b, s in enumerate(slots):
        at = {}
        if 0 <= s < S0.shape[0]:
            at[-1] = S0[s]
            for r in range(n):
                p = int(parents[b, r])
                if p < r and p in at:
                    at[r], o[b, r], u[b, r] = _token(at[p], q[b, r], k[b, r], v[b, r], g[b, r],
                                                     None if beta is None else beta[b, r])
        states.append(at)
    return o, u, states


TREES = [
    # B, n, H_qk, H_v, kind
    (1, 1, 1, 1, "chain"),
    (2, 5, 1, 2, "random"),
    (3, 16, 2, 2, "chain"),
    (2, 17, 1, 3, "star"),
    (4, 32, 2, 4, "random"),
    (2, 33, 1, 1, "broken"),
    (2, 64, 1, 2, "chain"),
    (3, 63, 2, 4, "random"),
    (3, 13, 1, 2, "broken"),
    (130, 9, 2, 4, "random"),     # 520 heads in all: both halves of the columns in one workgroup
    (130, 40, 2, 4, "broken"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,o_dtype,delta,fixed", [
    ("bf16", "bf16", True, False), ("bf16", "f32", False, False), ("f32", "f32", True, True), ("f32", "bf16", False, True)])
@pytest.mark.parametrize("B,n,Hqk,Hv,kind", TREES)
def test_tree(gdn, B, n, Hqk, Hv, kind, dtype, o_dtype, delta, fixed):
    n_slots = min(B, 6) + 2
    x = _draw(B, n, Hqk, Hv, n_slots, dtype, seed=n + B, fixed=fixed, delta=delta)
    parents = _parents(kind, B, n, seed=n)
    rs = np.random.RandomState(n)
    slots = rs.randint(0, n_slots, B)          # rows share slots: forks of one sequence
    if B > 2:
        slots[1], slots[2] = -1, n_slots
    o_ref, u_ref, states = _tree_ref(x, parents, slots)
    # what absent nodes hold must not matter
    dead = torch.tensor([[r not in states[b] for r in range(n)] for b in range(B)])
    for key in ("q", "k", "v", "beta") + (() if fixed else ("g",)):
        if x[key] is not None:
            x[key][dead] = float("nan")
    c = _cuda(x)
    dev = dict(parents=torch.from_numpy(parents).cuda(), slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    before = c["state"].clone()
    o, u = gdn.tree_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], dev["parents"], c["state"], slots=dev["slots"],
                        o_dtype=DT[o_dtype])
    assert torch.equal(c["state"], before)
    _close("o", o, o_ref, o_dtype == "bf16")
    _close("u", u, u_ref)
    # commit one node of every row; a slot takes its first row's
    last = rs.randint(-1, n + 1, B)
    last[0] = n - 1
    S_ref, seen = _np(before), set()
    for b, s in enumerate(slots):
        if 0 <= s < n_slots and s not in seen:
            seen.add(s)
            if last[b] >= 0 and last[b] in states[b]:
                S_ref[s] = states[b][last[b]]
    for name in ("u",):
        u[dead.cuda()] = float("nan")
    got = gdn.tree_commit(c["k"], u, c["g"], dev["parents"], torch.tensor(last, dtype=torch.int32, device="cuda"),
                          c["state"], slots=dev["slots"])
    assert got is c["state"]
    _close("state", got, S_ref)


@pytest.mark.gpu
def test_tree_of_a_chain_equals_steps(gdn):
    # decode 12 tokens one by one, or check them as a chain and commit the 9th
    B, n, Hqk, Hv = 3, 12, 2, 4
    x = _cuda(_draw(B, n, Hqk, Hv, 5, "bf16", seed=12))
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    parents = (torch.arange(n, dtype=torch.int32) - 1).repeat(B, 1).cuda()
    o, u = gdn.tree_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], parents, x["state"], slots=slots)
    pool = x["state"].clone()
    for t in range(9):
        ot = gdn.step(*(x[a][:, t].contiguous() for a in ("q", "k", "v", "g", "beta")), pool, slots=slots)
        assert float((ot - o[:, t]).abs().max()) <= 2e-5 * float(ot.square().mean().sqrt())
    gdn.tree_commit(x["k"], u, x["g"], parents, torch.tensor([8, 8, -1], dtype=torch.int32, device="cuda"), x["state"],
                    slots=slots)
    rms = float(pool.square().mean().sqrt())
    assert float((pool[[4, 0]] - x["state"][[4, 0]]).abs().max()) <= 2e-5 * rms
    assert not torch.equal(pool[2], x["state"][2])


@pytest.mark.gpu
@pytest.mark.parametrize("delta", [True, False])
def test_tree_resets(gdn, delta):
    # a hard reset on a path (g = -inf or below any exponent) makes the nodes behind it forget the state
    x = _draw(2, 24, 1, 2, 2, "f32", seed=5, delta=delta)
    parents = _parents("chain", 2, 24, 0)
    x["g"][0, 7], x["g"][1, 3], x["g"][1, 20] = float("-inf"), -3.0e38, -1000.0
    ref = dict(x, g=x["g"].clamp(min=-200.0))
    o_ref, u_ref, states = _tree_ref(ref, parents, [0, 1])
    c = _cuda(x)
    p = torch.from_numpy(parents).cuda()
    o, u = gdn.tree_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], p, c["state"])
    _close("o", o, o_ref)
    _close("u", u, u_ref)
    gdn.tree_commit(c["k"], u, c["g"], p, torch.tensor([23, 23], dtype=torch.int32, device="cuda"), c["state"])
    _close("state", c["state"], np.stack([states[b][23] for b in range(2)]))


@pytest.mark.gpu
def test_pool_calls_in_a_graph_and_on_another_stream(gdn):
    # check, commit and step recorded in one graph, replayed three times with
    # eager work between, each replay against the eager calls bit for bit
    B, n, Hqk, Hv = 3, 6, 2, 4
    x = _cuda(_draw(B, n, Hqk, Hv, 4, "bf16", seed=21))
    y = _cuda(_draw(B, None, Hqk, Hv, 4, "bf16", seed=22))
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    parents = torch.from_numpy(_parents("random", B, n, 3)).cuda()
    last = torch.tensor([5, 2, -1], dtype=torch.int32, device="cuda")
    pool = x["state"]

    def work(state):
        o, u = gdn.tree_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], parents, state, slots=slots)
        gdn.tree_commit(x["k"], u, x["g"], parents, last, state, slots=slots)
        return o, u, gdn.step(y["q"], y["k"], y["v"], y["g"], y["beta"], state, slots=slots)

    eager = pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(pool)
    for _ in range(3):
        ref = work(eager)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
        assert torch.equal(pool, eager)
    # a stream of the caller's, not the current one
    mine = torch.cuda.Stream()
    mine.wait_stream(torch.cuda.current_stream())
    a = gdn.step(y["q"], y["k"], y["v"], y["g"], y["beta"], pool, slots=slots, stream=mine)
    mine.synchronize()
    b = gdn.step(y["q"], y["k"], y["v"], y["g"], y["beta"], eager, slots=slots)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(pool, eager)


@pytest.mark.gpu
def test_step_far_into_a_large_pool(gdn):
    # a slot whose offset passes 2^31 elements (and 2^33 bytes)
    Hv = 32
    n_slots = 4200                        # 4200 x 32 x 16384 = 2.2e9 elements
    state = torch.empty((n_slots, Hv, DK, DK), device="cuda")
    x = _draw(2, None, 16, Hv, 2, "bf16", seed=8)
    slots = [n_slots - 1, 1]
    state[slots] = x["state"].cuda()
    o_ref, S_ref = _step_ref(x, [0, 1])
    c = _cuda(x)
    o = gdn.step(c["q"], c["k"], c["v"], c["g"], c["beta"], state,
                 slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    _close("o", o, o_ref)
    _close("state", state[slots], S_ref)


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


def test_pool_calls_refuse_bad_arguments(abi):
    import ctypes

    L = abi.lib()
    ok, odd, null = 1 << 20, (1 << 20) + 4, None
    sizes = dict(B=4, n=1, H_qk=2, H_v=4, d_k=128, d_v=128, n_slots=8, g_fixed=0, dtype=1, o_dtype=0)

    def shape(**kw):
        return abi.GdnPoolShape(*{**sizes, **kw}.values())

    calls = {
        # entry point: (pointers, those that may be NULL)
        "gdn_step": (L.gdn_step, 8, {4, 5}),              # q k v g beta slots state o
        "gdn_tree_fwd": (L.gdn_tree_fwd, 10, {4, 6}),     # q k v g beta parents slots state o u
        "gdn_tree_commit": (L.gdn_tree_commit, 7, {5}),   # k u g parents last slots state
    }
    for name, (f, count, optional) in calls.items():
        good = [ok] * count
        for i in range(count):
            if i not in optional:
                assert f(shape(), *(good[:i] + [null] + good[i + 1:]), null) == -1, (name, i)
            assert f(shape(), *(good[:i] + [odd] + good[i + 1:]), null) == -4, (name, i)
        for bad, status in ((dict(B=0), -2), (dict(n=0), -2), (dict(n=65), -2), (dict(H_qk=0), -2), (dict(H_v=5), -2),
                            (dict(d_k=64), -2), (dict(d_v=256), -2), (dict(n_slots=0), -2), (dict(g_fixed=2), -2),
                            (dict(dtype=3), -3), (dict(o_dtype=-1), -3), (dict(B=1 << 26, H_v=4), -2)):
            assert f(shape(**bad), *good, null) == status, (name, bad)
        # without slots every row needs a slot of its own
        no_slots = list(good)
        no_slots[max(optional)] = null
        assert f(shape(B=9), *no_slots, null) == -2, name
        assert f(None, *good, null) == -1, name
    assert L.gdn_step(shape(n=2), *([ok] * 8), null) == -2


def test_pool_sizes_that_no_launch_holds_are_refused(abi):
    # a launch holds fewer than 2^32 threads: two workgroups of 256 per state;
    # pointers that are refused later tell the largest size from one past it
    L = abi.lib()
    odd = (1 << 20) + 4
    for f, count in ((L.gdn_step, 8), (L.gdn_tree_fwd, 10), (L.gdn_tree_commit, 7)):
        for B, status in ((1 << 20, -4), ((1 << 20) + 1, -2)):
            shape = abi.GdnPoolShape(B, 1, 2, 4, 128, 128, 1 << 21, 0, 1, 0)
            assert f(shape, *([odd] * count), None) == status


def test_pool_bindings_refuse_host_tensors(abi):
    x = _draw(2, None, 1, 2, 2, "bf16", seed=1)
    with pytest.raises(ValueError):
        abi.step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"])
    with pytest.raises(TypeError):
        abi.step(x["q"].half(), x["k"].half(), x["v"].half(), x["g"], x["beta"], x["state"])
    with pytest.raises(ValueError):
        abi.tree_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], torch.zeros(2, 1, dtype=torch.int32), x["state"])


@pytest.mark.gpu
def test_pool_bindings_refuse_what_does_not_fit(gdn):
    B, n, Hqk, Hv = 2, 3, 1, 2
    x = _cuda(_draw(B, n, Hqk, Hv, 4, "bf16", seed=1))
    p = torch.tensor([[-1, 0, 1]] * B, dtype=torch.int32, device="cuda")
    args = dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], beta=x["beta"], parents=p, state=x["state"])
    bad = [("q", x["q"].float(), TypeError), ("q", x["q"][:, :2].contiguous(), ValueError), ("g", x["g"].double(), TypeError),
           ("g", x["g"][:1], ValueError), ("v", x["v"].transpose(0, 1), ValueError), ("beta", x["beta"][0], ValueError),
           ("parents", p.long(), TypeError), ("state", x["state"].bfloat16(), TypeError), ("state", x["state"][:, :1].contiguous(), ValueError),
           ("state", x["state"].cpu(), ValueError), ("state", x["state"].transpose(2, 3), ValueError)]
    for key, value, err in bad:
        with pytest.raises(err):
            gdn.tree_fwd(**dict(args, **{key: value}))
    with pytest.raises(TypeError):
        gdn.tree_fwd(**args, slots=torch.zeros(B, dtype=torch.int64, device="cuda"))
    with pytest.raises(gdn.GdnError):   # no slots and fewer states than rows
        gdn.tree_fwd(**dict(args, state=x["state"][:1]))
    many = 65
    big = {k: (None if v is None else v.cuda()) for k, v in _draw(B, many, Hqk, Hv, 4, "bf16", seed=2).items()}
    with pytest.raises(gdn.GdnError):
        gdn.tree_fwd(big["q"], big["k"], big["v"], big["g"], big["beta"],
                     torch.full((B, many), -1, dtype=torch.int32, device="cuda"), x["state"])
