"""The launch forms that only large calls select, against 64 bits on the GPU:
stores of states past the caches (more than 256 MB of states written), trees
checked with a whole state per workgroup (512 states or more) at every node
class, walks of more than 2048 tokens (256 walks or more, or a very long
sequence), the gradients' longest segment.

Tolerances.  Pool calls: those of test_states (2e-5 of the RMS; half a step of
bf16 more where o is bf16): the same sums.  Linear attention, per element,
relative to the tensor's RMS, whose largest element is below 8 times it in these
draws.  An error made in the state at one token decays with the state, so at
any time it holds those of M = 1 / (2 |g|) tokens (in squares): with log
sigmoid of N(9, 1), mean 2.0e-4, M = 2450.  Per 64 tokens a state element is
rounded at most 14 times (two chunks of 32 tokens, six plane products and a
scaling each; bf16 inputs need seven), and a product of 32 terms may round once
more inside: 28, sqrt(28 x 2450 / 64) = 33 independent roundings of 2^-24,
x 8: 1.6e-5.  Reading it with q adds 4 x 6 products, 48 roundings: 3.3e-6.  Of
fp32 inputs the products of three cut planes leave out at most 2^-21 of each
term, with the term's own sign: at most 2^-21 of the element and as much of
the RMS, x 8: 7.6e-6.  Together 2.7e-5; 5e-5 is asked.  bf16 outputs: half a
step, 2^-8 |x|, and 8 x 2^-17 for the two planes of state and scores, 1.2e-4.
The decays' gradient sums a segment's terms, at most 2048: 1e-4, as derived in
test_linear.
"""
import pytest
import torch

from test_linear import DT, D, _close as _close_linear, _reference, gdn  # noqa: F401


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _close(name, got, ref, bf16=False):
    _close_linear(name, got, ref, 2e-5, bf16=bf16)


def _pool(B, n, Hqk, Hv, n_slots, dtype, seed, delta):
    gen = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    lead = (B,) if n is None else (B, n)
    return dict(q=_unit(r(*lead, Hqk, D)).to(DT[dtype]), k=_unit(r(*lead, Hqk, D)).to(DT[dtype]), v=r(*lead, Hv, D).to(DT[dtype]),
                g=torch.nn.functional.logsigmoid(r(*lead, Hv) + 3.0), beta=torch.sigmoid(r(*lead, Hv)) if delta else None,
                state=0.3 * r(n_slots, Hv, D, D))


def _token(S, x, at, Hv):
    """The rule for one token of every row, in 64 bits; S [B, H, d_k, d_v], x's tensors indexed by `at`."""
    wide = lambda t: t[at].double().repeat_interleave(Hv // t.shape[-2], dim=-2)
    q, k, v = wide(x["q"]), wide(x["k"]), x["v"][at].double()
    S = S * x["g"][at].double().exp()[..., None, None]
    u = v if x["beta"] is None else x["beta"][at].double()[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    return S, (S * q[..., None]).sum(-2), u


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,delta", [("bf16", True), ("f32", False)])
def test_step_of_more_states_than_the_caches_hold(gdn, dtype, delta):  # noqa: F811
    B, Hqk, Hv, n_slots = 130, 16, 32, 135                       # 4160 states, 260 MB
    x = _pool(B, None, Hqk, Hv, n_slots, dtype, 81, delta)
    slots = torch.randperm(n_slots, generator=_gen(1), device="cuda")[:B].to(torch.int32)
    slots[[7, 128]] = -1
    on = slots >= 0
    at = slots[on].long()
    S, o_ref, _ = _token(x["state"][at].double(), x, on, Hv)
    before = x["state"].clone()
    o = gdn.step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"], slots=slots, o_dtype=DT[dtype])
    _close("o", o[on], o_ref, dtype == "bf16")
    _close("state", x["state"][at], S)
    assert torch.count_nonzero(o[~on]) == 0
    rest = torch.ones(n_slots, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert int(rest.sum()) == n_slots - B + 2 and torch.equal(x["state"][rest], before[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,delta", [("bf16", True), ("f32", True), ("bf16", False)])
def test_check_and_commit_of_more_states_than_the_caches_hold(gdn, dtype, delta):  # noqa: F811
    B, n, Hqk, Hv, n_slots = 132, 11, 16, 32, 140                # 4224 states
    x = _pool(B, n, Hqk, Hv, n_slots, dtype, 82, delta)
    slots = torch.randperm(n_slots, generator=_gen(2), device="cuda")[:B].to(torch.int32)
    parents = torch.tensor([-1, 0, 1, 1, 3, 4, 4, 6, 7, 8, 0], dtype=torch.int32, device="cuda").repeat(B, 1)
    last = torch.randint(-1, n, (B,), generator=_gen(3), device="cuda").to(torch.int32)
    before = x["state"].clone()
    states, o_ref, u_ref = _check_ref(x, parents, before[slots.long()].double(), Hv)
    o, u = gdn.tree_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], parents, x["state"], slots=slots, o_dtype=DT[dtype])
    assert torch.equal(x["state"], before)
    _close("o", o, o_ref, dtype == "bf16")
    _close("u", u, u_ref)
    gdn.tree_commit(x["k"], u, x["g"], parents, last, x["state"], slots=slots)
    ref = before.double()
    for b in range(B):
        if int(last[b]) >= 0:
            ref[int(slots[b])] = states[int(last[b])][b]
    _close("state", x["state"], ref)
    idle = slots[last < 0].long()
    assert idle.numel() and torch.equal(x["state"][idle], before[idle])


def _check_ref(x, parents, S0, Hv):
    """All rows have one tree: the states of its nodes, o and u in 64 bits."""
    states, o, u = [], [], []
    for r, p in enumerate(parents[0].tolist()):
        S, orow, urow = _token(states[p] if p >= 0 else S0, x, (slice(None), r), Hv)
        states.append(S)
        o.append(orow)
        u.append(urow)
    return states, torch.stack(o, 1), torch.stack(u, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,delta", [("bf16", True), ("f32", True), ("bf16", False), ("f32", False)])
@pytest.mark.parametrize("n", [16, 17, 32, 48, 49, 64])
def test_trees_with_a_whole_state_per_workgroup(gdn, n, dtype, delta):  # noqa: F811
    B, Hqk, Hv, n_slots = 130, 2, 4, 9                           # 520 states checked
    x = _pool(B, n, Hqk, Hv, n_slots, dtype, 83 + n, delta)
    slots = torch.randint(0, n_slots, (B,), generator=_gen(4), device="cuda").to(torch.int32)
    gen = torch.Generator().manual_seed(n)
    tree = [int(torch.randint(-1, r, (), generator=gen)) if r % 3 == 2 else r - 1 for r in range(n)]
    parents = torch.tensor(tree, dtype=torch.int32, device="cuda").repeat(B, 1)
    _, o_ref, u_ref = _check_ref(x, parents, x["state"][slots.long()].double(), Hv)
    o, u = gdn.tree_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], parents, x["state"], slots=slots, o_dtype=DT[dtype])
    _close("o", o, o_ref, dtype == "bf16")
    _close("u", u, u_ref)


# ---------------------------------------------------------------------------
# linear attention


def _draw(T, Hqk, Hv, dtype, seed, strength, grads):
    gen = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = dict(q=_unit(r(1, T, Hqk, D)).to(DT[dtype]), k=_unit(r(1, T, Hqk, D)).to(DT[dtype]), v=r(1, T, Hv, D).to(DT[dtype]),
             g=torch.nn.functional.logsigmoid(r(1, T, Hv) + strength), h0=0.1 * r(1, Hv, D, D))
    if grads:
        x.update(dO=r(1, T, Hv, D).to(DT[dtype]), dh_T=0.1 * r(1, Hv, D, D))
    return x


def _some(x, qk, R):
    """The query/key heads `qk` and the value heads that read them."""
    hv = [h * R + i for h in qk for i in range(R)]
    pick = lambda n, t: t[:, hv] if n in ("h0", "dh_T") else t[:, :, qk] if n in ("q", "k") else t[:, :, hv]
    return {n: pick(n, t).contiguous() for n, t in x.items()}, hv


def _forward_ref(x, C=512):
    """Chunk by chunk in 64 bits: o [1, T, H, D] and the last state."""
    T, Hv = x["v"].shape[1:3]
    R = Hv // x["k"].shape[2]
    S = x["h0"][0].double()
    t = torch.arange(C, device="cuda")
    out = []
    for lo in range(0, T, C):
        q, k = (x[n][0, lo:lo + C].double().transpose(0, 1).repeat_interleave(R, 0) for n in ("q", "k"))
        v, G = x["v"][0, lo:lo + C].double().transpose(0, 1), x["g"][0, lo:lo + C].double().T.cumsum(-1)
        c = t[:G.shape[1]]
        W = (G[:, :, None] - G[:, None]).masked_fill(c[:, None] < c, -torch.inf).exp()
        kt = k.transpose(1, 2).contiguous()
        out.append((((q @ kt) * W) @ v + G.exp()[..., None] * (q @ S)).transpose(0, 1))
        end = G[:, -1:]
        S = end.exp()[..., None] * S + kt @ ((end - G).exp()[..., None] * v)
    return torch.cat(out).unsqueeze(0), S.unsqueeze(0)


def _check_forward(gdn, x, qk, o_dtype):  # noqa: F811
    R = x["v"].shape[2] // x["k"].shape[2]
    o, hT = gdn.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], o_dtype=DT[o_dtype])
    part, hv = _some(x, qk, R)
    o_ref, h_ref = _forward_ref(part)
    _close_linear("o", o[:, :, hv], o_ref, 1.2e-4 if o_dtype == "bf16" else 5e-5, bf16=o_dtype == "bf16")
    _close_linear("h_T", hT[:, hv], h_ref, 5e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,o_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_forward_in_one_walk_of_2100_tokens(gdn, dtype, o_dtype):  # noqa: F811
    # 256 heads: one walk each over the whole sequence
    _check_forward(gdn, _draw(2100, 64, 256, dtype, 91, 9.0, False), [0, 31, 63], o_dtype)


@pytest.mark.gpu
def test_forward_of_262144_tokens(gdn):  # noqa: F811
    # 32 heads: eight segments of 32768 tokens each
    _check_forward(gdn, _draw(262144, 16, 32, "bf16", 92, 9.0, False), [0, 9], "bf16")


@pytest.mark.gpu
def test_packed_forward_of_long_walks(gdn):  # noqa: F811
    # 256 heads: sequences of 2100, 1 and 4000 tokens, one walk each, and rows behind the last
    lens, Hqk, Hv, qk = [2100, 1, 4000], 64, 256, [0, 40]
    cu = [0, 2100, 2101, 6101]
    x = _draw(6110, Hqk, Hv, "f32", 93, 9.0, False)
    h0 = 0.1 * torch.randn(3, Hv, D, D, generator=_gen(5), device="cuda")
    out = torch.full((1, 6110, Hv, D), 7.0, device="cuda")
    o, hT = gdn.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["g"], cu, h0, out=out)
    assert o is out and (o[:, 6101:] == 7).all()
    for i, n in enumerate(lens):
        one = {m: x[m][:, cu[i]:cu[i] + n] for m in ("q", "k", "v", "g")}
        part, hv = _some(dict(one, h0=h0[i:i + 1]), qk, Hv // Hqk)
        o_ref, h_ref = _forward_ref(part)
        _close_linear("o", o[:, cu[i]:cu[i] + n][:, :, hv], o_ref, 5e-5)
        _close_linear("h_T", hT[i:i + 1, hv], h_ref, 5e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,Hqk,Hv,strength,qk", [
    ("bf16", 2100, 64, 256, 9.0, [0, 47]),     # segments of 2048 (the longest) and 52 tokens
    ("f32", 2100, 64, 256, 9.0, [0, 47]),
    ("bf16", 20000, 16, 32, 3.0, [0, 11]),     # ten segments of 2048 at most
    ("bf16", 129, 2, 2, 3.0, [0, 1]),          # a last segment of one token
    ("f32", 65, 2, 2, 3.0, [0, 1]),
])
def test_gradients_of_the_longest_segments(gdn, dtype, T, Hqk, Hv, strength, qk):  # noqa: F811
    x = _draw(T, Hqk, Hv, dtype, 94, strength, True)
    got = gdn.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], h0=x["h0"], dh_T=x["dh_T"])
    part, hv = _some(x, qk, Hv // Hqk)
    _, _, ref = _reference(part, [(0, 0, T)], grads=True)
    for n in ("dq", "dk"):
        _close_linear(n, got[n][:, :, qk], ref[n], 5e-5, bf16=dtype == "bf16")
    _close_linear("dv", got["dv"][:, :, hv], ref["dv"], 5e-5, bf16=dtype == "bf16")
    _close_linear("dg", got["dg"][:, :, hv], ref["dg"], 1e-4)
    _close_linear("dh0", got["dh0"][:, hv], ref["dh0"], 5e-5)
