"""Cases and plain forms of the recurrent-state operators: linear attention
with a decay per head (chunked forward, packed forward, backward), the
single-token step, the check of a tree of drafted tokens and the commit of an
accepted path.

A case names one operator and its sizes; ``prepare`` makes its inputs on the
GPU from a seed, ``run`` makes one pass: the plain form in torch operations,
or, where ``own`` is true, the library's call.  ``exact`` computes the same
outputs in 64 bits from the definition, one token (or one token pair) at a
time.  Heads have 128 key and 128 value columns, states are fp32.
"""
from __future__ import annotations

import random

import torch

own = False

D = 128
CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # a layer's prompt: 4096 tokens, 16 query/key and 32 value heads
        dict(name="fwd_layer_4096", op="fwd", B=1, T=4096, Hqk=16, Hv=32, dtype="bf16", o="bf16", fixed=False, h0=True),
        # the small fp32 configuration, odd length
        dict(name="fwd_small_f32", op="fwd", B=1, T=509, Hqk=2, Hv=2, dtype="f32", o="f32", fixed=False, h0=False),
        # a serving batch of 16 prompts of 1 to 8192 tokens, one decay per head
        dict(name="fwd_packed_mix", op="varlen", n_seq=16, max_len=8192, lens=2000, Hqk=16, Hv=32, dtype="bf16",
             o="bf16", fixed=True, h0=True),
        # a training step of that layer
        dict(name="bwd_layer_4096", op="bwd", B=1, T=4096, Hqk=16, Hv=32, dtype="bf16", fixed=False, h0=True),
        # training in fp32 at an odd length, a decay per head to be learnt
        dict(name="bwd_f32_fixed", op="bwd", B=2, T=1001, Hqk=4, Hv=4, dtype="f32", fixed=True, h0=False),
        # decoding one sequence: latency
        dict(name="step_one", op="step", B=1, slots=8, Hqk=16, Hv=32, dtype="bf16", o="bf16", delta=True, fixed=False),
        # decoding a padded odd batch by the linear rule, fp32
        dict(name="step_linear_f32", op="step", B=37, slots=64, Hqk=16, Hv=32, dtype="f32", o="f32", delta=False, fixed=True),
        # decoding a full batch
        dict(name="step_batch", op="step", B=256, slots=300, Hqk=16, Hv=32, dtype="bf16", o="bf16", delta=True, fixed=False),
        # drafted tokens of a few sequences
        dict(name="tree_few", op="tree", B=4, slots=8, n=13, Hqk=16, Hv=32, dtype="bf16", o="bf16", delta=True),
        # large drafted trees of a batch
        dict(name="tree_batch", op="tree", B=48, slots=64, n=64, Hqk=16, Hv=32, dtype="bf16", o="bf16", delta=True),
        # accepting what those checks let through
        dict(name="commit_few", op="commit", B=4, slots=8, n=13, Hqk=16, Hv=32, dtype="bf16"),
        dict(name="commit_batch", op="commit", B=96, slots=128, n=64, Hqk=16, Hv=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["fwd", "varlen", "bwd", "step", "tree", "commit"])
    group = rng.choice([1, 2, 2, 3, 4])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    o = dtype if rng.random() < 0.75 else "f32"
    if op in ("fwd", "bwd"):
        B = rng.randint(1, 3)
        Hqk = rng.randint(1, 16 // group)
        case = dict(op=op, B=B, T=_log_int(rng, 1, 8192 // B), Hqk=Hqk, Hv=Hqk * group, dtype=dtype,
                    fixed=rng.random() < 0.4, h0=rng.random() < 0.6)
        return dict(case, o=o) if op == "fwd" else case
    if op == "varlen":
        Hqk = rng.randint(1, 16 // group)
        return dict(op=op, n_seq=_log_int(rng, 1, 16), max_len=_log_int(rng, 16, 8192), lens=rng.randrange(1 << 20),
                    Hqk=Hqk, Hv=Hqk * group, dtype=dtype, o=o, fixed=rng.random() < 0.4, h0=rng.random() < 0.6)
    Hqk = rng.randint(1, 32 // group)
    B = _log_int(rng, 1, 256 if op == "step" else 48)
    case = dict(op=op, B=B, slots=B + rng.randint(0, 20), Hqk=Hqk, Hv=Hqk * group, dtype=dtype)
    if op == "step":
        return dict(case, o=o, delta=rng.random() < 0.6, fixed=rng.random() < 0.4)
    case["n"] = _log_int(rng, 1, 64)
    return dict(case, o=o, delta=rng.random() < 0.7) if op == "tree" else case


def _lengths(case):
    r = random.Random(case["lens"])
    return [r.randint(1, case["max_len"]) for _ in range(case["n_seq"])]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    eo = 2 if case.get("o") == "bf16" else 4
    Hqk, Hv, op = case["Hqk"], case["Hv"], case["op"]
    state = Hv * D * D * 4
    if op in ("fwd", "varlen", "bwd"):
        if op == "varlen":
            tokens, rows = sum(_lengths(case)), case["n_seq"]
        else:
            tokens, rows = case["B"] * case["T"], case["B"]
        decay = (0 if case["fixed"] else tokens * Hv) * 4
        states = rows * state
        # per token and value head: half a chunk of scores and of their sums, the read of the state and its write
        flops = tokens * Hv * (2 * D * CHUNK + 4 * D * D)
        if op != "bwd":
            return {"bytes": tokens * D * (e * (2 * Hqk + Hv) + eo * Hv) + decay + states * (2 if case["h0"] else 1),
                    "flops": flops}
        return {"bytes": tokens * D * e * (4 * Hqk + 3 * Hv) + 2 * decay + states * (3 if case["h0"] else 2),
                "flops": tokens * Hv * (5 * D * CHUNK + 10 * D * D)}
    B = case["B"]
    if op == "step":
        return {"bytes": B * (2 * state + D * (e * (2 * Hqk + Hv) + eo * Hv)), "flops": B * Hv * 6 * D * D}
    n = case["n"]
    if op == "tree":
        return {"bytes": B * (state + n * (D * (e * (2 * Hqk + Hv) + (eo + 4) * Hv) + 8 * Hv)),
                "flops": B * Hv * (4 * n * D * D + 4 * n * n * D)}
    # of n drafted tokens about half a path is accepted; the state dominates
    return {"bytes": B * (2 * state + min(n, 8) * D * (e * Hqk + 4 * Hv)), "flops": B * Hv * 2 * D * D * min(n, 8)}


# ---------------------------------------------------------------------------
# inputs


def _unit(gen, shape, dtype, dev):
    x = torch.randn(shape, generator=gen, device=dev)
    return (x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)).to(dtype)


def _decays(gen, case, shape, dev):
    """Log decays: log sigmoid of N(3, 1), per token, or one for each head."""
    size = (case["Hv"],) if case.get("fixed") else shape
    return torch.nn.functional.logsigmoid(torch.randn(size, generator=gen, device=dev) + 3.0)


def _parents(gen, B, n, dev):
    """Drafted trees: half of the nodes continue the one before, the others branch off any earlier node or the state (-1);
    a row has n/2 to n nodes, the places behind them are absent (-2)."""
    r = torch.arange(n, device=dev)
    anyone = (torch.rand((B, n), generator=gen, device=dev) * (r + 1)).long().clamp(max=n) - 1
    parent = torch.where(torch.rand((B, n), generator=gen, device=dev) < 0.5, r - 1, torch.minimum(anyone, r - 1))
    live = (n + 1) // 2 + (torch.rand((B, 1), generator=gen, device=dev) * (n - (n + 1) // 2 + 1)).long()
    return torch.where(r < live, parent, -2).to(torch.int32)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt, op, Hqk, Hv = DTYPES[case["dtype"]], case["op"], case["Hqk"], case["Hv"]
    s = dict(case=dict(case))
    if op in ("fwd", "varlen", "bwd"):
        if op == "varlen":
            lens = _lengths(case)
            B, T, rows = 1, sum(lens), case["n_seq"]
            offsets = [0]
            for n in lens:
                offsets.append(offsets[-1] + n)
            s["cu"] = torch.tensor(offsets, dtype=torch.int32, device=dev)
        else:
            B, T, rows = case["B"], case["T"], case["B"]
        s["q"], s["k"] = _unit(gen, (B, T, Hqk, D), dt, dev), _unit(gen, (B, T, Hqk, D), dt, dev)
        s["v"] = torch.randn((B, T, Hv, D), generator=gen, device=dev).to(dt)
        s["g"] = _decays(gen, case, (B, T, Hv), dev)
        s["h0"] = torch.randn((rows, Hv, D, D), generator=gen, device=dev) * 0.02 if case["h0"] else None
        if op == "bwd":
            s["dO"] = torch.randn((B, T, Hv, D), generator=gen, device=dev).to(dt)
            s["dh_T"] = torch.randn((B, Hv, D, D), generator=gen, device=dev) * 0.1
        return s
    B, slots = case["B"], case["slots"]
    at = torch.argsort(torch.rand(slots, generator=gen, device=dev))[:B].to(torch.int32)
    if B > 8:
        at[-(B // 12 + 1):] = -1   # a batch padded at its end
    s["slots"] = at
    s["state"] = torch.randn((slots, Hv, D, D), generator=gen, device=dev) * 0.1
    lead = (B,) if op == "step" else (B, case["n"])
    s["k"] = _unit(gen, lead + (Hqk, D), dt, dev)
    s["g"] = _decays(gen, case, lead + (Hv,), dev)
    if op != "step":
        s["parents"] = _parents(gen, B, case["n"], dev)
    if op == "commit":
        s["u"] = torch.randn(lead + (Hv, D), generator=gen, device=dev)
        # the accepted node: any of the row's first half, or none
        s["last"] = ((torch.rand(B, generator=gen, device=dev) * ((case["n"] + 1) // 2 + 1)).long() - 1).to(torch.int32)
        return s
    s["q"] = _unit(gen, lead + (Hqk, D), dt, dev)
    s["v"] = torch.randn(lead + (Hv, D), generator=gen, device=dev).to(dt)
    s["beta"] = torch.sigmoid(torch.randn(lead + (Hv,), generator=gen, device=dev)) if case["delta"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms


def _heads(x, Hv, N):
    """[B, T, H, d] -> [B, H_v, N, C, d] in fp32, the last chunk padded with zeros, every value head with its key head."""
    x = x.float()
    B, T, H, d = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, N * CHUNK - T)).view(B, N, CHUNK, H, d).permute(0, 3, 1, 2, 4)
    return x if H == Hv else x.unsqueeze(2).expand(B, H, Hv // H, N, CHUNK, d).reshape(B, Hv, N, CHUNK, d)


def _tokens(x, T):
    """[B, H, N, C, d] -> [B, T, H, d]"""
    B, H, N, C, d = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(B, N * C, H, d)[:, :T]


def _token_decays(g, like):
    B, T, Hv = like.shape[:3]
    return g.expand(B, T, Hv) if g.dim() == 1 else g


def _chunk_decays(g, N):
    """Per chunk: the decay from token i to token r (zero for i > r), from the chunk's start to r and from i to its end;
    and, between chunks, from the end of chunk m to the start of chunk n and from the sequence's start to chunk n's (n up to
    N: the end)."""
    B, T, H = g.shape
    G = torch.nn.functional.pad(g.double(), (0, 0, 0, N * CHUNK - T)).view(B, N, CHUNK, H).permute(0, 3, 1, 2).cumsum(-1)
    r = torch.arange(CHUNK, device=g.device)
    within = (G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(r[:, None] < r, -torch.inf).exp().float()
    ends = G[..., -1].cumsum(-1)                                     # [B, H, N]: decay up to each chunk's end
    starts = torch.nn.functional.pad(ends, (1, 0))                   # [B, H, N + 1]: up to each chunk's start
    n, m = torch.arange(N + 1, device=g.device), torch.arange(N, device=g.device)
    between = (starts.unsqueeze(-1) - ends.unsqueeze(-2)).masked_fill(n[:, None] <= m, -torch.inf).exp().float()
    return within, G.exp().float().unsqueeze(-1), (G[..., -1:] - G).exp().float().unsqueeze(-1), between, starts.exp().float()


def _states_in(k, v, to_end, between, from_start, h0):
    """State at each chunk's start, and after the last: [B, H, N + 1, d_k, d_v]."""
    added = (k * to_end).transpose(-1, -2).contiguous() @ v
    B, H, N = added.shape[:3]
    h = (between @ added.view(B, H, N, D * D)).view(B, H, N + 1, D, D)
    return h if h0 is None else h + from_start[..., None, None] * h0.unsqueeze(2)


def _linear_fwd(q, k, v, g, h0, o_dtype):
    B, T, Hv = v.shape[:3]
    N = -(-T // CHUNK)
    q, k, v = _heads(q, Hv, N), _heads(k, Hv, N), _heads(v, Hv, N)
    within, from_start, to_end, between, chunk_start = _chunk_decays(g, N)
    h = _states_in(k, v, to_end, between, chunk_start, h0)
    o = ((q @ k.transpose(-1, -2).contiguous()) * within) @ v + (q * from_start) @ h[:, :, :-1]
    return _tokens(o, T).to(o_dtype).contiguous(), h[:, :, -1].contiguous()


def _linear_fwd_packed(q, k, v, g, cu, lens_max, h0, o_dtype):
    cu = cu.long()
    n = cu.numel() - 1
    t = torch.arange(lens_max, device=q.device)
    at = cu[:-1, None] + t
    here = at < cu[1:, None]
    at = at.clamp(max=q.shape[1] - 1)

    def padded(x):
        return torch.where(here.view(n, lens_max, *[1] * (x.dim() - 2)), x[0][at], torch.zeros((), dtype=x.dtype, device=x.device))

    o, h = _linear_fwd(padded(q), padded(k), padded(v), padded(g), h0, o_dtype)
    return o[here].unsqueeze(0), h


def _linear_bwd(q, k, v, g, h0, dO, dh_T, fixed):
    B, T, Hqk = q.shape[:3]
    Hv = v.shape[2]
    dt = q.dtype
    N = -(-T // CHUNK)
    q, k, v, dO = _heads(q, Hv, N), _heads(k, Hv, N), _heads(v, Hv, N), _heads(dO, Hv, N)
    within, from_start, to_end, between, chunk_start = _chunk_decays(g, N)
    h = _states_in(k, v, to_end, between, chunk_start, h0)
    # cotangents of the state after each chunk, from the last chunk backwards
    taken = (q * from_start).transpose(-1, -2).contiguous() @ dO      # into the state at each chunk's start
    B_, H_ = taken.shape[:2]
    # the state after chunk m reaches the start of chunk n > m: between[n, m]; the sequence's end: between[N, m]
    reach = between[..., :-1, :].transpose(-1, -2).contiguous()
    dh = (reach @ taken.view(B_, H_, N, D * D)).view(B_, H_, N, D, D)
    dh = dh + between[..., -1, :][..., None, None] * dh_T.unsqueeze(2)
    dh0 = (chunk_start[..., None, :-1] @ taken.view(B_, H_, N, D * D)).view(B_, H_, D, D) + chunk_start[..., -1, None, None] * dh_T
    P = (q @ k.transpose(-1, -2).contiguous()) * within
    dP = (dO @ v.transpose(-1, -2).contiguous()) * within
    dq = dP @ k + from_start * (dO @ h[:, :, :-1].transpose(-1, -2).contiguous())
    dk = dP.transpose(-1, -2).contiguous() @ q + to_end * (v @ dh.transpose(-1, -2).contiguous())
    dv = P.transpose(-1, -2).contiguous() @ dO + to_end * (k @ dh)
    # g_t scales every pair that crosses it: those inside the chunk that end at t or later less those that begin there,
    # and what leaves the chunk in its state
    leaves = (h[:, :, 1:].double() * dh.double()).sum((-1, -2))
    dG = (q.double() * dq.double()).sum(-1) - (k.double() * dk.double()).sum(-1)
    dg = torch.flip(torch.flip(dG, (-1,)).cumsum(-1), (-1,)) + leaves.unsqueeze(-1)
    dg = _tokens(dg.unsqueeze(-1), T).squeeze(-1)
    dg = dg.sum((0, 1)) if fixed else dg

    def shared(x):
        return _tokens(x, T).reshape(B, T, Hqk, Hv // Hqk, D).sum(3).to(dt)

    return dict(dq=shared(dq), dk=shared(dk), dv=_tokens(dv, T).to(dt).contiguous(), dg=dg.float().contiguous(), dh0=dh0)


def _shared_heads(x, Hv):
    """[.., H_qk, d] -> [.., H_v, d] in fp32"""
    return x.float().repeat_interleave(Hv // x.shape[-2], dim=-2)


def _step(q, k, v, g, beta, state, slots, o_dtype):
    Hv = v.shape[1]
    here = (slots >= 0) & (slots < state.shape[0])
    rows = torch.where(here, slots, 0).long()
    q, k, v = _shared_heads(q, Hv), _shared_heads(k, Hv), v.float()
    S = state[rows] * g.exp().expand(v.shape[:2])[..., None, None]
    u = v if beta is None else beta.unsqueeze(-1) * (v - (S * k.unsqueeze(-1)).sum(-2))
    S = S + k.unsqueeze(-1) * u.unsqueeze(-2)
    o = (S * q.unsqueeze(-1)).sum(-2).masked_fill(~here[:, None, None], 0.0)
    state[rows[here]] = S[here]
    return o.to(o_dtype), state


def _closure(M):
    """I + M + M^2 + ... of strictly lower triangular matrices of up to 64 rows."""
    X = torch.eye(M.shape[-1], dtype=M.dtype, device=M.device) + M
    M2 = M @ M
    X = X + X @ M2
    M4 = M2 @ M2
    X = X + X @ M4
    M8 = M4 @ M4
    X = X + X @ M8
    M16 = M8 @ M8
    X = X + X @ M16
    return X + X @ (M16 @ M16)


def _tree(parents):
    """[B, n] parents -> ancestor-or-self relation [B, n, n] and which nodes hang on the state."""
    B, n = parents.shape
    r = torch.arange(n, device=parents.device)
    valid = (parents >= -1) & (parents < r)
    step = ((parents.unsqueeze(-1) == r) & valid.unsqueeze(-1)).double()
    above = _closure(step)
    live = (above @ (~valid).double().unsqueeze(-1)).squeeze(-1) == 0
    return above, live


def _tree_fwd(q, k, v, g, beta, parents, state, slots, o_dtype):
    Hv = v.shape[2]
    above, live = _tree(parents)
    here = (slots >= 0) & (slots < state.shape[0])
    S0 = state[torch.where(here, slots, 0).long()]
    live = live & here[:, None]
    q, k, v = (_shared_heads(x, Hv).transpose(1, 2).contiguous() for x in (q, k, v))     # [B, H, n, d]
    G = (above @ g.double()).transpose(1, 2)                                             # along each node's path
    pair = (G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(above.unsqueeze(1) == 0, -torch.inf).exp()
    kt = k.transpose(-1, -2).contiguous()
    if beta is None:
        u = v
    else:
        b = beta.transpose(1, 2).unsqueeze(-1)
        S = (b * (k @ kt) * pair).tril(-1)
        u = (_closure(-S) @ (b * (v - G.exp().unsqueeze(-1) * (k @ S0))).double()).float()
    o = G.exp().unsqueeze(-1) * (q @ S0) + (((q @ kt) * pair).float() @ u)
    keep = live[:, None, :, None]
    o, u = (torch.where(keep, x, 0.0).transpose(1, 2) for x in (o, u))
    return o.to(o_dtype).contiguous(), u.float().contiguous()


def _commit(k, u, g, parents, last, state, slots):
    Hv = u.shape[2]
    above, live = _tree(parents)
    B, n = parents.shape
    at = last.clamp(0, n - 1).long()
    row = torch.arange(B, device=at.device)
    done = (slots >= 0) & (slots < state.shape[0]) & (last >= 0) & (last < n) & live[row, at]
    rows = torch.where(done, slots, 0).long()
    path = above[row, at]                                                                # [B, n]
    G = above @ g.double()
    w = ((G[row, at].unsqueeze(1) - G).masked_fill(path.unsqueeze(-1) == 0, -torch.inf).exp()).float()   # [B, n, H]
    kw = (_shared_heads(k, Hv) * w.unsqueeze(-1)).permute(0, 2, 3, 1).contiguous()       # [B, H, d_k, n]
    S = G[row, at].exp().float()[..., None, None] * state[rows] + kw @ u.transpose(1, 2).contiguous()
    state[rows[done]] = S[done]
    return state


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import linear_attention_rnn_gdn_amd as gdn

        if op == "fwd":
            return gdn.linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], o_dtype=DTYPES[c["o"]])
        if op == "varlen":
            return gdn.linear_chunk_fwd_varlen(s["q"], s["k"], s["v"], s["g"], s["cu"], h0=s["h0"], o_dtype=DTYPES[c["o"]])
        if op == "bwd":
            return gdn.linear_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["dO"], h0=s["h0"], dh_T=s["dh_T"])
        if op == "step":
            o = gdn.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], o_dtype=DTYPES[c["o"]])
            return o, s["state"]
        if op == "tree":
            return gdn.tree_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["parents"], s["state"], slots=s["slots"],
                                o_dtype=DTYPES[c["o"]])
        gdn.tree_commit(s["k"], s["u"], s["g"], s["parents"], s["last"], s["state"], slots=s["slots"])
        return s["state"]
    if op == "fwd":
        return _linear_fwd(s["q"], s["k"], s["v"], _token_decays(s["g"], s["v"]), s["h0"], DTYPES[c["o"]])
    if op == "varlen":
        return _linear_fwd_packed(s["q"], s["k"], s["v"], _token_decays(s["g"], s["v"]), s["cu"], max(_lengths(c)), s["h0"],
                                  DTYPES[c["o"]])
    if op == "bwd":
        return _linear_bwd(s["q"], s["k"], s["v"], _token_decays(s["g"], s["v"]), s["h0"], s["dO"], s["dh_T"], c["fixed"])
    if op == "step":
        return _step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slots"], DTYPES[c["o"]])
    if op == "tree":
        return _tree_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["parents"], s["state"], s["slots"], DTYPES[c["o"]])
    return _commit(s["k"], s["u"], s["g"], s["parents"], s["last"], s["state"], s["slots"])


# ---------------------------------------------------------------------------
# 64-bit values from the definitions


def _exact_pairs(q, k, v, g, h0):
    """One sequence of one head, every pair of tokens: o, the state behind the last token, and the decays."""
    T = q.shape[0]
    G = g.cumsum(0)
    t = torch.arange(T, device=q.device)
    W = torch.where(t[:, None] >= t, torch.exp(torch.minimum(G[:, None] - G, torch.zeros((), dtype=G.dtype, device=G.device))), 0.0)
    o = ((q @ k.T) * W) @ v
    h = k.T @ (torch.exp(G[-1] - G)[:, None] * v)
    if h0 is not None:
        o = o + torch.exp(G)[:, None] * (q @ h0)
        h = h + torch.exp(G[-1]) * h0
    return o, h, G, W


def _exact_chunked(s, c):
    q, k, v = (s[x].double() for x in "qkv")
    g = s["g"].double()
    B, T, Hv = v.shape[:3]
    rep = Hv // c["Hqk"]
    g = g.expand(B, T, Hv) if g.dim() == 1 else g
    h0 = None if s["h0"] is None else s["h0"].double()
    if c["op"] == "varlen":
        cu = s["cu"].tolist()
        spans = [(0, cu[i], cu[i + 1], i) for i in range(c["n_seq"])]
    else:
        spans = [(b, 0, T, b) for b in range(B)]
    o = torch.zeros((B, T, Hv, D), dtype=torch.float64, device=q.device)
    hT = torch.zeros((len(spans), Hv, D, D), dtype=torch.float64, device=q.device)
    grads = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v), dg=torch.zeros_like(v[..., 0]),
                 dh0=torch.zeros_like(hT))
    for b, lo, hi, i in spans:
        for h in range(Hv):
            qh, kh, vh, gh = q[b, lo:hi, h // rep], k[b, lo:hi, h // rep], v[b, lo:hi, h], g[b, lo:hi, h]
            oh, sh, G, W = _exact_pairs(qh, kh, vh, gh, None if h0 is None else h0[i, h])
            o[b, lo:hi, h], hT[i, h] = oh, sh
            if c["op"] != "bwd":
                continue
            dO, dS = s["dO"][b, lo:hi, h].double(), s["dh_T"][b, h].double()
            scores, dscores = (qh @ kh.T) * W, (dO @ vh.T) * W
            tail = torch.exp(G[-1] - G)[:, None]
            dqh, dkh = dscores @ kh, dscores.T @ qh + tail * (vh @ dS.T)
            grads["dv"][b, lo:hi, h] = scores.T @ dO + tail * (kh @ dS)
            grads["dh0"][b, h] = qh.T @ (torch.exp(G)[:, None] * dO) + torch.exp(G[-1]) * dS
            # what crosses a token: pairs with it between them, later ones from h0, earlier ones into h_T
            pairs = (qh @ kh.T) * dscores
            crossing = pairs.sum(1) - pairs.sum(0)
            crossing = crossing - (tail[:, 0] * ((kh @ dS) * vh).sum(1))
            if h0 is not None:
                from_h0 = torch.exp(G)[:, None] * (dO @ h0[i, h].T)
                dqh = dqh + from_h0
                crossing = crossing + (from_h0 * qh).sum(1)
            grads["dg"][b, lo:hi, h] = crossing.flip(0).cumsum(0).flip(0) + (sh * dS).sum()
            grads["dq"][b, lo:hi, h // rep] += dqh
            grads["dk"][b, lo:hi, h // rep] += dkh
    if c["op"] == "bwd":
        if c["fixed"]:
            grads["dg"] = grads["dg"].sum((0, 1))
        return grads
    return o, hT


def _advance(S, k, v, g, beta):
    """One token's rule on states [.., d_k, d_v]."""
    S = torch.exp(g)[..., None, None] * S
    u = v if beta is None else beta[..., None] * (v - torch.einsum("...kv,...k->...v", S, k))
    return S + k[..., :, None] * u[..., None, :], u


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op in ("fwd", "varlen", "bwd"):
        return _exact_chunked(s, c)
    Hv, rep = c["Hv"], c["Hv"] // c["Hqk"]
    heads = torch.arange(Hv, device=s["k"].device) // rep
    state = s["state"].double()
    slots = s["slots"].tolist()
    g = s["g"].double()
    if op == "step":
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device=state.device)
        for b, slot in enumerate(slots):
            if not 0 <= slot < c["slots"]:
                continue
            S, _ = _advance(state[slot], s["k"][b, heads].double(), s["v"][b].double(), g if g.dim() == 1 else g[b],
                            None if s["beta"] is None else s["beta"][b].double())
            state[slot] = S
            o[b] = torch.einsum("hkv,hk->hv", S, s["q"][b, heads].double())
        return o, state
    parents = s["parents"].tolist()
    if op == "tree":
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device=state.device)
        u = torch.zeros_like(o)
        for b, slot in enumerate(slots):
            if not 0 <= slot < c["slots"]:
                continue
            at = {-1: state[slot]}
            for r, p in enumerate(parents[b]):
                if p >= r or p not in at:
                    continue
                at[r], u[b, r] = _advance(at[p], s["k"][b, r, heads].double(), s["v"][b, r].double(), g[b, r],
                                          None if s["beta"] is None else s["beta"][b, r].double())
                o[b, r] = torch.einsum("hkv,hk->hv", at[r], s["q"][b, r, heads].double())
        return o, u
    for b, slot in enumerate(slots):
        last, path = int(s["last"][b]), []
        while 0 <= last < c["n"]:
            path.append(last)
            nxt = parents[b][last]
            if nxt >= last:
                nxt = -2
            last = nxt
        if not path or last != -1 or not 0 <= slot < c["slots"]:
            continue
        for r in reversed(path):
            state[slot] = torch.exp(g[b, r])[:, None, None] * state[slot] + s["k"][b, r, heads].double()[:, :, None] * s["u"][b, r].double()[:, None, :]
    return state
