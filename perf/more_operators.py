"""Cases and plain forms of the operators around a recurrent layer: the short
causal convolution, the selective state space scan (prompts, packed prompts,
gradients, single tokens of both) and the verification of drafted tokens.

A case names one operator and its sizes; ``prepare`` makes its inputs on the
GPU from a seed, ``run`` makes one pass: the plain form in torch operations,
or, where ``own`` is true, the library's call.  ``exact`` computes the same
outputs in 64 bits from the definitions, one token at a time.
"""
from __future__ import annotations

import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 64   # tokens per block of the plain scan


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # q, k and v of a layer's prompt: 4096 tokens, 16 + 16 query/key and 32 value heads of 128
        dict(name="conv_layer_4096", op="conv_fwd", B=1, T=4096, C=8192, W=4, dtype="bf16", silu=True, bias=False, h0=False),
        # a serving batch of prompts that go on from their windows, fp32, an odd width and no activation
        dict(name="conv_packed_f32", op="conv_varlen", n_seq=13, max_len=1500, lens=2001, C=1001, W=3, dtype="f32", silu=False,
             bias=True, h0=True),
        # a training step of that layer
        dict(name="conv_bwd_layer", op="conv_bwd", B=1, T=4096, C=8192, W=4, dtype="bf16", silu=True, bias=True, h0=False),
        # decoding a padded batch
        dict(name="conv_step_batch", op="conv_step", B=256, slots=300, C=8192, W=4, dtype="bf16", silu=True, bias=False),
        # a layer's prompt: 4096 tokens and channels, 16 states each
        dict(name="ssm_layer_4096", op="ssm_fwd", B=1, T=4096, C=4096, N=16, G=1, dtype="bf16", o="bf16", full=True, h0=False),
        # a serving batch of prompts of 1 to 2048 tokens, each from its own state
        dict(name="ssm_packed_mix", op="ssm_varlen", n_seq=12, max_len=2048, lens=2002, C=2000, N=16, G=1, dtype="bf16",
             o="bf16", full=True, h0=True),
        # a training step of the 4096-token layer
        dict(name="ssm_bwd_layer", op="ssm_bwd", B=1, T=4096, C=4096, N=16, G=1, dtype="bf16", full=True, h0=False),
        # training a small fp32 layer at an odd length, two groups, no gate
        dict(name="ssm_bwd_small_f32", op="ssm_bwd", B=2, T=509, C=200, N=8, G=2, dtype="f32", full=False, h0=True),
        # decoding one sequence: latency
        dict(name="ssm_step_one", op="ssm_step", B=1, slots=8, C=4096, N=16, G=1, dtype="bf16", o="bf16", full=True),
        # decoding a full, padded batch
        dict(name="ssm_step_batch", op="ssm_step", B=256, slots=300, C=4096, N=16, G=1, dtype="bf16", o="bf16", full=True),
        # five sampled draft tokens of one sequence: latency
        dict(name="verify_one_chain", op="verify", B=1, n=5, V=32003, tree=False, draft=True),
        # a batch's trees of likely tokens, a large vocabulary
        dict(name="verify_batch_tree", op="verify", B=32, n=16, V=131072, tree=True, draft=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_varlen", "conv_bwd", "conv_step", "ssm_fwd", "ssm_fwd", "ssm_varlen", "ssm_bwd", "ssm_bwd",
                     "ssm_step", "verify", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "verify":
        n = _log_int(rng, 1, 64)
        V = _log_int(rng, 100, 131072)
        B = _log_int(rng, 1, max(1, min(64, (32 * 16 * 131072) // (n * V))))
        return dict(op=op, B=B, n=n, V=V, tree=rng.random() < 0.6, draft=rng.random() < 0.6)
    if op.startswith("conv"):
        case = dict(op=op, C=_log_int(rng, 16, 8192) if rng.random() < 0.4 else 64 * _log_int(rng, 1, 128), W=rng.choice([2, 3, 4, 4]),
                    dtype=dtype, silu=rng.random() < 0.7, bias=rng.random() < 0.5)
        if op == "conv_step":
            B = _log_int(rng, 1, 256)
            return dict(case, B=B, slots=B + rng.randint(0, 40))
        most = 4096 * 8192 // case["C"]
        if op == "conv_varlen":
            n_seq = _log_int(rng, 1, min(32, most))
            return dict(case, n_seq=n_seq, max_len=_log_int(rng, 1, max(1, min(8192, most // n_seq))), lens=rng.randrange(1 << 20),
                        h0=rng.random() < 0.6)
        B = rng.randint(1, 3)
        return dict(case, B=B, T=_log_int(rng, 1, min(16384, most) // B), h0=rng.random() < 0.4)
    G = rng.choice([1, 1, 1, 2, 4])
    case = dict(op=op, C=G * _log_int(rng, 8, 4096 // G), N=rng.choice([8, 16, 16, 16, 32]), G=G, dtype=dtype, full=rng.random() < 0.7)
    o = dtype if rng.random() < 0.75 else "f32"
    if op == "ssm_step":
        B = _log_int(rng, 1, 256 * 16 // case["N"] // 2)
        return dict(case, B=B, slots=B + rng.randint(0, 40), o=o)
    most = 4096 * 4096 * 16 // (case["C"] * case["N"])
    if op == "ssm_varlen":
        n_seq = _log_int(rng, 1, 24)
        return dict(case, n_seq=n_seq, max_len=_log_int(rng, 1, min(8192, most // n_seq)), lens=rng.randrange(1 << 20), o=o,
                    h0=rng.random() < 0.6)
    B = rng.randint(1, 4)
    case = dict(case, B=B, T=_log_int(rng, 1, min(8192, most) // B), h0=rng.random() < 0.4)
    return dict(case, o=o) if op == "ssm_fwd" else case


def _lengths(case):
    """Tokens of each sequence; of several, one in six is empty."""
    if "n_seq" not in case:
        return [case["T"]] * case["B"]
    r = random.Random(case["lens"])
    lens = [0 if r.random() < 1 / 6 else r.randint(1, case["max_len"]) for _ in range(case["n_seq"])]
    if not any(lens):
        lens[0] = 1
    return lens


def work(case):
    op = case["op"]
    if op == "verify":
        return {"bytes": case["B"] * 4 * (case["V"] * (2 if case["draft"] else 1) + 8 * case["n"]),
                "flops": case["B"] * case["V"] * (5 if case["draft"] else 2)}
    e, C = 2 if case["dtype"] == "bf16" else 4, case["C"]
    rows = case["B"] if op.endswith("step") else sum(_lengths(case))
    if op.startswith("conv"):
        W = case["W"]
        params = C * 4 * (W + case["bias"])
        if op == "conv_step":
            return {"bytes": rows * C * e * (2 + 2 * (W - 1)) + params, "flops": rows * C * (2 * W + 8)}
        if op == "conv_bwd":
            return {"bytes": rows * C * e * 3 + 2 * params, "flops": rows * C * (6 * W + 16)}
        return {"bytes": rows * C * e * 2 + params, "flops": rows * C * (2 * W + 8)}
    N, G = case["N"], case["G"]
    eo = 2 if case.get("o") == "bf16" else 4
    z = 1 if case["full"] else 0
    params = C * 4 * (N + 2)
    if op == "ssm_step":
        return {"bytes": rows * (2 * C * N * 4 + C * (e * (2 + z) + eo) + 2 * G * N * e) + params, "flops": rows * C * (7 * N + 20)}
    states = len(_lengths(case)) * C * N * 4
    if op == "ssm_bwd":
        return {"bytes": rows * (C * e * (5 + 2 * z) + 4 * G * N * e) + 2 * params + (2 if case["h0"] else 1) * states,
                "flops": rows * C * (24 * N + 40)}
    return {"bytes": rows * (C * (e * (2 + z) + eo) + 2 * G * N * e) + params + (2 if case["h0"] else 1) * states,
            "flops": rows * C * (7 * N + 20)}


# ---------------------------------------------------------------------------
# inputs


def _offsets(case):
    cu = [0]
    for n in _lengths(case):
        cu.append(cu[-1] + n)
    return cu


def _slots(gen, case, dev):
    B = case["B"]
    at = torch.argsort(torch.rand(case["slots"], generator=gen, device=dev))[:B].to(torch.int32)
    if B > 8:
        at[-(B // 12 + 1):] = -1   # a batch padded at its end
    return at


def _parents(gen, B, n, dev):
    """Drafted trees: half of the nodes continue the one before, the others branch off any earlier node or the root (-1); a row
    has n/2 to n nodes, the places behind them are absent (-2)."""
    r = torch.arange(n, device=dev)
    anyone = (torch.rand((B, n), generator=gen, device=dev) * (r + 1)).long().clamp(max=n) - 1
    parent = torch.where(torch.rand((B, n), generator=gen, device=dev) < 0.5, r - 1, torch.minimum(anyone, r - 1))
    live = (n + 1) // 2 + (torch.rand((B, 1), generator=gen, device=dev) * (n - (n + 1) // 2 + 1)).long()
    return torch.where(r < live, parent, -2).to(torch.int32)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = dict(case=dict(case))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    if op == "verify":
        B, n, V = case["B"], case["n"], case["V"]
        r = torch.arange(n, device=dev, dtype=torch.int32)
        s["parents"] = _parents(gen, B, n, dev) if case["tree"] else (r - 1).expand(B, n).contiguous()
        logits = 3.0 * normal(B, n + 1, V)
        guess = 0.9 * logits[:, :n] + 0.8 * normal(B, n, V)
        s["target"] = torch.softmax(logits, -1)
        s["draft"] = torch.softmax(guess, -1) if case["draft"] else None
        # node r's token is drawn from the draft's probabilities behind its parent; without them it is one of the likeliest there
        tokens = torch.empty((B, n), dtype=torch.int32, device=dev)
        for i in range(n):
            at = (s["parents"][:, i].long() + 1).clamp(min=0)
            noise = -torch.log(-torch.log(uniform(B, V).clamp(1e-20, 1 - 1e-7)))
            tokens[:, i] = (guess[torch.arange(B, device=dev), at] + (1.0 if case["draft"] else 0.2) * noise).argmax(-1).to(torch.int32)
        s["tokens"] = tokens
        s["uniform"] = uniform(B, n + 1)
        return s
    dt, C = DTYPES[case["dtype"]], case["C"]
    if op.endswith("step"):
        lead, n = (case["B"],), case["B"]
        s["slots"] = _slots(gen, case, dev)
    elif "n_seq" in case:
        cu = _offsets(case)
        lead, n = (1, cu[-1]), case["n_seq"]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    else:
        lead, n = (case["B"], case["T"]), case["B"]
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = normal(*lead, C).to(dt)
        s["weight"] = (uniform(C, W) * 2 - 1) * W ** -0.5
        s["bias"] = 0.1 * normal(C) if case["bias"] else None
        if op == "conv_step":
            s["state"] = normal(case["slots"], W - 1, C).to(dt)
        else:
            s["h0"] = normal(n, W - 1, C).to(dt) if case["h0"] else None
        if op == "conv_bwd":
            s["dy"] = normal(*lead, C).to(dt)
            s["dh_T"] = 0.1 * normal(n, W - 1, C).to(dt) if case["h0"] else None
        return s
    N, G = case["N"], case["G"]
    # x and its gate are the halves of one projection, B and C of another, as a layer's weights give them
    xz = normal(*lead, 2 * C).to(dt)
    s["x"], s["z"] = xz[..., :C], xz[..., C:] if case["full"] else None
    s["dt"] = (0.5 * normal(*lead, C)).to(dt)
    bc = normal(*lead, 2 * G * N).to(dt)
    s["Bm"], s["Cm"] = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
    # decay rates 1 .. N; steps of 0.001 to 0.1 at dt = 0, by the inverse of softplus
    s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32).expand(C, N) * (0.75 + 0.5 * uniform(C, N))
    step = 0.001 * 100.0 ** uniform(C)
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = 1 + 0.1 * normal(C) if case["full"] else None
    if op == "ssm_step":
        s["state"] = 0.1 * normal(case["slots"], C, N)
    else:
        s["h0"] = 0.1 * normal(n, C, N) if case["h0"] else None
    if op == "ssm_bwd":
        s["dy"] = normal(*lead, C).to(dt)
        s["dh_T"] = 0.1 * normal(n, C, N) if case["h0"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms


def _rows(x):
    """[B, T, ...] -> [B T, ...]"""
    return x.reshape(-1, *x.shape[2:])


def _sequences(cu, M):
    """Of each of M packed tokens: its sequence, and its place there."""
    t = torch.arange(M, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, t - cu[seq]


def _cu(s, B, T):
    return s["cu"].long() if "cu" in s else torch.arange(B + 1, device=s["x"].device) * T


def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


def _conv_taps(x, h0, seq, pos, W):
    """x at tap w of every token [M, C], and the row of the window that tap reads where it lies before the sequence."""
    taps = []
    for w in range(W):
        back = W - 1 - w
        inside = pos >= back
        X = torch.roll(x, back, 0) if back else x
        X = torch.where(inside.unsqueeze(-1), X, 0.0)
        row = (W - 1 - back + pos).clamp(0, max(W - 2, 0))
        if h0 is not None and back:
            out = torch.nonzero(~inside).squeeze(-1)
            X = X.index_copy(0, out, h0[seq[out], row[out]])
        taps.append((X, inside, row, back))
    return taps


def _conv_plain(s):
    c = s["case"]
    W, x = c["W"], s["x"]
    B, T, C = x.shape
    cu = _cu(s, B, T)
    n = cu.numel() - 1
    X = _rows(x).float()
    h0 = None if s["h0"] is None else s["h0"].float()
    seq, pos = _sequences(cu, B * T)
    taps = _conv_taps(X, h0, seq, pos, W)
    weight = s["weight"]
    pre = sum(tap[0] * weight[:, w] for w, tap in enumerate(taps))
    if s["bias"] is not None:
        pre = pre + s["bias"]
    if c["op"] != "conv_bwd":
        y = _silu(pre) if c["silu"] else pre
        at = cu[1:, None] - (W - 1) + torch.arange(W - 1, device=x.device)     # the last W - 1 tokens of each sequence
        before = at - cu[:-1, None]
        hT = X[at.clamp(min=0)]
        old = (before + W - 1).clamp(0, max(W - 2, 0))
        earlier = torch.zeros_like(hT) if h0 is None else torch.gather(h0, 1, old.unsqueeze(-1).expand(n, W - 1, C))
        hT = torch.where((before >= 0).unsqueeze(-1), hT, earlier)
        return y.to(x.dtype).view(B, T, C), hT.to(x.dtype)
    d = _rows(s["dy"]).float()
    if c["silu"]:
        d = d * _dsilu(pre)
    dx = torch.zeros_like(X)
    dh0 = torch.zeros((n, W - 1, C), device=x.device)
    dw = torch.empty((C, W), device=x.device)
    for w, (tap, inside, row, back) in enumerate(taps):
        dw[:, w] = (d * tap).sum(0, dtype=torch.float64).float()
        part = torch.where(inside.unsqueeze(-1), d * weight[:, w], 0.0)
        dx[:B * T - back] += part[back:] if back else part
        if back:
            out = torch.nonzero(~inside).squeeze(-1)
            dh0.index_put_((seq[out], row[out]), d[out] * weight[:, w], accumulate=True)
    if s["dh_T"] is not None:
        for j in range(W - 1):
            at = cu[1:] - (W - 1) + j
            inside = at >= cu[:-1]
            g = s["dh_T"][:, j].float()
            dx.index_add_(0, at[inside], g[inside])
            out = torch.nonzero(~inside).squeeze(-1)
            dh0.index_put_((out, (at - cu[:-1] + W - 1)[out]), g[out], accumulate=True)
    grads = dict(dx=dx.to(x.dtype).view(B, T, C), dweight=dw, dh0=dh0.to(x.dtype))
    if s["bias"] is not None:
        grads["dbias"] = d.sum(0, dtype=torch.float64).float()
    return grads


def _conv_step_plain(s):
    c = s["case"]
    x, state = s["x"], s["state"]
    here = (s["slots"] >= 0) & (s["slots"] < state.shape[0])
    rows = torch.where(here, s["slots"], 0).long()
    window = torch.cat([state[rows], x.unsqueeze(1)], 1)                       # [B, W, C]
    pre = (window.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = (_silu(pre) if c["silu"] else pre).masked_fill(~here.unsqueeze(-1), 0.0)
    state[rows[here]] = window[here][:, 1:]
    return y.to(x.dtype), state


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, from zero: doubling within blocks of tokens, then over the blocks' ends."""
    T = a.shape[0]
    L = min(BLOCK, T)
    K = -(-T // L)
    if K * L != T:
        rest = a.new_ones((K * L - T,) + a.shape[1:])
        a, b = torch.cat([a, rest]), torch.cat([b, rest * 0])
    a, b = a.reshape(K, L, *a.shape[1:]), b.reshape(K, L, *b.shape[1:])
    d = 1
    while d < L:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    if K > 1:
        ends = _scan(a[:, -1], b[:, -1])
        b = torch.cat([b[:1], b[1:] + a[1:] * ends[:-1].unsqueeze(1)])
    return b.reshape(K * L, *b.shape[2:])[:T]


def _ssm_parts(s):
    """Per token in fp32: step, its input to the state, decays and what is added, x, B, C, gate; sequences."""
    x = s["x"]
    B, T, C = x.shape
    N = s["A"].shape[1]
    cu = _cu(s, B, T)
    v = _rows(s["dt"]).float() + s["dt_bias"]
    step = torch.nn.functional.softplus(v, threshold=40.0)
    X = _rows(x).float()
    per = C // s["Bm"].shape[2]
    Bm, Cm = (_rows(s[k]).float().repeat_interleave(per, 1) for k in ("Bm", "Cm"))      # [M, C, N]
    a = torch.exp(step.unsqueeze(-1) * s["A"])
    b = (step * X).unsqueeze(-1) * Bm
    lens = cu[1:] - cu[:-1]
    first, seqs = cu[:-1][lens > 0], torch.nonzero(lens > 0).squeeze(-1)
    a0 = a[first]
    if s["h0"] is not None:
        b[first] += a0 * s["h0"][seqs]
    open_a = a.clone() if s["case"]["op"] == "ssm_bwd" else None
    a[first] = 0
    return X, v, step, Bm, Cm, a, b, open_a, cu, first, seqs


def _ssm_plain(s):
    c = s["case"]
    x = s["x"]
    B, T, C = x.shape
    X, v, step, Bm, Cm, a, b, open_a, cu, first, seqs = _ssm_parts(s)
    M, N = B * T, s["A"].shape[1]
    n = cu.numel() - 1
    h = _scan(a, b)
    out = (h * Cm).sum(-1)
    if s["D"] is not None:
        out = out + s["D"] * X
    z = None if s["z"] is None else _rows(s["z"]).float()
    last = cu[1:][seqs] - 1
    if c["op"] != "ssm_bwd":
        y = out if z is None else out * _silu(z)
        hT = torch.zeros((n, C, N), device=x.device) if s["h0"] is None else s["h0"].clone()
        hT[seqs] = h[last]
        return y.to(DTYPES[c["o"]]).view(B, T, C), hT
    dt = x.dtype
    dy = _rows(s["dy"]).float()
    ds = dy if z is None else dy * _silu(z)
    # the cotangent of h_t comes from its own output and from h_{t+1}
    add = ds.unsqueeze(-1) * Cm
    if s["dh_T"] is not None:
        add[last] += s["dh_T"][seqs]
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])            # (zero where the next token starts a sequence)
    dh = _scan(nxt.flip(0), add.flip(0)).flip(0)
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[first] = 0.0 if s["h0"] is None else s["h0"][seqs]
    g = open_a * prev * dh
    G = s["Bm"].shape[2]
    du = (Bm * dh).sum(-1)
    dstep = X * du + (s["A"] * g).sum(-1)
    dv = dstep * torch.sigmoid(v)
    dx = step * du
    if s["D"] is not None:
        dx = dx + s["D"] * ds
    dh0 = torch.zeros((n, C, N), device=x.device) if s["dh_T"] is None else s["dh_T"].clone()
    dh0[seqs] = (open_a * dh)[first]
    grads = dict(dx=dx.to(dt).view(B, T, C), ddt=dv.to(dt).view(B, T, C),
                 dA=(step.unsqueeze(-1) * g).sum(0, dtype=torch.float64).float(),
                 dB=((step * X).unsqueeze(-1) * dh).view(M, G, C // G, N).sum(2).to(dt).view(B, T, G, N),
                 dC=(ds.unsqueeze(-1) * h).view(M, G, C // G, N).sum(2).to(dt).view(B, T, G, N),
                 ddt_bias=dv.sum(0, dtype=torch.float64).float(), dh0=dh0)
    if s["D"] is not None:
        grads["dD"] = (ds * X).sum(0, dtype=torch.float64).float()
    if z is not None:
        grads["dz"] = (dy * out * _dsilu(z)).to(dt).view(B, T, C)
    return grads


def _ssm_step_plain(s):
    c = s["case"]
    x, state = s["x"], s["state"]
    C = x.shape[1]
    here = (s["slots"] >= 0) & (s["slots"] < state.shape[0])
    rows = torch.where(here, s["slots"], 0).long()
    step = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"], threshold=40.0)
    per = C // s["Bm"].shape[1]
    Bm, Cm = (s[k].float().repeat_interleave(per, 1) for k in ("Bm", "Cm"))
    h = torch.exp(step.unsqueeze(-1) * s["A"]) * state[rows] + (step * x.float()).unsqueeze(-1) * Bm
    y = (h * Cm).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * x.float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    y = y.masked_fill(~here.unsqueeze(-1), 0.0)
    state[rows[here]] = h[here]
    return y.to(DTYPES[c["o"]]), state


def _verify_plain(s):
    """One sweep over the nodes: those that hang on the node reached are its children, in their order.  Probabilities are held
    in 64 bits: what is compared and summed decides a token."""
    tokens, parents, target, draft, uniform = s["tokens"].long(), s["parents"].long(), s["target"], s["draft"], s["uniform"].double()
    B, n = tokens.shape
    dev = tokens.device
    row = torch.arange(B, device=dev)
    at = torch.full((B,), -1, device=dev)
    p = target[row, 0].double()
    mass = torch.ones(B, dtype=torch.float64, device=dev)          # of p, which is held unscaled
    path = torch.full((B, n), -1, dtype=torch.int32, device=dev)
    count = torch.zeros(B, dtype=torch.long, device=dev)
    taken = torch.zeros(B, dtype=torch.float64, device=dev)        # with draft probabilities: how often they were taken off
    for r in range(n):
        child = parents[:, r] == at
        x = tokens[:, r]
        px = p[row, x]
        if draft is None:
            ok = child & (uniform[:, r] * mass < px)
            no = child & ~ok
            mass = torch.where(no, mass - px, mass)
            p[row[no], x[no]] = 0.0
        else:
            q = draft[row, (at + 1).clamp(max=n - 1)].double()
            ok = child & (uniform[:, r] * mass * q[row, x] < px)
            no = child & ~ok
            rest = torch.clamp(target[row, at + 1].double() - (taken + mass).unsqueeze(-1) * q, min=0.0)
            left = rest.sum(-1)
            no = no & (left > 0)
            taken = torch.where(no, taken + mass, taken)
            p = torch.where(no.unsqueeze(-1), rest, p)
            mass = torch.where(no, left, mass)
        at = torch.where(ok, r, at)
        mass, taken = torch.where(ok, 1.0, mass), torch.where(ok, 0.0, taken)
        p = torch.where(ok.unsqueeze(-1), target[row, at + 1].double(), p)
        path[row[ok], count[ok]] = r
        count = count + ok
    total = p.cumsum(-1)
    beyond = total > (uniform[:, n] * total[:, -1]).unsqueeze(-1)
    token = torch.where(beyond.any(-1), beyond.int().argmax(-1), -1)
    return at.to(torch.int32), token.to(torch.int32), path


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "verify":
            return _verify_plain(s)
        if op.startswith("conv"):
            return _conv_step_plain(s) if op == "conv_step" else _conv_plain(s)
        return _ssm_step_plain(s) if op == "ssm_step" else _ssm_plain(s)
    import linear_attention_rnn_gdn_amd as gdn

    if op == "verify":
        return gdn.tree_verify(s["tokens"], s["parents"], s["target"], s["uniform"], draft=s["draft"])
    if op.startswith("conv"):
        kw = dict(bias=s["bias"], activation="silu" if c["silu"] else None)
        if op == "conv_step":
            return gdn.conv_step(s["x"], s["weight"], s["state"], slots=s["slots"], **kw), s["state"]
        if op == "conv_fwd":
            return gdn.conv_fwd(s["x"], s["weight"], h0=s["h0"], **kw)
        if op == "conv_varlen":
            return gdn.conv_fwd_varlen(s["x"], s["weight"], s["cu"], h0=s["h0"], **kw)
        return gdn.conv_bwd(s["x"], s["weight"], s["dy"], h0=s["h0"], dh_T=s["dh_T"], **kw)
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "ssm_step":
        return gdn.ssm_step(*args, s["state"], slots=s["slots"], o_dtype=DTYPES[c["o"]], **kw), s["state"]
    if op == "ssm_fwd":
        return gdn.ssm_fwd(*args, h0=s["h0"], o_dtype=DTYPES[c["o"]], **kw)
    if op == "ssm_varlen":
        return gdn.ssm_fwd_varlen(*args, s["cu"], h0=s["h0"], o_dtype=DTYPES[c["o"]], **kw)
    return gdn.ssm_bwd(*args, s["dy"], h0=s["h0"], dh_T=s["dh_T"], **kw)


# ---------------------------------------------------------------------------
# 64-bit values from the definitions: every sequence by itself, gradients by differentiating the definition


def _spans(s):
    c = s["case"]
    if "n_seq" in c:
        cu = _offsets(c)
        return [(0, cu[i], cu[i + 1]) for i in range(c["n_seq"])]
    return [(b, 0, c["T"]) for b in range(c["B"])]


def _exact_conv(s):
    c = s["case"]
    W, C = c["W"], c["C"]
    grads = c["op"] == "conv_bwd"
    x, weight = s["x"].double(), s["weight"].double()
    bias = None if s["bias"] is None else s["bias"].double()
    spans = _spans(s)
    h0 = torch.zeros((len(spans), W - 1, C), dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    y, hT = torch.zeros_like(x), torch.zeros_like(h0)
    leaves = [t for t in (x, weight, bias, h0) if t is not None]
    if grads:
        for t in leaves:
            t.requires_grad_(True)
    total = 0.0
    for i, (b, lo, hi) in enumerate(spans):
        long = torch.cat([h0[i], x[b, lo:hi]])
        out = torch.einsum("tcw,cw->tc", long.unfold(0, W, 1), weight) if hi > lo else long[:0]
        out = out if bias is None else out + bias
        out = torch.nn.functional.silu(out) if c["silu"] else out
        if grads:
            total = total + (out * s["dy"][b, lo:hi].double()).sum()
            if s["dh_T"] is not None:
                total = total + (long[-(W - 1):] * s["dh_T"][i].double()).sum()
        else:
            y[b, lo:hi], hT[i] = out, long[-(W - 1):]
    if not grads:
        return y, hT
    got = dict(zip(("dx", "dweight") + (("dbias",) if bias is not None else ()) + ("dh0",), torch.autograd.grad(total, leaves)))
    return got


def _exact_ssm(s):
    c = s["case"]
    if sum(_lengths(c)) > 80000:   # a token at a time: too long
        return None
    grads = c["op"] == "ssm_bwd"
    names = ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias"]
    v = {k: None if s[k] is None else s[k].double().contiguous() for k in names}
    spans = _spans(s)
    C, N = c["C"], c["N"]
    h0 = torch.zeros((len(spans), C, N), dtype=torch.float64, device=v["x"].device) if s["h0"] is None else s["h0"].double()
    v["h0"] = h0
    if grads:
        for t in v.values():
            if t is not None:
                t.requires_grad_(True)
    per = C // c["G"]
    step = torch.nn.functional.softplus(v["dt"] + v["dt_bias"], threshold=200.0)
    y, hT, total = torch.zeros_like(v["x"]), torch.zeros_like(h0), 0.0
    for i, (b, lo, hi) in enumerate(spans):
        h, outs = h0[i], []
        for d, x, Bt, Ct in zip(*(t[b, lo:hi].unbind(0) for t in (step, v["x"], v["Bm"], v["Cm"]))):
            d = d.unsqueeze(-1)
            Bt, Ct = (t.unsqueeze(1).expand(c["G"], per, N).reshape(C, N) for t in (Bt, Ct))
            h = torch.exp(d * v["A"]) * h + d * x.unsqueeze(-1) * Bt
            outs.append((h * Ct).sum(-1))
        if hi > lo:
            out = torch.stack(outs)
            if v["D"] is not None:
                out = out + v["D"] * v["x"][b, lo:hi]
            if v["z"] is not None:
                out = out * torch.nn.functional.silu(v["z"][b, lo:hi])
            if grads:
                total = total + (out * s["dy"][b, lo:hi].double()).sum()
            else:
                y[b, lo:hi] = out
        if not grads:
            hT[i] = h
        elif s["dh_T"] is not None:
            total = total + (h * s["dh_T"][i].double()).sum()
    if not grads:
        return y, hT
    called = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", z="dz", dt_bias="ddt_bias", h0="dh0")
    keys = [k for k in v if v[k] is not None]
    return {called[k]: g for k, g in zip(keys, torch.autograd.grad(total, [v[k] for k in keys]))}


def _exact_steps(s):
    c = s["case"]
    state = s["state"].double()
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device=state.device)
    for b, slot in enumerate(s["slots"].tolist()):
        if not 0 <= slot < c["slots"]:
            continue
        x = s["x"][b].double()
        if c["op"] == "conv_step":
            window = torch.cat([state[slot], x.unsqueeze(0)])
            out = torch.einsum("wc,cw->c", window, s["weight"].double())
            out = out if s["bias"] is None else out + s["bias"].double()
            y[b] = torch.nn.functional.silu(out) if c["silu"] else out
            state[slot] = window[1:]
            continue
        d = torch.log1p(torch.exp(s["dt"][b].double() + s["dt_bias"].double()))
        per = c["C"] // c["G"]
        group = torch.arange(c["C"], device=x.device) // per
        h = torch.exp(torch.einsum("c,cn->cn", d, s["A"].double())) * state[slot] + torch.einsum("c,cn->cn", d * x, s["Bm"][b].double()[group])
        out = torch.einsum("cn,cn->c", h, s["Cm"][b].double()[group])
        out = out if s["D"] is None else out + s["D"].double() * x
        y[b] = out if s["z"] is None else out * torch.nn.functional.silu(s["z"][b].double())
        state[slot] = h
    return y, state


def _exact_verify(s):
    B, n = s["tokens"].shape
    tokens, parents, u = s["tokens"].tolist(), s["parents"].tolist(), s["uniform"].double().tolist()
    last, token, paths = [], [], []
    for b in range(B):
        at, path = -1, []
        while True:
            p = s["target"][b, at + 1].double()
            q = None if s["draft"] is None or at + 1 >= n else s["draft"][b, at + 1].double()
            whole, found = 1.0, None
            for r in range(n):
                if parents[b][r] != at or r <= at:
                    continue
                x = tokens[b][r]
                if q is None:
                    if u[b][r] * whole < float(p[x]):
                        found = r
                        break
                    whole -= float(p[x])
                    p = p.clone()
                    p[x] = 0.0
                else:
                    if u[b][r] * float(q[x]) < float(p[x]):
                        found = r
                        break
                    rest = torch.clamp(p - q, min=0.0)
                    left = float(rest.sum())
                    p = rest / left if left > 0 else p
            if found is None:
                break
            at = found
            path.append(at)
        total = p.cumsum(0)
        beyond = torch.nonzero(total > u[b][n] * total[-1])
        last.append(at)
        token.append(int(beyond[0]) if len(beyond) else -1)
        paths.append(path + [-1] * (n - len(path)))
    dev = s["tokens"].device
    return tuple(torch.tensor(v, dtype=torch.int32, device=dev) for v in (last, token, paths))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(s)
    if op.endswith("step"):
        return _exact_steps(s)
    return _exact_conv(s) if op.startswith("conv") else _exact_ssm(s)
