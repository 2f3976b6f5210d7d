"""The verification of drafted tokens against its definition in fp64: integers,
which have to be equal.  Probabilities, random numbers and their comparisons
are drawn, so a comparison lies within fp64 rounding of a tie (2^-50 of the
whole, say) with a chance of 1e-15 each."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_rnn_gdn_amd as g

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()
    return g


def _draw(B, n, V, seed, draft=True, tree=True, near=0.8):
    gen = torch.Generator().manual_seed(seed)
    logits = 2.0 * torch.randn(B, n + 1, V, generator=gen)
    guess = near * logits[:, :n] + 0.8 * torch.randn(B, n, V, generator=gen)
    r = torch.arange(n)
    parents = torch.where(torch.rand(B, n, generator=gen) < 0.4, r - 1, (torch.rand(B, n, generator=gen) * (r + 1)).long() - 1) if tree else (r - 1).expand(B, n)
    parents = torch.minimum(parents, r - 1).to(torch.int32).contiguous()
    q = torch.softmax(guess, -1)
    tokens = torch.zeros(B, n, dtype=torch.int32)
    for b in range(B):
        for i in range(n):
            tokens[b, i] = torch.multinomial(q[b, int(parents[b, i]) + 1], 1, generator=gen)
    return dict(tokens=tokens, parents=parents, target=torch.softmax(logits, -1), uniform=torch.rand(B, n + 1, generator=gen),
                draft=q if draft else None)


def _reference(x):
    """Row by row, child by child, every residual scaled as defined."""
    B, n = x["tokens"].shape
    V = x["target"].shape[2]
    tokens, parents = x["tokens"].tolist(), x["parents"].tolist()
    out = []
    for b in range(B):
        at, path = -1, []
        while True:
            p = np.nan_to_num(x["target"][b, at + 1].numpy().astype(np.float64), nan=0.0).clip(0)
            found, mass = None, 1.0
            for r in range(max(at + 1, 0), n):
                t = tokens[b][r]
                if parents[b][r] != at or not 0 <= t < V:
                    continue
                u = float(x["uniform"][b, r])
                if x["draft"] is None:
                    if u * mass < p[t]:
                        found = r
                        break
                    mass -= p[t]
                    p[t] = 0.0
                else:
                    q = x["draft"][b, at + 1].numpy().astype(np.float64)
                    if u * q[t] < p[t]:
                        found = r
                        break
                    rest = np.maximum(p - q, 0)
                    if rest.sum() > 0:
                        p = rest / rest.sum()
            if found is None:
                break
            at = found
            path.append(at)
        total = np.cumsum(p)
        beyond = np.nonzero(total > float(x["uniform"][b, n]) * total[-1])[0]
        out.append((at, int(beyond[0]) if len(beyond) else -1, path + [-1] * (n - len(path))))
    return [torch.tensor([o[i] for o in out], dtype=torch.int32) for i in range(3)]


def _same(gdn, x):
    want = _reference(x)
    got = gdn.tree_verify(*(x[k].cuda() for k in ("tokens", "parents", "target", "uniform")),
                          draft=None if x["draft"] is None else x["draft"].cuda())
    for name, a, b in zip(("last", "token", "path"), got, want):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b), (name, a.cpu(), b)
    return want


@pytest.mark.parametrize("draft", [True, False])
def test_reference_draws_from_the_target(draft):
    # the first token (accepted at the root, or drawn there) follows the target's probabilities, whatever the draft's: 20000 rows
    # of two siblings; a frequency is off by more than 5 sqrt(p (1 - p) / 20000) once in 10^6
    rows, V = 20000, 4
    gen = torch.Generator().manual_seed(3)
    p, q = torch.tensor([0.1, 0.5, 0.25, 0.15]), torch.tensor([0.4, 0.2, 0.2, 0.2])
    tokens = torch.multinomial(q, rows * 2, replacement=True, generator=gen).view(rows, 2).int() if draft else torch.tensor([[0, 2]]).expand(rows, 2).int()
    x = dict(tokens=tokens, parents=torch.full((rows, 2), -1, dtype=torch.int32), target=p.expand(rows, 3, V),
             uniform=torch.rand(rows, 3, generator=gen), draft=q.expand(rows, 2, V) if draft else None)
    last, token, _ = _reference(x)
    first = torch.where(last >= 0, tokens.gather(1, last.clamp(min=0).long().unsqueeze(1)).squeeze(1), token)
    seen = torch.bincount(first.long(), minlength=V) / rows
    assert ((seen - p).abs() <= 5 * (p * (1 - p) / rows).sqrt()).all(), seen


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (1, 1, 7), (3, 5, 64), (7, 16, 1001), (2, 64, 300), (2, 3, 4096), (2, 4, 4097), (1, 6, 40003), (65, 2, 130)])
def test_drawn_trees(gdn, B, n, V, tree, draft):
    for seed in (1, 2):
        for near in (0.95, 0.3):
            _same(gdn, _draw(B, n, V, 10 * seed + n, draft, tree, near))


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_many_siblings(gdn, draft):
    # all nodes hang on the root: many refusals in a row, and the same token twice
    x = _draw(6, 40, 50, 5, draft, near=0.0)
    x["parents"][:] = -1
    x["tokens"][:, 1::2] = x["tokens"][:, ::2]
    last, _, _ = _same(gdn, x)
    x["uniform"][:, :40] = 1 - 2.0 ** -24   # refuse wherever that is possible
    _same(gdn, x)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_absent_nodes_and_rows(gdn, draft):
    x = _draw(6, 8, 200, 6, draft)
    x["uniform"][:, :8] = 0.0                       # accept whatever has a probability
    x["parents"][0] = -2                            # a padded row
    x["parents"][1, 0], x["parents"][2, 3], x["parents"][3, 2] = 5, 3, -7
    x["tokens"][4, 0], x["tokens"][4, 1], x["tokens"][5, 2] = -1, 200, 2 ** 31 - 1
    _same(gdn, x)
    x["target"][0] = 0.0                            # no mass, no number, less than nothing
    x["target"][1, 0, 3:9] = float("nan")
    x["target"][2, :, ::3] *= -1
    _same(gdn, x)
    x["target"][0] = float("nan")
    want = _same(gdn, x)
    assert int(want[1][0]) == -1


@pytest.mark.gpu
def test_a_draft_equal_to_the_target_is_accepted(gdn):
    x = _draw(5, 7, 500, 8, True, tree=False)
    x["draft"] = x["target"][:, :7].contiguous()
    x["uniform"][:, :7] = 1 - 2.0 ** -24
    last, _, path = _same(gdn, x)
    assert (last == 6).all() and (path == torch.arange(7)).all()
    # refused all the same where the target has nothing, and then there is no residual: the next token is the target's
    x["tokens"][:, 0] = 3
    x["target"][:, 0, 3] = 0
    x["draft"] = x["target"][:, :7].contiguous()
    last, _, _ = _same(gdn, x)
    assert (last == -1).all()


@pytest.mark.gpu
def test_ends_of_the_random_numbers(gdn):
    x = _draw(4, 2, 9000, 9, False)
    x["target"][0], x["target"][1] = 0, 0
    x["target"][0, :, 8999] = 1                    # one token has all
    x["target"][1, :, 4096] = 0.5
    x["target"][1, :, 4095] = 0.5
    for u in (0.0, 0.5, 1 - 2.0 ** -24):
        x["uniform"][:] = u
        _same(gdn, x)


@pytest.mark.gpu
def test_check_verify_commit_step(gdn):
    # as a server runs them: the drafted tree's outputs, the path that verification accepts, its commit, the next token
    B, n, V = 3, 9, 120
    x = _draw(B, n, V, 10, True, near=0.9)
    gen = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    q, k, v = unit(r(B, n, 2, 128)), unit(r(B, n, 2, 128)), r(B, n, 4, 128)
    g, beta, state = -r(B, n, 4).abs(), torch.sigmoid(r(B, n, 4)), 0.3 * r(5, 4, 128, 128)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    parents = x["parents"].cuda()
    o, u = gdn.tree_fwd(q, k, v, g, beta, parents, state, slots)
    last, token, path = gdn.tree_verify(x["tokens"].cuda(), parents, x["target"].cuda(), x["uniform"].cuda(), draft=x["draft"].cuda())
    before = state.clone()
    gdn.tree_commit(k, u, g, parents, last, state, slots)
    assert (last >= 0).any() and torch.equal(last.cpu(), _reference(x)[0])
    for b in range(B):   # the accepted tokens one at a time
        one = before.clone()
        for t in [t for t in path[b].tolist() if t >= 0]:
            got = gdn.step(q[b:b + 1, t], k[b:b + 1, t], v[b:b + 1, t], g[b:b + 1, t], beta[b:b + 1, t], one, slots[b:b + 1].clone())
            assert (got[0] - o[b, t]).abs().max() <= 2e-5 * o.abs().max()
        s = int(slots[b])
        assert (one[s] - state[s]).abs().max() <= 2e-5 * state.abs().max()


@pytest.mark.gpu
def test_streams_graphs_and_workspaces(gdn):
    x = {k: t.cuda() for k, t in _draw(8, 12, 9001, 12).items()}
    call = lambda **kw: gdn.tree_verify(x["tokens"], x["parents"], x["target"], x["uniform"], draft=x["draft"], **kw)
    ref = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, here = call(stream=side), call()
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(ref, got, here))
    ws = torch.full((gdn._verify_plan(8, 12, 9001)[1],), 255, dtype=torch.uint8, device="cuda")
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
def test_refusals(gdn):
    x = {k: t.cuda() for k, t in _draw(2, 4, 30, 13).items()}
    f = lambda **kw: gdn.tree_verify(**{**x, **kw})
    for error, call in (
            (TypeError, lambda: f(tokens=x["tokens"].long())), (TypeError, lambda: f(target=x["target"].bfloat16())),
            (ValueError, lambda: f(parents=x["parents"][:1])), (ValueError, lambda: f(target=x["target"][:, :4].contiguous())),
            (ValueError, lambda: f(draft=x["draft"][:, :3].contiguous())), (ValueError, lambda: f(uniform=x["uniform"][:, :4].contiguous())),
            (ValueError, lambda: f(target=x["target"].transpose(1, 2).contiguous().transpose(1, 2))), (ValueError, lambda: f(tokens=x["tokens"].cpu())),
            (TypeError, lambda: f(draft=[1])), (ValueError, lambda: f(workspace=x["target"].view(-1).view(torch.uint8))),
            (gdn.GdnError, lambda: f(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
            (gdn.GdnError, lambda: gdn.tree_verify(torch.zeros(1, 65, dtype=torch.int32, device="cuda"), torch.zeros(1, 65, dtype=torch.int32, device="cuda"),
                                                   torch.ones(1, 66, 3, device="cuda"), torch.zeros(1, 66, device="cuda")))):
        with pytest.raises(error):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("V", [60, 1001, 9000, 32768, 32769, 40003])
def test_draft_values_below_zero_or_no_numbers_count_as_zero(gdn, V, tree):
    # the reference takes the draft with zeros in their place; most of the target's mass lies on tokens whose draft value is no
    # number, or every token without a probability has one below zero, so that a residual which took these as they are would
    # lose the one and draw the other
    x = _draw(4, 10, V, V + tree, True, tree, near=0.0)
    if tree:
        x["parents"][:3] = -1
    bad = torch.arange(V) % 5 == 2
    x["target"][0, :, bad] *= 50
    x["draft"][0, :, bad] = float("nan")
    x["target"][1, :, bad] = 0
    x["draft"][1, :, bad] = -0.25
    x["draft"][2] = float("nan")
    x["draft"][3, :, bad] *= -1
    clean = dict(x, draft=torch.nan_to_num(x["draft"], nan=0.0).clamp(min=0))
    for refuse in (False, True):
        if refuse:
            x["uniform"][:, :10] = 1 - 2.0 ** -24
        for u in (0.0, 0.3, 0.7, 1 - 2.0 ** -24):
            x["uniform"][:, 10] = u
            want = _reference(clean)
            got = gdn.tree_verify(*(x[k].cuda() for k in ("tokens", "parents", "target", "uniform")), draft=x["draft"].cuda())
            for name, a, b in zip(("last", "token", "path"), got, want):
                assert torch.equal(a.cpu(), b), (name, refuse, u, a.cpu(), b)
