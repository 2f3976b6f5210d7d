"""Outputs that a caller passes must lie apart from the inputs and from each
other: workgroups that still read an input run beside those that write.  The
gradients' walks, for one, each read dh_T (and the one of dq h0) while the walk
of dv writes dh0.  Such calls are refused before a launch."""
import pytest
import torch

from test_linear import D, _cuda, _draw


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_rnn_gdn_amd as g

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()
    return g


def test_spans():
    # (the check looks at addresses only: host tensors do)
    from linear_attention_rnn_gdn_amd import _check_apart

    x = torch.zeros(64)
    y = torch.zeros(8)
    _check_apart(((x[:16], "o"), (x[16:32], "u")), ((x[32:], "q"), (y, "k"), (None, "h0")))
    _check_apart(((None, "o"), (x[:0], "u")), ((x, "q"),))          # nothing is written there
    _check_apart(((x, "o"),), ((x[5:5], "q"),))                     # nothing is read there
    for out, into in ((x, x), (x[:16], x[15:]), (x[15:], x[:16]), (x, x[5:6]), (x[5:6], x), (x.view(torch.uint8)[60:64], x[15:16])):
        with pytest.raises(ValueError, match="h_T overlaps h0"):
            _check_apart(((out, "h_T"),), ((y, "q"), (into, "h0")))
    with pytest.raises(ValueError, match="u overlaps o"):
        _check_apart(((x[:16], "o"), (x[8:24], "u")), ((y, "q"),))


@pytest.mark.gpu
def test_gradients_refuse_outputs_over_inputs(gdn):
    x = _cuda(_draw(2, 40, 2, 2, "bf16", seed=71))
    args = dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], dO=x["dO"], h0=x["h0"], dh_T=x["dh_T"])
    ref = gdn.linear_chunk_bwd(**args)
    out = {n: torch.empty_like(t) for n, t in ref.items()}
    for name, over in (("dh0", "dh_T"), ("dh0", "h0"), ("dq", "q"), ("dk", "k"), ("dk", "q"), ("dv", "v"), ("dv", "dO"), ("dg", "g")):
        with pytest.raises(ValueError, match=f"{name} overlaps {over}"):
            gdn.linear_chunk_bwd(**args, out=dict(out, **{name: x[over]}))
    with pytest.raises(ValueError, match="dk overlaps dq"):
        gdn.linear_chunk_bwd(**args, out=dict(out, dk=out["dq"]))
    # a state's place shifted by one row of a pool
    pool = torch.zeros((3, 2, D, D), device="cuda")
    with pytest.raises(ValueError, match="dh0 overlaps dh_T"):
        gdn.linear_chunk_bwd(**dict(args, dh_T=pool[:2]), out=dict(out, dh0=pool[1:]))
    # nothing was launched: the inputs are as they were, and the call itself works
    got = gdn.linear_chunk_bwd(**args, out=out)
    assert got is out and all(torch.equal(got[n], ref[n]) for n in ref)


@pytest.mark.gpu
def test_forward_refuses_outputs_over_inputs(gdn):
    x = _cuda(_draw(2, 300, 2, 2, "bf16", seed=72))
    args = dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], o_dtype=torch.bfloat16)
    pool = torch.zeros((3, 2, D, D), device="cuda")
    for final in (pool[:2], pool[1:]):
        with pytest.raises(ValueError, match="h_T overlaps h0"):
            gdn.linear_chunk_fwd(**args, h0=pool[:2], final_state=final)
    for name in ("q", "k", "v"):
        with pytest.raises(ValueError, match=f"o overlaps {name}"):
            gdn.linear_chunk_fwd(**args, out=x[name])
    with pytest.raises(ValueError, match="workspace overlaps h0"):
        gdn.linear_chunk_fwd(**args, h0=pool[:2], workspace=pool.view(torch.uint8).view(-1))
    one = {n: x[n][:1] for n in ("q", "k", "v", "g")}
    with pytest.raises(ValueError, match="h_T overlaps h0"):
        gdn.linear_chunk_fwd_varlen(**one, cu_seqlens=[0, 100, 300], h0=pool[:2], final_state=pool[1:])
    o, h = gdn.linear_chunk_fwd(**args, h0=pool[:2])
    o2, h2 = gdn.linear_chunk_fwd(**args, h0=pool[:2], out=torch.empty_like(o), final_state=torch.empty_like(h))
    assert torch.equal(o, o2) and torch.equal(h, h2)


@pytest.mark.gpu
def test_pool_calls_refuse_outputs_over_inputs(gdn):
    B, n, H = 2, 3, 2
    r = lambda *s: torch.randn(*s, device="cuda")
    q, k, v = r(B, H, D), r(B, H, D), r(B, H, D)
    g, beta, state = -r(B, H).abs(), r(B, H).sigmoid(), r(4, H, D, D)
    for name, over in (("q", q), ("k", k), ("v", v), ("state", state[0, 0, :B * H].view(B, H, D))):
        with pytest.raises(ValueError, match=f"o overlaps {name}"):
            gdn.step(q, k, v, g, beta, state, out=over)
    q, k, v = r(B, n, H, D), r(B, n, H, D), r(B, n, H, D)
    g, beta = -r(B, n, H).abs(), r(B, n, H).sigmoid()
    p = torch.tensor([[-1, 0, 1]] * B, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="u overlaps v"):
        gdn.tree_fwd(q, k, v, g, beta, p, state, values=v)
    both = torch.empty_like(v)
    with pytest.raises(ValueError, match="u overlaps o"):
        gdn.tree_fwd(q, k, v, g, beta, p, state, out=both, values=both)
    o, u = gdn.tree_fwd(q, k, v, g, beta, p, state)
    o2, u2 = gdn.tree_fwd(q, k, v, g, beta, p, state, out=torch.empty_like(o), values=both)
    assert torch.equal(o, o2) and torch.equal(u, u2) and u2 is both
