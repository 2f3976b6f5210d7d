"""The commit of accepted paths where rows of a call share a slot: drafts
forked from one sequence, of which one is accepted.  Of the rows that name a
slot, the first one that commits anything is run; a row that commits nothing
(its last node is outside the tree, or absent) claims nothing.

Tolerance: that of the other operators on a pool (2e-5 of the tensor's RMS).  A
committed element is the old one times a decay plus at most 64 products, one
rounding of 2^-24 each and three for the weight: 67 roundings, fewer than the
256 from which that bound is derived.
"""
import numpy as np
import pytest
import torch

from test_states import DK, TREES, _close, _cuda, _draw, _np, _parents, _tree_ref, gdn  # noqa: F401


def _accepted(parents, last):
    """The node whose path row b commits, or None."""
    if not 0 <= last < len(parents):
        return None
    at = last
    while at != -1:
        p = int(parents[at])
        if not -1 <= p < at:
            return None
        at = p
    return last


def _commit_ref(S, states, parents, last, slots):
    """First row of a slot that commits something; returns (pool, rows run)."""
    S, rows = S.copy(), {}
    for b, s in enumerate(slots):
        if 0 <= s < S.shape[0] and s not in rows and _accepted(parents[b], int(last[b])) is not None:
            rows[s] = b
            S[s] = states[b][int(last[b])]
    return S, rows


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,delta", [("bf16", True), ("f32", False)])
@pytest.mark.parametrize("Hv", [2, 32])          # 32 and 64 columns of a state per workgroup
def test_a_row_that_accepts_nothing_leaves_the_slot_to_the_next(gdn, Hv, dtype, delta):  # noqa: F811
    n = 7
    tree = [-1, 0, 1, 1, -2, 4, 0]               # nodes 4 and 5 are absent
    rows = [  # slot, last
        (0, -1), (0, 3),                         # nothing accepted, then a path
        (1, 4), (1, 2),                          # an absent node, then a path
        (2, 5), (2, 6),                          # a node that hangs on an absent one, then a path
        (3, n), (3, 1),                          # past the tree
        (4, -2 ** 31), (4, 2 ** 31 - 1), (4, -1), (4, 0),
        (5, 3), (5, 6), (5, -1),                 # two paths: the first of them
        (6, -1), (6, 4),                         # none
        (-1, 3), (9, 3),                         # rows without a state
    ]
    slots, last = [r[0] for r in rows], [r[1] for r in rows]
    B, n_slots = len(rows), 9
    x = _draw(B, n, 1, Hv, n_slots, dtype, seed=61, delta=delta)
    parents = np.array([tree] * B, dtype=np.int32)
    _, _, states = _tree_ref(x, parents, slots)
    S_ref, ran = _commit_ref(_np(x["state"]), states, parents, last, slots)
    assert ran == {0: 1, 1: 3, 2: 5, 3: 7, 4: 11, 5: 12}
    c = _cuda(x)
    _, u = gdn.tree_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], _i32(parents), c["state"], slots=_i32(slots))
    gdn.tree_commit(c["k"], u, c["g"], _i32(parents), _i32(last), c["state"], slots=_i32(slots))
    _close("state", c["state"], S_ref)
    for s in (6, 7, 8):
        assert torch.equal(c["state"][s].cpu(), x["state"][s])


@pytest.mark.gpu
def test_forks_of_one_sequence_far_apart_in_the_batch(gdn):  # noqa: F811
    # 600 forks of two sequences: the accepted one stands behind more rows than a workgroup has threads
    B, n, Hv = 600, 3, 2
    x = _draw(B, n, 1, Hv, 2, "bf16", seed=62)
    parents = _parents("chain", B, n, 0)
    slots, last = [b % 2 for b in range(B)], [-1] * B
    last[530], last[577], last[598], last[599] = 2, 1, 0, 2
    _, _, states = _tree_ref(x, parents, slots)
    S_ref, ran = _commit_ref(_np(x["state"]), states, parents, last, slots)
    assert ran == {0: 530, 1: 577}
    c = _cuda(x)
    _, u = gdn.tree_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], _i32(parents), c["state"], slots=_i32(slots))
    for _ in range(2):   # the same call on the same pool: the same bits
        state = c["state"].clone()
        gdn.tree_commit(c["k"], u, c["g"], _i32(parents), _i32(last), state, slots=_i32(slots))
        _close("state", state, S_ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,o_dtype,delta,fixed", [
    ("bf16", "bf16", True, False), ("bf16", "f32", False, False), ("f32", "f32", True, True), ("f32", "bf16", False, True)])
@pytest.mark.parametrize("B,n,Hqk,Hv,kind", TREES)
def test_check_and_commit_of_drawn_trees(gdn, B, n, Hqk, Hv, kind, dtype, o_dtype, delta, fixed):  # noqa: F811
    # the trees, slots and accepted nodes of test_states.test_tree, all its checks, with this rule for shared slots
    n_slots = min(B, 6) + 2
    x = _draw(B, n, Hqk, Hv, n_slots, dtype, seed=n + B, fixed=fixed, delta=delta)
    parents = _parents(kind, B, n, seed=n)
    rs = np.random.RandomState(n)
    slots = rs.randint(0, n_slots, B)
    if B > 2:
        slots[1], slots[2] = -1, n_slots
    o_ref, u_ref, states = _tree_ref(x, parents, slots)
    dead = torch.tensor([[r not in states[b] for r in range(n)] for b in range(B)])
    for key in ("q", "k", "v", "beta") + (() if fixed else ("g",)):
        if x[key] is not None:
            x[key][dead] = float("nan")
    c = _cuda(x)
    before = c["state"].clone()
    o, u = gdn.tree_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], _i32(parents), c["state"], slots=_i32(slots),
                        o_dtype={"bf16": torch.bfloat16, "f32": torch.float32}[o_dtype])
    assert torch.equal(c["state"], before)
    _close("o", o, o_ref, o_dtype == "bf16")
    _close("u", u, u_ref)
    last = rs.randint(-1, n + 1, B)
    last[0] = n - 1
    S_ref, _ = _commit_ref(_np(before), states, parents, last, slots)
    u[dead.cuda()] = float("nan")
    got = gdn.tree_commit(c["k"], u, c["g"], _i32(parents), _i32(last), c["state"], slots=_i32(slots))
    assert got is c["state"] and got.shape[-1] == DK
    _close("state", got, S_ref)
