"""Verification: entries of the probabilities that count nothing, in the walk as in the draw."""

import numpy as np
import pytest
import torch

from oracle import step as oracle

gpu = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")


# (target row of the root, draft row of the first token or None, parents, tokens, uniforms, rows kept, next token):
# the row of every kept token puts all on token 6
WALKS = [
    # a chain's token with an entry of infinity, NaN, below zero
    ([0.1, INF, 0.3, 0, 0, 0, 0], None, None, [0, 1], [0.9, 0.5], 1, 2),
    ([0.1, NAN, 0.3, 0, 0, 0, 0], None, None, [0, 1], [0.9, 0.0], 1, 2),
    ([0.1, -0.5, 0.3, 0, 0, 0, 0], None, None, [0, 1], [0.9, 0.0], 1, 2),
    # the same with draft probabilities, of any kind
    ([0.1, INF, 0.3, 0, 0, 0, 0], [0, 0.5, 0, 0, 0, 0, 0], None, [0, 1], [0.9, 0.5], 1, 2),
    ([0.1, -0.1, 0.3, 0, 0, 0, 0], [0, -0.5, 0, 0, 0, 0, 0], None, [0, 1], [0.0, 0.5], 1, 0),
    ([0.1, 0.2, 0.3, 0, 0, 0, 0], [0, NAN, 0, 0, 0, 0, 0], None, [0, 1], [0.9, 0.0], 1, 2),
    ([0.1, 0.2, 0.3, 0, 0, 0, 0], [0, INF, 0, 0, 0, 0, 0], None, [0, 1], [0.9, 0.0], 1, 2),
    # siblings behind one whose entry counts nothing: what is left is 1 (0.25 < 0.3, 0.45 >= 0.3)
    ([0.1, NAN, 0.3, 0.2, 0, 0, 0], None, [0, 0, 0], [0, 1, 2], [0.5, 0.5, 0.25], 2, 6),
    ([0.1, INF, 0.3, 0.2, 0, 0, 0], None, [0, 0, 0], [0, 1, 2], [0.5, 0.5, 0.25], 2, 6),
    ([0.1, INF, 0.3, 0.2, 0, 0, 0], None, [0, 0, 0], [0, 1, 2], [0.9, 0.5, 0.45], 1, 3),
    ([0.1, -4.0, 0.3, 0.2, 0, 0, 0], None, [0, 0, 0], [0, 1, 2], [0.5, 0.5, 0.25], 2, 6),
]


def build_case(walk):
    row, draft, parents, tokens, uniforms, kept, following = walk
    target = torch.zeros(len(tokens), len(row))
    target[:, 6] = 1.0
    target[0] = torch.tensor(row)
    q = None
    if draft is not None:
        q = torch.zeros(target.shape)
        q[1] = torch.tensor(draft)
    return target, tokens, [0, len(tokens)], torch.tensor(uniforms), q, parents


@pytest.mark.parametrize("walk", WALKS)
def test_oracle_by_hand(walk):
    target, tokens, off, u, q, parents = build_case(walk)
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    kept, following, _ = oracle.verify(f(target), tokens, off, f(u), f(q), parents)
    assert (kept, following) == ([walk[5]], [walk[6]])


@gpu
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("walk", WALKS)
def test_entries_that_count_nothing(jg, walk, half):
    target, tokens, off, u, q, parents = build_case(walk)
    dtype = torch.bfloat16 if half else torch.float32
    target, q = target.to(dtype), None if q is None else q.to(dtype)
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    want = oracle.verify(f(target), tokens, off, f(u), f(q), parents)
    got = jg.jgdpa_verify(target.cuda(), i32(tokens), i32(off), u.cuda(), draft_probs=None if q is None else q.cuda(),
                          parents=None if parents is None else i32(parents))
    assert [g.cpu().tolist() for g in got[:3]] == [list(w) for w in want]
