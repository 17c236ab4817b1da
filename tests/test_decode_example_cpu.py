"""The drafting of examples/decode_draft.py, which needs no GPU."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import decode_draft as ex  # noqa: E402


@pytest.mark.parametrize("vocab", [1, 2, 50, 96, 97, 211])
@pytest.mark.parametrize("nodes", [1, 2, 13])
def test_drafted_trees_stay_within_the_vocabulary(vocab, nodes):
    for token in range(vocab):
        for table in ({}, {token: [vocab - 1, 0, vocab // 2]}):
            tokens, parents = ex.tree(table, token, nodes, vocab)
            assert len(tokens) == len(parents) == nodes and tokens[0] == token and parents[0] == -1
            assert all(0 <= t < vocab for t in tokens) and all(0 <= p < i for i, p in enumerate(parents) if i)


@pytest.mark.parametrize("n0,n_tokens,nodes,budget", [(40, 24, 8, 0), (40, 24, 8, 16), (5, 1, 3, 0), (50, 30, 6, 40),
                                                     (10, 7, 4, 500)])
def test_the_capacity_holds_the_most_uneven_acceptance(n0, n_tokens, nodes, budget):
    """One sequence accepts every node of every step, the other only its last token."""
    cap = ex.capacity(n0, n_tokens, nodes, budget)
    slow, rows = 1, n0
    assert rows <= cap
    while slow < n_tokens:
        rows = min(rows, budget) if budget else rows
        rows += nodes
        assert rows <= cap
        slow += 1
