"""Pins of the drafted-tree oracle (CPU only)."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from tests._np import to_np
from tests._trees import random_parents
from workload import TINY, append_inputs, mla_inputs


def test_ancestors_by_hand():
    parent = [-1, 0, 0, 1, -1, -2, 4]
    assert oracle.ancestors(parent, 3) == [3, 1, 0]
    assert oracle.ancestors(parent, 6) == [6, 4]
    assert oracle.ancestors(parent, 5) is None
    for bad in ([0], [-3], [-1, 1], [-2, 0], [-1, 2, 0]):
        with pytest.raises(ValueError):
            for s in range(len(bad)):
                oracle.ancestors(bad, s)


def test_chain_is_the_causal_decode_and_append():
    S, T = 5, [9, 5]
    x = mla_inputs(TINY, 2, S, T, 12, "f32", 3)
    chain = random_parents(2, S, 0, absent=False, chain=True)
    args = [to_np(x[k]) for k in ("q", "Lc", "Rc")]
    want = oracle.decode_absorbed(*args, T, to_np(x["kv_b"]), TINY.qk_nope, TINY.softmax_scale)
    got = oracle.decode_tree(*args, T, chain, to_np(x["kv_b"]), TINY.qk_nope, TINY.softmax_scale)
    assert np.allclose(got, want, rtol=0, atol=1e-12)
    a = append_inputs(TINY, 2, S, "f32", 4)
    comp, ln = to_np(a["comp"]), to_np(a["kv_a_ln"])
    for g, w in zip(oracle.cache_append_tree(comp, ln, 1e-6, T, chain, TINY.kv_lora),
                    oracle.cache_append(comp, ln, 1e-6, T, TINY.kv_lora)):
        assert np.allclose(g, w, rtol=0, atol=1e-12)


def test_a_branch_sees_only_its_ancestors():
    """A leaf's output is that of a chain made of its ancestors alone."""
    S, base = 6, 4
    parent = np.array([[-1, 0, 0, 1, 2, -2]])
    x = mla_inputs(TINY, 1, S, [base + S], base + S, "f32", 5)
    q, Lc, Rc, kv_b = (to_np(x[k]) for k in ("q", "Lc", "Rc", "kv_b"))
    got = oracle.decode_tree(q, Lc, Rc, [base + S], parent, kv_b, TINY.qk_nope, TINY.softmax_scale)
    pick = [0, 2, 4]
    rows = list(range(base)) + [base + j for j in pick]
    want = oracle.decode_absorbed(q[:, pick], Lc[:, rows], Rc[:, rows], [base + 3], kv_b, TINY.qk_nope, TINY.softmax_scale)
    assert np.allclose(got[0, pick], want[0], rtol=0, atol=1e-12)
    assert np.all(got[0, 5] == 0)


def _emitted(p, q, parent, draft_law, grid):
    """Distribution of the first emitted token, summed over every draw of the drafts
    and every cell of a grid of u (values at the cells' middles: exact when all
    thresholds lie on the cells' edges)."""
    V, S = len(p[0]), len(parent)
    law = [Fraction(0)] * V

    def spread(tokens, weight):
        if len(tokens) < S:
            for x in range(V):
                if draft_law[x]:
                    spread(tokens + [x], weight * draft_law[x])
            return
        cells = grid ** (S + 1)
        for cell in range(cells):
            u = [((cell // grid ** k) % grid + 0.5) / grid for k in range(S + 1)]
            path, token = oracle.tree_verify(p, q, tokens, parent, u)
            law[tokens[path[0]] if path else token] += weight / cells
    spread([], Fraction(1))
    return law


def test_emitted_token_has_the_targets_law():
    """Two siblings drawn from q: the first token out is distributed as p.  With
    these quarters every threshold on u is a multiple of 1/24."""
    p = [[0.5, 0.25, 0.25]] * 3
    q = [[0.25, 0.25, 0.5]] * 3
    law = _emitted(p, q, [-1, -1], [Fraction(1, 4), Fraction(1, 4), Fraction(1, 2)], 24)
    assert law == [Fraction(1, 2), Fraction(1, 4), Fraction(1, 4)]


def test_point_drafts_have_the_targets_law():
    p = [[0.5, 0.25, 0.25]] * 3
    law = [Fraction(0)] * 3
    n = 12
    for cell in range(n ** 3):
        u = [((cell // n ** k) % n + 0.5) / n for k in range(3)]
        path, token = oracle.tree_verify(p, None, [1, 0], [-1, -1], u)
        law[[1, 0][path[0]] if path else token] += Fraction(1, n ** 3)
    assert law == [Fraction(1, 2), Fraction(1, 4), Fraction(1, 4)]


def test_verify_by_hand():
    p = [[0.5, 0.5, 0.0], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]]
    q = [[0.0, 0.5, 0.5], [0.5, 0.5, 0.0], [0.5, 0.0, 0.5]]
    # node 0 (token 2, p 0) is rejected, what is left is all on token 0: node 1 (token 1) is too
    assert oracle.tree_verify(p, q, [2, 1], [-1, -1], [0.0, 0.0, 0.9]) == ([], 0)
    # node 0 accepted (u q = 0.2 < 0.5), node 1 below it accepted (p 1 > q 0.5), then a draw at node 1
    assert oracle.tree_verify(p, q, [1, 1], [-1, 0], [0.4, 0.9, 0.6]) == ([0, 1], 2)
    # the draw's threshold on a boundary belongs to the next token
    assert oracle.tree_verify(p, q, [1], [-2], [0.0, 0.5]) == ([], 1)


def test_commit_by_hand():
    cache = np.arange(8).reshape(1, 8, 1)
    got, T = oracle.tree_commit(cache, [7], [[1, 2, 4, -1, -1]], [3])
    assert T == [5] and got[0, :, 0].tolist() == [0, 1, 3, 4, 6, 5, 6, 7]
