"""The fp64 references of the draft-tree operators against the recurrence's oracle, closed forms and each other."""
import numpy as np
import pytest

from oracle import oracle, sublayer, tree


def _chain(T, H, d, seed):
    r = np.random.default_rng(seed)
    q, k = (sublayer.l2norm(r.standard_normal((T, H, d)), 0.0) for _ in range(2))
    return (q, k, r.standard_normal((T, H, d)), -np.exp(r.normal(-1, 0.5, (T, H, d))),
            1 / (1 + np.exp(-r.standard_normal((T, H)))), 0.1 * r.standard_normal((1, H, d, d)))


def test_a_chain_is_the_recurrence():
    q, k, v, g, beta, S0 = _chain(7, 2, 16, 1)
    o, u, states = tree.tree_step(q, k, v, g, beta, [-1, 0, 1, 2, 3, 4, 5], [0, 7], [0], S0)
    o_ref, S_ref, _ = oracle.run(q, k, v, g, beta, [0, 7], S0=S0)
    assert oracle.rel_err(o, o_ref) < 1e-13 and oracle.rel_err(states[6], S_ref[0]) < 1e-13


def test_every_path_of_a_tree_is_a_chain():
    q, k, v, g, beta, S0 = _chain(6, 1, 16, 2)
    parent = [-1, 0, 0, 1, 2, 2]
    o, _, states = tree.tree_step(q, k, v, g, beta, parent, [0, 6], [0], S0)
    for leaf, path in ((3, [0, 1, 3]), (5, [0, 2, 5])):
        o_ref, S_ref, _ = oracle.run(*(x[path] for x in (q, k, v, g, beta)), [0, len(path)], S0=S0)
        assert oracle.rel_err(o[leaf], o_ref[-1]) < 1e-13 and oracle.rel_err(states[leaf], S_ref[0]) < 1e-13


@pytest.mark.parametrize("W", [1, 4])
def test_the_convolution_of_a_chain_is_the_short_convolution(W):
    r = np.random.default_rng(3)
    x, w, pool = r.standard_normal((5, 8)), r.standard_normal((8, W)), r.standard_normal((1, W - 1, 8))
    y = tree.tree_conv(x, w, [-1, 0, 1, 2, 3], [0, 5], [0], pool)
    y_ref, _ = sublayer.short_conv(x, w, [0, 5], pool)
    assert np.abs(y - y_ref).max() < 1e-14


def test_verification_by_hand():
    logits = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.1, 0.8], [1 / 3, 1 / 3, 1 / 3]]))
    q = np.array([[0.2, 0.7, 0.1]] * 3)
    # token 1 at the root: accepted while u < 0.3 / 0.7; then the child's own row gives the next token
    hit = tree.draft_verify(logits[:2], [0, 1], [-1, 0], [0, 2], [0, 0.42], [0.5], q)
    assert hit == ([[0, 1]], [2])
    # rejected: the excess is (0.3, 0, 0.1) / 0.4
    for u, token in ((0.74, 0), (0.76, 2)):
        assert tree.draft_verify(logits[:2], [0, 1], [-1, 0], [0, 2], [0, 0.43], [u], q) == ([[0]], [token])
    # chosen drafts: token 0 rejected with u = 0.6 leaves (0, 0.6, 0.4), in which token 1 is accepted below 0.6
    assert tree.draft_verify(logits, [0, 0, 1], [-1, 0, 0], [0, 3], [0, 0.6, 0.59], [0.5]) == ([[0, 2]], [1])
    assert tree.draft_verify(logits, [0, 0, 1], [-1, 0, 0], [0, 3], [0, 0.6, 0.61], [0.5]) == ([[0]], [2])
    # greedy: only the most likely token is accepted
    assert tree.draft_verify(logits, [0, 0, 1], [-1, 0, 0], [0, 3], [0, 0.9, 0.0], [0.9], None, [0.0]) == ([[0, 1]], [2])


def test_verification_keeps_the_target_distribution():
    """With drafts drawn from q and any number of siblings, the first kept token follows p: integrated exactly over
    the drafts and on a fine grid over the random numbers."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.7, 0.1])
    grid = (np.arange(20) + 0.5) / 20
    got = np.zeros(3)
    for a in range(3):
        for b in range(3):
            for ua in grid:
                for ub in grid:
                    for un in grid:
                        paths, nxt = tree.draft_verify(np.log([p, p, p]), [0, a, b], [-1, 0, 0], [0, 3], [0, ua, ub], [un], [q] * 3)
                        got[[a, b][paths[0][1] - 1] if len(paths[0]) > 1 else nxt[0]] += q[a] * q[b] / 8000
    assert np.abs(got - p).max() < 0.04  # the grid's own resolution: 1/20 in each of its decisions
