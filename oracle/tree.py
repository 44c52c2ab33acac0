"""fp64 references of the draft-tree operators.

TEST INFRASTRUCTURE ONLY: tests may use this module; the library path never does, and nothing here is shared with
the CUDA code.  Each function goes by its operator's definition, one request, node and token at a time:

  tree_step     S_i = D_i S_p + k_i u_i^T with u_i = beta_i (v_i - (D_i S_p)^T k_i), o_i = S_i^T q_i, from a copy of
                the state per node (p: the node's parent; the pool's state for the root)
  tree_conv     y_i = sum_j w[:, j] x(j-th input before and at node i), carried inputs before the root
  draft_verify  children tried in order with the renormalised excess after each rejection, then inversion of the
                cumulative sum
"""
from __future__ import annotations

import numpy as np


def tree_step(q, k, v, g, beta, parent, cu, slots, pool):
    """(o, u [T, H, d], states [T, H, d, d]) in fp64."""
    q, k, v, g, beta, pool = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g, beta, pool))
    T, H, d = q.shape
    o, u, states = np.zeros((T, H, d)), np.zeros((T, H, d)), np.zeros((T, H, d, d))
    for n in range(len(cu) - 1):
        for r in range(cu[n], cu[n + 1]):
            before = pool[slots[n]] if parent[r] < 0 else states[cu[n] + parent[r]]
            S = np.exp(g[r])[:, :, None] * before
            u[r] = beta[r][:, None] * (v[r] - np.einsum("hcd,hc->hd", S, k[r]))
            states[r] = S + k[r][:, :, None] * u[r][:, None, :]
            o[r] = np.einsum("hcd,hc->hd", states[r], q[r])
    return o, u, states


def path_inputs(x, parent, row0, node, carried):
    """All inputs up to and with `node`, oldest first: carried inputs, then the path from the root."""
    path = []
    while node >= 0:
        path.append(x[row0 + node])
        node = parent[row0 + node]
    return np.array(list(carried) + path[::-1])


def tree_conv(x, w, parent, cu, slots, pool):
    x, w, pool = (np.asarray(a, dtype=np.float64) for a in (x, w, pool))
    W = w.shape[1]
    y = np.zeros_like(x)
    for n in range(len(cu) - 1):
        for i in range(cu[n + 1] - cu[n]):
            seq = path_inputs(x, parent, cu[n], i, pool[slots[n]])
            for j in range(W):
                y[cu[n] + i] += w[:, j] * seq[len(seq) - 1 - j]
    return y


def target_probabilities(logits, temperature):
    """p of one row; None where no logit is above -inf."""
    l = np.asarray(logits, dtype=np.float64).copy()
    l[np.isnan(l)] = -np.inf
    top = l.max()
    if top == -np.inf:
        return None
    if not temperature > 0:
        p = np.zeros_like(l)
        p[int(np.argmax(l))] = 1.0
        return p
    w = (l == top).astype(np.float64) if top == np.inf else np.exp((l - top) / temperature)
    return w / w.sum()


def draft_verify(logits, tokens, parent, cu, u_accept, u_next, draft_probs=None, temperature=None):
    """(paths, next tokens): a list of node lists and an int list."""
    paths, following = [], []
    for n in range(len(cu) - 1):
        M = cu[n + 1] - cu[n]
        path, node, token = [], 0, -1
        while M:
            path.append(node)
            row = cu[n] + node
            p = target_probabilities(logits[row], 1.0 if temperature is None else float(temperature[n]))
            if p is None:
                break
            first, accepted = p, None
            for c in range(node + 1, M):
                if parent[cu[n] + c] != node:
                    continue
                t = int(tokens[cu[n] + c])
                if not 0 <= t < len(p):
                    continue
                q = np.zeros_like(p)
                q[t] = 1.0
                if draft_probs is not None:
                    q = np.asarray(draft_probs[row], dtype=np.float64)
                if float(u_accept[cu[n] + c]) * q[t] < p[t]:
                    accepted = c
                    break
                if draft_probs is None:
                    p = np.where(q > 0, 0.0, p)
                else:
                    p = np.maximum(p - q, 0.0)
                if p.sum() <= 0:
                    p = np.zeros_like(p)
                    continue
                p = p / p.sum()
            if accepted is not None:
                node = accepted
                continue
            p = p if p.sum() > 0 else first
            cum = np.cumsum(p)
            token = int(np.searchsorted(cum, float(u_next[n]) * cum[-1], side="right"))
            break
        paths.append(path)
        following.append(token)
    return paths, following
