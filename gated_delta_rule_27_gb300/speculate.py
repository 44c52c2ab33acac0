"""Speculative serving with the KDA sublayer: draft trees, one pass of the model over them, verification, commit.

A round for a batch of requests, whose recurrent and convolution states live in pools:

  1. the draft proposes a small tree of tokens behind each request's last token;
  2. ``tree_forward`` runs the sublayer over every node of every tree, reading the pools and leaving them alone;
  3. ``libkda.kda_draft_verify`` keeps the path that the target's distribution accepts and draws the next token;
  4. ``tree_commit`` moves the pools along the kept paths.  A rejected node has changed nothing, so there is no
     rollback (Lecture 11, section 2, "Serving state" row).

``Model`` is the smallest model that can be run that way: an embedding, one sublayer with its residual, and a head,
with random weights; its draft is the same without the sublayer.  ``python -m gated_delta_rule_27_gb300.speculate``
generates with it.
"""
from __future__ import annotations

import dataclasses

import torch

from . import libkda, sublayer
from .sublayer import CONV_W


@dataclasses.dataclass
class Trees:
    """Packed draft trees (include/kda.h): request n owns rows [cu_nodes[n], cu_nodes[n + 1])."""
    parent: torch.Tensor    # [T] int32, local indices, -1 for a root
    cu_nodes: torch.Tensor  # [N + 1] int32
    seq_idx: torch.Tensor   # [N] int32 pool slots
    max_nodes: int


class Pools:
    """The states of `slots` requests: S [slots, H, d, d] and the carried inputs of the three convolutions."""

    def __init__(self, slots: int, H: int, d: int, device):
        self.S = torch.zeros((slots, H, d, d), dtype=torch.float32, device=device)
        self.conv = [torch.zeros((slots, CONV_W - 1, H * d), dtype=torch.float32, device=device) for _ in range(3)]


class TreeBuffers(sublayer.Buffers):
    """Every intermediate of one pass over trees with T nodes in all."""

    def __init__(self, T: int, H: int, d: int, device):
        super().__init__(T, 0, H, d, device)
        self.u = torch.empty((T, H, d), dtype=torch.float32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)


def tree_forward(x, trees: Trees, pools: Pools, w: sublayer.Weights, H: int, d: int, bufs: TreeBuffers, eps=1e-6):
    """The sublayer over every node: x [T, D] bf16 -> y [T, D].  The pools are only read."""
    T = x.shape[0]
    sublayer._project(x, w, bufs)
    for src, cw, pool, dst in ((bufs.q, w.conv_q, pools.conv[0], bufs.qc), (bufs.k, w.conv_k, pools.conv[1], bufs.kc),
                               (bufs.v, w.conv_v, pools.conv[2], bufs.vc)):
        libkda.kda_tree_conv(src, cw, trees.parent, trees.cu_nodes, trees.seq_idx, pool, dst, trees.max_nodes,
                             status=bufs.status)
    heads = lambda t: t.view(T, H, d)
    libkda.kda_tree_step(heads(bufs.qc), heads(bufs.kc), heads(bufs.vc), heads(bufs.g), bufs.beta, trees.parent,
                         trees.cu_nodes, trees.seq_idx, pools.S, bufs.o, bufs.u, trees.max_nodes, status=bufs.status,
                         qk_l2norm=True, qk_eps=eps, out_gate=heads(bufs.z), out_weight=w.out_weight, out_eps=eps)
    return bufs.o.view(T, H * d) @ w.W_o


def tree_commit(trees: Trees, path, path_len, pools: Pools, H: int, d: int, bufs: TreeBuffers, eps=1e-6) -> None:
    """Moves the pools along the kept paths, from what tree_forward left in `bufs`."""
    T = bufs.q.shape[0]
    for src, pool in zip((bufs.q, bufs.k, bufs.v), pools.conv):
        libkda.kda_tree_conv_commit(src, trees.cu_nodes, path, path_len, trees.seq_idx, pool, status=bufs.status)
    libkda.kda_tree_commit(bufs.kc.view(T, H, d), bufs.g.view(T, H, d), bufs.u, trees.cu_nodes, path, path_len,
                           trees.seq_idx, pools.S, status=bufs.status, qk_l2norm=True, qk_eps=eps)


@dataclasses.dataclass
class Model:
    embed: torch.Tensor   # [V, D] bf16
    head: torch.Tensor    # [D, V] bf16
    weights: sublayer.Weights
    H: int
    d: int

    @classmethod
    def random(cls, V: int, H: int, d: int, seed: int, device, sharpness: float = 3.0):
        D = H * d
        gen = torch.Generator().manual_seed(seed)
        mat = lambda *s, scale=1.0: (scale * torch.randn(s, generator=gen)).to(torch.bfloat16).to(device)
        return cls(mat(V, D), mat(D, V, scale=sharpness / D ** 0.5), sublayer.synthetic_weights(D, H, d, seed + 1, device),
                   H, d)

    def draft_logits(self, tokens):
        return self.embed[tokens.long()] @ self.head

    def target_logits(self, tokens, y):
        return (self.embed[tokens.long()] + y) @ self.head


def draft_trees(model: Model, last, shape, temperature, gen):
    """Tokens [N, len(shape)] of one tree per request, drawn node by node from the draft, and the draft's
    distributions [N, len(shape), V]; `shape` is the tree's parent list, `last` the requests' last tokens."""
    N, M = last.numel(), len(shape)
    tokens = torch.zeros((N, M), dtype=torch.int32, device=last.device)
    probs = []
    tokens[:, 0] = last
    for i in range(M):
        probs.append(torch.softmax(model.draft_logits(tokens[:, i]).float() / max(temperature, 0.1), -1))
        for j in range(i + 1, M):
            if shape[j] == i:
                tokens[:, j] = torch.multinomial(probs[i], 1, generator=gen)[:, 0].to(torch.int32)
    return tokens, torch.stack(probs, 1)


def generate(model: Model, last, slots, pools: Pools, rounds: int, shape=(-1, 0, 0, 1, 1, 2, 3), temperature=1.0, seed=0):
    """`rounds` speculative rounds for requests with last tokens `last` [N] and pool slots `slots` [N]; returns each
    request's new tokens and the mean number of tokens per request and round."""
    device, N, M, H, d = last.device, last.numel(), len(shape), model.H, model.d
    gen = torch.Generator(device=device).manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
    trees = Trees(i32(list(shape) * N), i32([n * M for n in range(N + 1)]), slots, M)
    bufs = TreeBuffers(N * M, H, d, device)
    path, path_len, next_token = i32([[0] * M] * N).view(N, M), i32([0] * N), last.clone()
    heat = torch.full((N,), float(temperature), device=device)
    new = [[] for _ in range(N)]
    for _ in range(rounds):
        tokens, probs = draft_trees(model, next_token, shape, temperature, gen)
        flat = tokens.view(-1)
        y = tree_forward(model.embed[flat.long()], trees, pools, model.weights, H, d, bufs)
        libkda.kda_draft_verify(model.target_logits(flat, y), flat, trees.parent, trees.cu_nodes,
                                torch.rand(N * M, generator=gen, device=device), torch.rand(N, generator=gen, device=device),
                                path, path_len, next_token, draft_probs=probs.flatten(0, 1), temperature=heat,
                                status=bufs.status)
        tree_commit(trees, path, path_len, pools, H, d, bufs)
        kept, lengths, drawn = path.tolist(), path_len.tolist(), next_token.tolist()
        for n, token in enumerate(drawn):
            if token < 0:  # and a round on top of it would embed row -1
                raise ValueError("request %d: no token to go on with; its last node has no logit above -inf" % n)
        for n, row in enumerate(tokens.tolist()):
            new[n] += [row[i] for i in kept[n][1:lengths[n]]] + [drawn[n]]
    if int(bufs.status):
        raise libkda.KdaError(int(bufs.status), "a speculative round")
    return new, sum(map(len, new)) / max(1, N * rounds)


if __name__ == "__main__":
    dev = torch.device("cuda")
    m = Model.random(V=4096, H=4, d=128, seed=1, device=dev)
    pools_ = Pools(12, m.H, m.d, dev)
    start = torch.arange(8, dtype=torch.int32, device=dev)
    for T_ in (0.0, 1.0):
        out, rate = generate(m, start, start + 3, pools_, rounds=16, temperature=T_)
        print("temperature %.1f: %.2f tokens per request and round; request 0: %s" % (T_, rate, out[0][:12]))
