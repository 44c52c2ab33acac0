"""The operators of speculative serving with KDA layers: inputs, plain forms and 64-bit results of each.

A serving step drafts a small tree of tokens behind each request's last token, runs the target model once over all
trees, keeps the drafted tokens that the target's distribution accepts, and moves each request's state along the
accepted path.  Trees are packed: request n owns rows [cu_nodes[n], cu_nodes[n + 1]) of every tensor, its first row
is the tree's root (the request's last token) and parent[row] is a local index below the row's own (-1: the root).

  step    KDA attention of every node over its request's slot of the state pool (the pool is only read), with the
          nodes' write vectors u, from which the state along any path follows without a second recurrence
  commit  the slots' states moved along the accepted paths, in place
  conv    the short causal convolution along each node's path over a pool of convolution states, then those states
          moved along the accepted paths
  verify  drafted tokens accepted or rejected against the target's distribution, and the next token drawn
"""
import math
import random

import numpy as np
import torch

own = False

CONV_W = 4
EPS = 1e-6


def listed():
    return [
        # one request, a chain of four drafted tokens behind its last one: the latency of a small batch
        _step("step_chain5_n1_h16", N=1, H=16, lo=5, hi=5, shape="chain"),
        # 64 requests, small trees: an ordinary serving batch
        _step("step_tree16_n64_h32", N=64, H=32, lo=9, hi=16),
        # few requests with the largest trees
        _step("step_tree64_n16_h32", N=16, H=32, lo=33, hi=64),
        # the decode benchmark's batch with a tree behind every request: the largest
        _step("step_tree16_n256_h32", N=256, H=32, lo=9, hi=16),
        # single precision, a smaller head, an odd batch, no fused normalisation
        _step("step_fp32_d64_n17_h5", N=17, H=5, lo=1, hi=13, d=64, dtype="fp32", fused=False),
        # the accepted path of one request
        {"name": "commit_n1_h16", "op": "commit", "N": 1, "H": 16, "d": 128, "dtype": "bf16", "lo": 3, "hi": 3, "nodes": 5},
        # the accepted paths of the decode benchmark's batch, some of them empty
        {"name": "commit_n256_h32", "op": "commit", "N": 256, "H": 32, "d": 128, "dtype": "bf16", "lo": 0, "hi": 6, "nodes": 16},
        # one projection's convolution for one request
        {"name": "conv_chain5_n1_c2048", "op": "conv", "N": 1, "C": 2048, "W": CONV_W, "dtype": "bf16", "lo": 5, "hi": 5, "shape": "chain"},
        # the same for the decode benchmark's batch
        {"name": "conv_tree16_n256_c4096", "op": "conv", "N": 256, "C": 4096, "W": CONV_W, "dtype": "bf16", "lo": 9, "hi": 16, "shape": "bushy"},
        # one request's chain of sampled drafts, single-precision logits
        {"name": "verify_chain5_n1_v32768", "op": "verify", "N": 1, "V": 32768, "dtype": "fp32", "lo": 5, "hi": 5, "shape": "chain", "probs": True},
        # small trees of sampled drafts over a large vocabulary
        {"name": "verify_tree16_n64_v131072", "op": "verify", "N": 64, "V": 131072, "dtype": "bf16", "lo": 9, "hi": 16, "shape": "bushy", "probs": True},
        # chains of greedy drafts (no draft distribution), an odd vocabulary, a large batch
        {"name": "verify_chain8_n256_v100003", "op": "verify", "N": 256, "V": 100003, "dtype": "bf16", "lo": 4, "hi": 8, "shape": "chain", "probs": False},
    ]


def _step(name, N, H, lo, hi, shape="bushy", d=128, dtype="bf16", fused=True):
    return {"name": name, "op": "step", "N": N, "H": H, "d": d, "dtype": dtype, "lo": lo, "hi": hi, "shape": shape, "fused": fused}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "step", "commit", "conv", "verify", "verify"])
    N = _log_int(rng, 1, 256)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    shape = rng.choice(["chain", "bushy"])
    if op in ("step", "commit"):
        H = rng.randint(1, 32)
        d = rng.choice([128, 128, 128, 64, 16])
        if op == "commit":
            N, hi = min(N, 7000 // H), rng.randint(1, 16)
            return {"op": op, "N": N, "H": H, "d": d, "dtype": dtype, "lo": rng.randint(0, hi), "hi": hi, "nodes": _log_int(rng, hi, 64)}
        hi = _log_int(rng, 1, 64 if dtype == "bf16" else 16)
        if N * H * (16 + hi) > 256 * 32 * 32:  # no more work than the largest listed case
            N = max(1, 256 * 32 * 32 // (H * (16 + hi)))
        return {"op": op, "N": N, "H": H, "d": d, "dtype": dtype, "lo": rng.randint(1, hi), "hi": hi, "shape": shape, "fused": rng.random() < 0.7}
    hi = _log_int(rng, 1, 16)
    lo = rng.randint(1, hi)
    if op == "conv":
        return {"op": op, "N": N, "C": _log_int(rng, 64, 4096), "W": rng.choice([4, 4, 4, 2, 8]), "dtype": dtype, "lo": lo, "hi": hi, "shape": shape}
    V = _log_int(rng, 1000, 131072)
    N = max(1, min(N, (64 * 16 * 131072) // (hi * V)))
    return {"op": op, "N": N, "V": V, "dtype": dtype, "lo": lo, "hi": hi, "shape": shape, "probs": rng.random() < 0.6}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case, r):
    """From lo to hi in even steps, in random order."""
    lengths = [case["lo"] + i * (case["hi"] - case["lo"] + 1) // case["N"] for i in range(case["N"])]
    r.shuffle(lengths)
    if case["N"] == 1:
        lengths = [case["hi"]]
    return lengths


def _trees(case, seed):
    """(lengths, parents): the tree of each request; a bushy tree's node hangs from one of the four before it."""
    r = random.Random(seed * 7919 + 17)
    lengths = _lengths(case, r)
    back = 1 if case["shape"] == "chain" else 4
    return lengths, [[-1] + [i - r.randint(1, min(i, back)) for i in range(1, n)] for n in lengths]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _packed(lengths, parents, M):
    """The packed layout of the trees, and tables of the same trees padded to M nodes."""
    N, T = len(lengths), sum(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    rows, flat, anc = np.zeros((N, M), np.int64), np.zeros(T, np.int64), np.zeros((N, M, M), bool)
    for n, p in enumerate(parents):
        rows[n, :len(p)] = cu[n] + np.arange(len(p))
        flat[cu[n]:cu[n + 1]] = n * M + np.arange(len(p))
        for i, j in enumerate(p):
            if j >= 0:
                anc[n, i] = anc[n, j]
            anc[n, i, i] = True
    return {"cu": _i32(cu), "parent": _i32([j for p in parents for j in p]), "rows": torch.tensor(rows, device="cuda"),
            "flat": torch.tensor(flat, device="cuda"), "anc": torch.tensor(anc, device="cuda")}


def _slots(N, seed):
    """Distinct slots of a pool a quarter larger than the batch, in no order."""
    total = N + N // 4 + 1
    return total, _i32(random.Random(seed * 31 + 5).sample(range(total), N))


def prepare(case, seed):
    return {"step": _prepare_step, "commit": _prepare_commit, "conv": _prepare_conv, "verify": _prepare_verify}[case["op"]](case, seed)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _prepare_step(case, seed):
    H, d, dt, g = case["H"], case["d"], _dtype(case), _gen(seed)
    lengths, parents = _trees(case, seed)
    s = _packed(lengths, parents, max(lengths))
    T = sum(lengths)
    total, slots = _slots(case["N"], seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    q, k = randn(T, H, d), randn(T, H, d)
    if not case["fused"]:
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    s.update(op="step", parents=parents, fused=case["fused"], slots=slots, max_nodes=max(lengths), q=q.to(dt), k=k.to(dt), v=randn(T, H, d).to(dt),
             g=-torch.exp(0.5 * randn(T, H, d) - 1.0), beta=torch.sigmoid(randn(T, H)), S=0.1 * randn(total, H, d, d),
             z=randn(T, H, d).to(dt), weight=1.0 + 0.1 * randn(d), o=torch.empty((T, H, d), dtype=dt, device="cuda"),
             u=torch.empty((T, H, d), device="cuda"))
    return s


def _prepare_commit(case, seed):
    N, H, d, dt, g = case["N"], case["H"], case["d"], _dtype(case), _gen(seed)
    r = random.Random(seed * 7919 + 17)
    L = max(1, case["hi"])
    taken = _lengths(case, r)
    path = [([0] + sorted(r.sample(range(1, case["nodes"]), n - 1)) if n else []) + [-1] * (L - n) for n in taken]
    T = N * case["nodes"]
    total, slots = _slots(N, seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    path = torch.tensor(path, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, T + 1, case["nodes"], dtype=torch.int32, device="cuda")
    return {"op": "commit", "cu": cu, "path": path, "path_len": _i32(taken), "slots": slots, "k": randn(T, H, d).to(dt),
            "g": -torch.exp(0.5 * randn(T, H, d) - 1.0), "u": 0.5 * randn(T, H, d), "S": 0.1 * randn(total, H, d, d)}


def _prepare_conv(case, seed):
    C, W, dt, g = case["C"], case["W"], _dtype(case), _gen(seed)
    lengths, parents = _trees(case, seed)
    s = _packed(lengths, parents, max(lengths))
    T = sum(lengths)
    total, slots = _slots(case["N"], seed)
    # ancestors of each row as positions in [that request's carried inputs, oldest first; its tree's rows]
    tap, cu = np.zeros((T, W), np.int64), np.concatenate([[0], np.cumsum(lengths)])
    order = slots.tolist()
    for n, p in enumerate(parents):
        for i, j in enumerate(p):
            row = cu[n] + i
            tap[row, 0] = total * (W - 1) + row
            tap[row, 1:] = tap[cu[n] + j, :-1] if j >= 0 else order[n] * (W - 1) + np.arange(W - 2, -1, -1)
    leaf = [random.Random(seed + n).randrange(m) for n, m in enumerate(lengths)]  # the path that was accepted ends here
    path = [[i for i in range(m) if _is_above(p, i, e)] for m, p, e in zip(lengths, parents, leaf)]
    s.update(op="conv", slots=slots, max_nodes=max(lengths), tap=torch.tensor(tap, device="cuda"),
             last=torch.tensor([cu[n] + e for n, e in enumerate(leaf)], device="cuda"), path_len=_i32([len(p) for p in path]),
             path=_i32([p + [-1] * (max(lengths) - len(p)) for p in path]), x=torch.randn((T, C), generator=g, device="cuda").to(dt),
             w=0.5 * torch.randn((C, W), generator=g, device="cuda"), pool=torch.randn((total, W - 1, C), generator=g, device="cuda").to(dt).float(),
             y=torch.empty((T, C), dtype=dt, device="cuda"))
    return s


def _is_above(parent, i, leaf):
    while leaf > i:
        leaf = parent[leaf]
    return leaf == i


def _prepare_verify(case, seed):
    V, dt, g = case["V"], _dtype(case), _gen(seed)
    N = case["N"]
    lengths, parents = _trees(case, seed)
    s = _packed(lengths, parents, max(lengths))
    T, M = sum(lengths), max(lengths)
    r = random.Random(seed * 101 + 3)
    # a fifth of the requests decode greedily (temperature 0)
    temperature = torch.tensor([r.choice([0.0, 0.7, 0.9, 1.0, 1.2]) for _ in range(N)], device="cuda")
    row_temperature = torch.repeat_interleave(torch.where(temperature > 0, temperature, torch.ones(N, device="cuda")), torch.tensor(lengths, device="cuda"))
    # the draft's logits are peaked like a language model's; the target's are the draft's with an error
    draft = 3.5 * torch.randn((T, V), generator=g, device="cuda")
    logits = (draft + 0.8 * torch.randn((T, V), generator=g, device="cuda")).to(dt)
    # each node's children, in order: they are tried in this order
    children = [[[j for j in range(len(p)) if p[j] == i] for i in range(len(p))] for p in parents]
    ranks = max([1] + [len(c) for t in children for c in t])
    cu = np.concatenate([[0], np.cumsum(lengths)])
    child = np.full((T, ranks), -1, np.int64)
    rank, above = np.zeros(T, np.int64), np.zeros(T, np.int64)
    for n, t in enumerate(children):
        for i, c in enumerate(t):
            for k, j in enumerate(c):
                child[cu[n] + i, k], rank[cu[n] + j], above[cu[n] + j] = cu[n] + j, k, cu[n] + i
    above, rank = torch.tensor(above, device="cuda"), torch.tensor(rank, device="cuda")
    probs = None
    if case["probs"]:  # drafted tokens are drawn from the draft's distribution at their parent
        probs = torch.softmax(draft / row_temperature[:, None], dim=-1)
        race = torch.empty((T, V), device="cuda").exponential_(generator=g)
        tokens = (probs[above] / race).argmax(dim=-1)
    else:  # or they are the draft's most likely ones
        tokens = draft.topk(min(V, ranks), dim=-1).indices[above, rank]
    s.update(op="verify", N=N, logits=logits, probs=probs, tokens=tokens.to(torch.int32), temperature=temperature, max_nodes=M,
             u=torch.rand(T, generator=g, device="cuda"), u_next=torch.rand(N, generator=g, device="cuda"), child=torch.tensor(child, device="cuda"),
             above=above, seq=torch.repeat_interleave(torch.arange(N, device="cuda"), torch.tensor(lengths, device="cuda")),
             path=torch.empty((N, M), dtype=torch.int32, device="cuda"), path_len=torch.empty(N, dtype=torch.int32, device="cuda"),
             next_token=torch.empty(N, dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"step": _plain_step, "commit": _plain_commit, "conv": _plain_conv, "verify": _plain_verify}[s["op"]](s)


def _own(s):
    from gated_delta_rule_27_gb300 import libkda
    if s["op"] == "step":
        fusion = dict(qk_l2norm=True, qk_eps=EPS, out_gate=s["z"], out_weight=s["weight"], out_eps=EPS) if s["fused"] else {}
        libkda.kda_tree_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["parent"], s["cu"], s["slots"], s["S"], s["o"], s["u"], s["max_nodes"], **fusion)
        return {"o": s["o"], "u": s["u"]}
    if s["op"] == "commit":
        libkda.kda_tree_commit(s["k"], s["g"], s["u"], s["cu"], s["path"], s["path_len"], s["slots"], s["S"], qk_l2norm=True, qk_eps=EPS)
        return s["S"]
    if s["op"] == "conv":
        libkda.kda_tree_conv(s["x"], s["w"], s["parent"], s["cu"], s["slots"], s["pool"], s["y"], s["max_nodes"])
        libkda.kda_tree_conv_commit(s["x"], s["cu"], s["path"], s["path_len"], s["slots"], s["pool"])
        return {"y": s["y"], "pool": s["pool"]}
    libkda.kda_draft_verify(s["logits"], s["tokens"], s["parent"], s["cu"], s["u"], s["u_next"], s["path"], s["path_len"], s["next_token"],
                            draft_probs=s["probs"], temperature=s["temperature"])
    return {"path": s["path"], "path_len": s["path_len"], "next_token": s["next_token"]}


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _plain_step(s):
    pad = lambda x: x[s["rows"]].float().transpose(1, 2)  # noqa: E731  [N, H, M, ...]
    q, k, v, g, beta = (pad(s[x]) for x in ("q", "k", "v", "g", "beta"))
    if s["fused"]:
        q, k = _unit(q), _unit(k)
    anc = s["anc"][:, None]
    b = torch.matmul(anc.float(), g)  # log-decay from the pool's state to each node
    ke, qe, ki = k * torch.exp(b), q * torch.exp(b), (k * torch.exp(-b)).transpose(-1, -2)
    eye = torch.eye(anc.shape[-1], device="cuda", dtype=torch.bool)
    zero = torch.zeros((), device="cuda")
    A = torch.where(anc & ~eye, torch.matmul(ke, ki) * beta[..., None], zero)
    P = torch.where(anc, torch.matmul(qe, ki), zero)
    S = s["S"][s["slots"].long()]
    R = beta[..., None] * (v - torch.matmul(ke, S))
    # (I + A)^-1 R with A^64 = 0: (I - A)(I + A^2)(I + A^4) ... (I + A^32) R
    A2 = A @ A
    A4 = A2 @ A2
    A8 = A4 @ A4
    A16 = A8 @ A8
    U = R + (A16 @ A16) @ R
    U = U + A16 @ U
    U = U + A8 @ U
    U = U + A4 @ U
    U = U + A2 @ U
    U = U - A @ U
    o = torch.matmul(qe, S) + torch.matmul(P, U)
    unpad = lambda x: x.transpose(1, 2).flatten(0, 1)[s["flat"]]  # noqa: E731
    o = unpad(o)
    if s["fused"]:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"] * torch.sigmoid(s["z"].float())
    return {"o": o.to(s["o"].dtype), "u": unpad(U).contiguous()}


def _plain_commit(s):
    slots = s["slots"].long()
    on = (s["path"] >= 0)[..., None, None]
    rows = (s["cu"][:-1, None] + s["path"].clamp_min(0)).long()
    g = torch.where(on, s["g"][rows], torch.zeros((), device="cuda"))
    b = torch.cumsum(g, 1)
    end = b[:, -1:]
    k = torch.where(on, _unit(s["k"][rows].float()) * torch.exp(end - b), torch.zeros((), device="cuda"))
    S = torch.exp(end[:, 0])[..., None] * s["S"][slots] + torch.matmul(k.permute(0, 2, 3, 1), s["u"][rows].transpose(1, 2))
    s["S"][slots] = S
    return s["S"]


def _plain_conv(s):
    C, W = s["w"].shape
    rows = torch.cat([s["pool"].reshape(-1, C), s["x"].float()])
    y = (rows[s["tap"]] * s["w"].t()).sum(1).to(s["y"].dtype)
    if W > 1:  # the last W - 1 inputs of the path, oldest first
        s["pool"][s["slots"].long()] = rows[s["tap"][s["last"]][:, :W - 1].flip(1)]
    return {"y": y, "pool": s["pool"]}


FIXED = float(2 ** 40)  # sums over the vocabulary count steps of 2^-40, so that they depend on no order


def _fixed(x):
    return (x * FIXED).to(torch.int64)


def _plain_verify(s):
    N, T, M = s["N"], s["logits"].shape[0], s["max_nodes"]
    row, zero = torch.arange(T, device="cuda"), torch.zeros((), device="cuda")
    temperature = s["temperature"][s["seq"]]
    l = s["logits"].float()
    top, place = l.max(-1, keepdim=True).values, torch.arange(l.shape[1], device="cuda")
    best = torch.where(l == top, place, l.shape[1]).min(-1, keepdim=True).values  # ties: the lowest
    scale = 1.4426950408889634 / temperature.clamp_min(1e-30)
    w = torch.where((temperature > 0)[:, None], torch.exp2((l - top) * scale[:, None]), (place == best).float())
    # every row's children are tried in order: what is left of the row's weight after each rejection, and its sum
    left, took, done = w, torch.full((T,), -1, device="cuda"), torch.zeros(T, dtype=torch.bool, device="cuda")
    coef = torch.zeros(T, device="cuda")
    for k in range(s["child"].shape[1]):
        total = _fixed(left).sum(-1).float() / FIXED
        c = s["child"][:, k]
        there = (c >= 0) & ~done
        token = s["tokens"][c.clamp_min(0)].long()
        q = s["probs"][row, token] if s["probs"] is not None else torch.ones(T, device="cuda")
        accept = there & (s["u"][c.clamp_min(0)] * q * total < left[row, token])
        took, done, there = torch.where(accept, c, took), done | accept, there & ~accept
        if s["probs"] is not None:
            coef = torch.where(there, coef + total, coef)
            left = torch.where(there[:, None], (w - coef[:, None] * s["probs"]).clamp_min(0), left)
        else:
            left = left.index_put((row, token), torch.where(there, zero, left[row, token]))
    # a node is on the path if it and all above it were taken by their parents
    taken = took[s["above"]] == row
    taken[s["cu"][:-1].long()] = True
    on = torch.zeros(N * M, dtype=torch.bool, device="cuda").index_put((s["flat"],), taken).view(N, M)
    on = (s["anc"].sum(-1) > 0) & ((s["anc"] & ~on[:, None]).sum(-1) == 0)
    length = on.sum(-1)
    place = torch.where(on, torch.arange(M, device="cuda"), M).sort(-1).values
    path = torch.where(place < M, place, -1)
    last = s["rows"][torch.arange(N, device="cuda"), path.gather(1, (length - 1)[:, None])[:, 0]]
    f = _fixed(left[last])
    f = torch.where(f.sum(-1, keepdim=True) > 0, f, _fixed(w[last]))  # nothing is left: the target's own
    cum = f.cumsum(-1)
    at = (s["u_next"].double() * cum[:, -1].double()).to(torch.int64)
    token = (cum <= at[:, None]).sum(-1)
    return {"path": path.to(torch.int32), "path_len": length.to(torch.int32), "next_token": token.to(torch.int32)}


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    N = case["N"]
    el = 2 if case["dtype"] == "bf16" else 4
    mean = 0.5 * (case["lo"] + case["hi"])
    if case["op"] == "step":  # the state once; q, k, v, o (and the gate), g and u per node
        H, d = case["H"], case["d"]
        nodes = N * H * mean
        return {"bytes": N * H * d * d * 4 + nodes * (d * el * (5 if case["fused"] else 4) + d * 8 + 4),
                "flops": nodes * (4 * d * d + 2 * mean * d * 2)}
    if case["op"] == "commit":  # the state once each way; k, g and u per node of the path
        H, d = case["H"], case["d"]
        return {"bytes": N * H * (2 * d * d * 4 + mean * d * (el + 8)), "flops": N * H * d * d * (1 + 2 * mean)}
    if case["op"] == "conv":  # every input and output once, the carried inputs once each way
        C, W = case["C"], case["W"]
        return {"bytes": N * C * (mean * 2 * el + 2 * (W - 1) * 4) + C * W * 4, "flops": N * C * mean * 2 * W}
    # the rows that the walk visits (about three in four first tries are accepted) and the last one's draft row
    depth = mean - 1 if case["shape"] == "chain" else (mean - 1) / 2.5
    visited = (1 - 0.75 ** (depth + 1)) / 0.25
    return {"bytes": N * case["V"] * (visited * el + (4 if case["probs"] else 0)), "flops": N * case["V"] * visited * 3}


# ---------------------------------------------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "verify":  # whole numbers only
        return None
    return {"step": _exact_step, "commit": _exact_commit, "conv": _exact_conv}[case["op"]](case, prepare(case, seed))


def _exact_rows(s, name, heads):
    x = s[name][:, heads].double()
    if name in ("q", "k") and s.get("fused", True):
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)
    return x


def _exact_step(case, s):
    """Node by node, each from its parent's state: S = D S' + k u^T, u = beta (v - (D S')^T k), o = S^T q."""
    parents = s["parents"]
    N, H, d, M = case["N"], case["H"], case["d"], max(len(p) for p in parents)
    cu = s["cu"].tolist()
    o = torch.zeros((s["q"].shape[0], H, d), dtype=torch.float64, device="cuda")
    u = torch.zeros_like(o)
    some = max(1, int(4e9 // (N * M * d * d * 8)))
    for h in range(0, H, some):
        heads = slice(h, min(H, h + some))
        q, k, v, g, beta = (_exact_rows(s, x, heads) for x in ("q", "k", "v", "g", "beta"))
        root = s["S"][s["slots"].long()][:, heads].double()
        tree = torch.zeros((M, N, q.shape[1], d, d), dtype=torch.float64, device="cuda")
        for i in range(M):
            at = [n for n in range(N) if len(parents[n]) > i]
            rows = torch.tensor([cu[n] + i for n in at], device="cuda")
            n = torch.tensor(at, device="cuda")
            S = root[n] if i == 0 else tree[torch.tensor([parents[m][i] for m in at], device="cuda"), n]
            S = torch.exp(g[rows])[..., None] * S
            err = beta[rows][..., None] * (v[rows] - (S * k[rows][..., None]).sum(-2))
            S = S + k[rows][..., None] * err[..., None, :]
            tree[i, n] = S
            u[rows, heads], o[rows, heads] = err, (S * q[rows][..., None]).sum(-2)
    if s["fused"]:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"].double() / (1 + torch.exp(-s["z"].double()))
    return {"o": o, "u": u}


def _exact_commit(case, s):
    """Token by token along each path: S = D S + k u^T."""
    S, path, cu, slots = s["S"].double(), s["path"].tolist(), s["cu"].tolist(), s["slots"].tolist()
    k, g, u = _exact_rows(s, "k", slice(None)), s["g"].double(), s["u"].double()
    for n, nodes in enumerate(path):
        for i in nodes:
            if i >= 0:
                r = cu[n] + i
                S[slots[n]] = torch.exp(g[r])[..., None] * S[slots[n]] + k[r][..., None] * u[r][..., None, :]
    return S


def _exact_conv(case, s):
    """Each node's inputs are found by going up its tree and then back through the carried inputs."""
    x, w, pool, W = s["x"].double(), s["w"].double(), s["pool"].double(), case["W"]
    cu, parent, slots, path = s["cu"].tolist(), s["parent"].tolist(), s["slots"].tolist(), s["path"].tolist()
    y = torch.zeros_like(x)
    end = pool.clone()
    for n, slot in enumerate(slots):
        for r in range(cu[n], cu[n + 1]):
            at, carried = r - cu[n], W - 2
            for j in range(W):
                if at >= 0:
                    y[r] += w[:, j] * x[cu[n] + at]
                    at = parent[cu[n] + at]
                else:
                    y[r] += w[:, j] * pool[slot, carried]
                    carried -= 1
        if W > 1:
            whole = torch.cat([pool[slot], x[[cu[n] + i for i in path[n] if i >= 0]]])
            end[slot] = whole[len(whole) - (W - 1):]
    return {"y": y, "pool": end}
