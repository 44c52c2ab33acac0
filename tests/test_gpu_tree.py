"""The draft-tree operators against fp64 references.

Tolerances (fixed before measuring), max|x - ref| / max|ref|: 1e-4 for fp32 values (u, states, fp32 outputs), which
leaves the fp32 sums of up to 64 path nodes and 128 channels an order of magnitude; 2e-2 for bf16 outputs.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from oracle import oracle, sublayer, tree
from tests.gpu_helpers import f64, rel

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 1e-4, torch.bfloat16: 2e-2}
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_trees(lengths, seed, back=4):
    r = np.random.default_rng(seed)
    parent = [p for n in lengths for p in [-1] + [int(i - r.integers(1, min(i, back) + 1)) for i in range(1, n)] if n]
    return parent, np.concatenate([[0], np.cumsum(lengths)]).astype(int).tolist()


def step_inputs(lengths, H, d, dtype, seed, back=4, extreme=False):
    parent, cu = make_trees(lengths, seed, back)
    T, N = cu[-1], len(lengths)
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g)
    q, k = (torch.nn.functional.normalize(randn(T, H, d), dim=-1).to(dtype) for _ in range(2))
    decay = -torch.exp(0.5 * randn(T, H, d) - 1.0)
    beta = torch.sigmoid(randn(T, H))
    if extreme:  # gates that leave nothing or everything, write strengths of zero and one
        decay = torch.where(torch.rand((T, H, d), generator=g) < 0.5, torch.tensor(-10.0), torch.tensor(-1e-4))
        beta = torch.randint(0, 2, (T, H), generator=g).float()
    slots = torch.randperm(N + 3, generator=g)[:N].tolist()
    return dict(q=q, k=k, v=randn(T, H, d).to(dtype), g=decay, beta=beta, parent=parent, cu=cu, slots=slots,
                pool=0.1 * randn(N + 3, H, d, d), z=randn(T, H, d).to(dtype), weight=1 + 0.1 * randn(d))


def run_step(x, max_nodes, with_u=True, **fusion):
    q = x["q"].cuda()
    o = torch.full_like(q, float("nan"))
    u = torch.full(q.shape, float("nan"), device="cuda") if with_u else None
    pool = x["pool"].cuda()
    status = i32([0])
    libkda.kda_tree_step(q, x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), x["beta"].cuda(), i32(x["parent"]), i32(x["cu"]),
                         i32(x["slots"]), pool, o, u, max_nodes, status=status, **fusion)
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(pool.cpu(), x["pool"])
    return o, u, pool


SHAPES = [([1], 1, 1), ([5], 3, 5), ([0, 4, 0, 1], 2, 4), ([16, 1, 9], 2, 16), ([17, 31, 33], 1, 40), ([64, 63], 2, 64),
          ([8] * 40, 1, 8)]


@pytest.mark.parametrize("d,dtype", [(16, F32), (16, BF), (64, F32), (64, BF), (128, F32), (128, BF)])
@pytest.mark.parametrize("lengths,H,max_nodes", SHAPES)
def test_step_and_commit(lengths, H, max_nodes, d, dtype):
    x = step_inputs(lengths, H, d, dtype, seed=sum(lengths) + d, back=1 if len(lengths) == 40 else 4)
    o, u, pool = run_step(x, max_nodes)
    o_ref, u_ref, states = tree.tree_step(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta")), x["parent"], x["cu"],
                                          x["slots"], f64(x["pool"]))
    assert rel(o, o_ref) <= TOL[dtype] and rel(u, u_ref) <= 1e-4
    # the path to the last node of each tree (the empty one to none)
    path = np.full((len(lengths), max_nodes), -1)
    want, taken = f64(x["pool"]).copy(), []
    for n, m in enumerate(lengths):
        nodes, at = [], m - 1
        while at >= 0:
            nodes.append(at)
            at = x["parent"][x["cu"][n] + at]
        path[n, :len(nodes)] = nodes[::-1]
        taken.append(len(nodes))
        if m:
            want[x["slots"][n]] = states[x["cu"][n] + m - 1]
    status = i32([0])
    libkda.kda_tree_commit(x["k"].cuda(), x["g"].cuda(), u, i32(x["cu"]), i32(path), i32(taken), i32(x["slots"]), pool,
                           status=status)
    assert int(status) == 0 and rel(pool, want) <= 1e-4
    others = [s for s in range(pool.shape[0]) if s not in [x["slots"][n] for n, m in enumerate(lengths) if m]]
    assert torch.equal(pool.cpu()[others], x["pool"][others])


@pytest.mark.parametrize("d,dtype", [(16, F32), (64, F32), (128, F32), (128, BF)])
def test_step_with_fused_norms(d, dtype):
    x = step_inputs([3, 0, 20, 64, 1], 2, d, dtype, seed=d)
    x["q"], x["k"] = (3 * x["q"].float()).to(dtype), (0.2 * x["k"].float()).to(dtype)
    o, u, pool = run_step(x, 64, qk_l2norm=True, qk_eps=1e-6, out_gate=x["z"].cuda(), out_weight=x["weight"].cuda(), out_eps=1e-5)
    q, k = (sublayer.l2norm(f64(x[n]), 1e-6) for n in "qk")
    o_ref, u_ref, states = tree.tree_step(q, k, *(f64(x[n]) for n in ("v", "g", "beta")), x["parent"], x["cu"], x["slots"], f64(x["pool"]))
    assert rel(u, u_ref) <= 1e-4
    assert rel(o, sublayer.gated_rmsnorm(o_ref, f64(x["z"]), f64(x["weight"]), 1e-5)) <= TOL[dtype]
    path, want = np.full((5, 64), -1), f64(x["pool"]).copy()
    path[:, 0] = 0
    for n in (0, 2, 3, 4):
        want[x["slots"][n]] = states[x["cu"][n]]
    libkda.kda_tree_commit(x["k"].cuda(), x["g"].cuda(), u, i32(x["cu"]), i32(path), i32([1, 0, 1, 1, 1]), i32(x["slots"]), pool,
                           qk_l2norm=True, qk_eps=1e-6)
    assert rel(pool, want) <= 1e-4


@pytest.mark.parametrize("d,dtype", [(16, F32), (128, F32), (128, BF)])
@pytest.mark.parametrize("back", [1, 4])
def test_extreme_gates(d, dtype, back):
    x = step_inputs([64, 12], 2, d, dtype, seed=5 + back, back=back, extreme=True)
    o, u, _ = run_step(x, 64)
    o_ref, u_ref, _ = tree.tree_step(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta")), x["parent"], x["cu"], x["slots"], f64(x["pool"]))
    assert rel(o, o_ref) <= TOL[dtype] and rel(u, u_ref) <= 1e-4


@pytest.mark.parametrize("d,dtype", [(16, F32), (128, F32), (128, BF)])
def test_a_decay_of_minus_infinity_forgets(d, dtype):
    """A log-decay of -inf clears its channels: what is above it on the path is gone, nothing becomes NaN."""
    x = step_inputs([20, 40], 1, d, dtype, seed=3)
    x["g"][torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(1)) < 0.1] = -float("inf")
    o, u, pool = run_step(x, 64)
    o_ref, u_ref, states = tree.tree_step(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta")), x["parent"], x["cu"], x["slots"], f64(x["pool"]))
    assert rel(o, o_ref) <= TOL[dtype] and rel(u, u_ref) <= 1e-4
    path, want = [[0] + [i for i in range(1, 20) if _above(x["parent"], i, 19)] + [-1] * 19, [-1] * 20], f64(x["pool"]).copy()
    taken = sum(i >= 0 for i in path[0])
    want[x["slots"][0]] = states[19]
    libkda.kda_tree_commit(x["k"].cuda(), x["g"].cuda(), u, i32(x["cu"]), i32([path[0][:20], path[1]]), i32([taken, 0]), i32(x["slots"]), pool)
    assert rel(pool, want) <= 1e-4


def _above(parent, i, leaf):
    while leaf > i:
        leaf = parent[leaf]
    return leaf == i


@pytest.mark.parametrize("d,dtype", [(64, F32), (128, F32), (128, BF)])
@pytest.mark.parametrize("M", [12, 30, 60])
def test_a_bad_node_only_reaches_its_descendants(M, d, dtype):
    """NaN or infinite values of one node leave every node that is not below it untouched."""
    clean = step_inputs([M], 2, d, dtype, seed=M)
    # a node with some of the later ones below it, and some not
    bad = next(b for b in range(1, M) if 1 < sum(_above(clean["parent"], b, i) for i in range(M)) < M - b)
    below = [_above(clean["parent"], bad, i) for i in range(M)]
    want = run_step(clean, M)[:2]
    for name, value in (("v", float("nan")), ("v", float("inf")), ("k", float("nan")), ("q", float("nan")), ("g", float("nan")), ("beta", float("inf"))):
        x = dict(clean, **{name: clean[name].clone()})
        x[name][bad, 1] = value
        for got, ref in zip(run_step(x, M)[:2], want):
            keep = [i for i in range(M) if not below[i]]
            assert torch.equal(got[:, 0], ref[:, 0])
            assert rel(got[keep], f64(ref[keep])) <= TOL[got.dtype]
    assert not torch.isfinite(run_step(dict(clean, v=torch.where(torch.arange(M)[:, None, None] == bad, float("nan"), clean["v"].float()).to(dtype)), M)[0][bad]).any()


@pytest.mark.parametrize("d,dtype", [(64, F32), (128, BF)])
def test_step_is_independent_of_the_batch_and_of_u(d, dtype):
    """A request alone, without u and under a larger bound gives the bits it gives in a batch."""
    x = step_inputs([7, 16, 3], 2, d, dtype, seed=9)
    o, u, _ = run_step(x, 16)
    one = dict(x, cu=[0, 16], slots=[x["slots"][1]], parent=x["parent"][7:23], **{n: x[n][7:23] for n in ("q", "k", "v", "g", "beta")})
    alone, _, _ = run_step(one, 16, with_u=False)
    assert torch.equal(alone, o[7:23])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("C", [1, 130, 2048])
def test_conv(C, W, dtype):
    lengths = [1, 9, 0, 64]
    parent, cu = make_trees(lengths, W)
    g = torch.Generator().manual_seed(C + W)
    x, w = torch.randn((cu[-1], C), generator=g).to(dtype), torch.randn((C, W), generator=g)
    pool, slots = torch.randn((6, W - 1, C), generator=g), [5, 0, 3, 2]
    y, dpool, status = torch.empty((cu[-1], C), dtype=dtype, device="cuda"), pool.cuda(), i32([0])
    libkda.kda_tree_conv(x.cuda(), w.cuda(), i32(parent), i32(cu), i32(slots), dpool, y, 64, status=status)
    assert int(status) == 0 and torch.equal(dpool.cpu(), pool)
    assert rel(y, tree.tree_conv(f64(x), f64(w), parent, cu, slots, f64(pool))) <= TOL[dtype]
    leaf, path, want, taken = [0, 6, -1, 40], np.full((4, 64), -1), pool.clone(), []
    for n, at in enumerate(leaf):
        nodes, end = [], at
        while at >= 0:
            nodes.append(at)
            at = parent[cu[n] + at]
        path[n, :len(nodes)] = nodes[::-1]
        taken.append(len(nodes))
        if W > 1:
            seq = tree.path_inputs(f64(x), parent, cu[n], end, f64(pool[slots[n]]))
            want[slots[n]] = torch.tensor(seq[len(seq) - (W - 1):]).float()
    libkda.kda_tree_conv_commit(x.cuda(), i32(cu), i32(path), i32(taken), i32(slots), dpool, status=status)
    assert int(status) == 0 and torch.equal(dpool.cpu(), want)  # inputs are only moved


def verify_inputs(lengths, V, dtype, seed, probs, back=4, temperature=None):
    parent, cu = make_trees(lengths, seed, back)
    g = torch.Generator().manual_seed(seed)
    T, N = cu[-1], len(lengths)
    draft = 2.5 * torch.randn((T, V), generator=g)
    logits = (draft + 0.8 * torch.randn((T, V), generator=g)).to(dtype)
    q = torch.softmax(draft, -1)
    above = torch.tensor([cu[n] + max(0, parent[r]) for n in range(N) for r in range(cu[n], cu[n + 1])], dtype=torch.long)
    tokens = torch.multinomial(q[above], 1, generator=g)[:, 0] if T else torch.zeros(0, dtype=torch.long)
    return dict(logits=logits, tokens=tokens.tolist(), parent=parent, cu=cu, u=torch.rand(T, generator=g),
                u_next=torch.rand(N, generator=g), probs=q if probs else None, temperature=temperature)


def run_verify(x, M):
    N = len(x["cu"]) - 1
    path, length, token, status = (torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((N, M), (N,), (N,), (1,)))
    status.zero_()
    cuda = lambda t: None if t is None else t.cuda()
    libkda.kda_draft_verify(x["logits"].cuda(), i32(x["tokens"]), i32(x["parent"]), i32(x["cu"]), x["u"].cuda(), x["u_next"].cuda(),
                            path, length, token, draft_probs=cuda(x["probs"]), temperature=cuda(x["temperature"]), status=status)
    torch.cuda.synchronize()
    return path.tolist(), length.tolist(), token.tolist(), int(status)


def check_verify(x, M, status=0):
    paths, following = tree.draft_verify(x["logits"].float().numpy(), x["tokens"], x["parent"], x["cu"], x["u"].numpy(),
                                         x["u_next"].numpy(), None if x["probs"] is None else x["probs"].numpy(), x["temperature"])
    path, length, token, got = run_verify(x, M)
    assert got == status and length == [len(p) for p in paths]
    assert path == [p + [-1] * (M - len(p)) for p in paths]
    assert token == following
    return paths


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("V", [1, 2, 37, 1000, 4099, 50001, 200003])
def test_verify(V, probs, dtype):
    lengths = [1, 8, 0, 16] * (8 if V <= 5000 else 2)
    temperature = torch.tensor([1.0, 0.7, 1.3, 0.0] * (len(lengths) // 4))
    check_verify(verify_inputs(lengths, V, dtype, V + probs, probs, temperature=temperature.roll(V)), 16)


@pytest.mark.parametrize("probs", [True, False])
def test_verify_long_chains_and_wide_trees(probs):
    for back in (1, 63):
        x = verify_inputs([64, 40, 64], 300, BF, back, probs, back=back)
        x["u"] *= 0.3  # more is accepted
        paths = check_verify(x, 64)
        assert not probs or max(len(p) for p in paths) > 2


def test_verify_accepts_a_whole_chain():
    """Greedy drafts that the target agrees with: all 64 nodes are kept, and the last row gives the next token."""
    x = verify_inputs([64, 3], 300, BF, 2, False, back=1, temperature=torch.tensor([0.0, 0.0]))
    best = x["logits"].float().argmax(-1).tolist()
    x["tokens"] = [0] + best[:63] + [0] + best[64:66]
    assert [len(p) for p in check_verify(x, 64)] == [64, 3]


def test_verify_odd_rows():
    """Rows without a distribution, infinities, NaN, ties, equal distributions, tokens outside the vocabulary."""
    V, inf, nan = 70, float("inf"), float("nan")
    x = verify_inputs([2] * 8, V, F32, 3, True)
    l = x["logits"]
    l[0] = -inf                      # no distribution: the root alone, no next token
    l[2] = nan
    l[4] = -inf; l[4, 11] = 1.0      # one token has all of it
    l[6, 5] = inf; l[6, 60] = inf    # infinities share it
    l[8, ::2] = nan                  # masked places weigh nothing
    l[10, 1:] = -inf
    x["probs"][12] = torch.softmax(l[12], -1)  # p = q: nothing is left but rounding, if anything is rejected
    x["tokens"][15] = V              # not a token
    x["u"][13] = 0.999
    check_verify(x, 2, status=libkda.KDA_ERR_INVALID_ARG)
    for token in (-1, V):
        x["tokens"][15] = token
        x["probs"] = None
        check_verify(x, 2, status=libkda.KDA_ERR_INVALID_ARG)
    tie = verify_inputs([1, 2], V, BF, 4, False, temperature=torch.tensor([0.0, 0.0]))
    tie["logits"][:] = 0.0
    tie["logits"][:, [9, 33]] = 2.0  # greedy ties go to the lowest index
    tie["tokens"][2] = 33
    assert run_verify(tie, 2)[1:3] == ([1, 1], [9, 9])
    edge = verify_inputs([1] * 4, V, F32, 5, False)
    edge["u_next"] = torch.tensor([0.0, 1.0, -1.0, nan])  # numbers outside [0, 1) are taken to its ends
    edge["logits"][:] = 0.0
    assert run_verify(edge, 1)[2] == [0, V - 1, 0, 0]


def test_verify_keeps_the_target_distribution():
    """With siblings drawn from q, the first kept token is distributed as p (chi-square, 11 degrees of freedom: above
    50 with a probability of 6e-7)."""
    V, N = 12, 200000
    g = torch.Generator().manual_seed(0)
    lp, lq = torch.randn(V, generator=g), torch.randn(V, generator=g)
    p, q = torch.softmax(lp, -1), torch.softmax(lq, -1)
    tokens = torch.multinomial(q, 4 * N, replacement=True, generator=g)
    x = dict(logits=lp.repeat(4 * N, 1), tokens=tokens.tolist(), parent=[-1, 0, 0, 0] * N, cu=list(range(0, 4 * N + 1, 4)),
             u=torch.rand(4 * N, generator=g), u_next=torch.rand(N, generator=g), probs=q.repeat(4 * N, 1), temperature=None)
    path, length, token, status = run_verify(x, 4)
    path, token, length = torch.tensor(path), torch.tensor(token), torch.tensor(length)
    kept = torch.where(length > 1, tokens[torch.arange(N) * 4 + path[:, 1].clamp_min(0)], token)
    expected = p.double() * N
    chi2 = ((torch.bincount(kept, minlength=V).double() - expected) ** 2 / expected).sum()
    assert status == 0 and 0.5 < (length > 1).double().mean() < 0.99 and chi2 < 50


def test_invalid_requests_are_skipped():
    """Broken trees, slots and paths are reported and change nothing; the others are served."""
    x = step_inputs([4, 4, 4, 4], 1, 128, BF, 11)
    x["parent"][5] = 1               # request 1: its own parent
    x["slots"][2] = 7                # request 2: outside the pool
    q = x["q"].cuda()
    o, u, status, pool = torch.zeros_like(q), torch.zeros(q.shape, device="cuda"), i32([0]), x["pool"].cuda()
    args = [q, x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), x["beta"].cuda(), i32(x["parent"])]
    libkda.kda_tree_step(*args, i32(x["cu"]), i32(x["slots"]), pool, o, u, 4, status=status)
    assert int(status) == libkda.KDA_ERR_INVALID_ARG
    assert not o[4:12].any() and not u[4:12].any() and bool(o[:4].any()) and bool(o[12:].any())
    for cu in ([0, 4, 3, 12, 16], [0, 4, 8, 12, 17], [0, 5, 9, 13, 16], [-1, 4, 8, 12, 16]):  # not a cut of the rows into trees
        o.zero_(), status.zero_()
        libkda.kda_tree_step(*args, i32(cu), i32(x["slots"]), pool, o, u, 4, status=status)
        assert int(status) == libkda.KDA_ERR_INVALID_ARG
    x["slots"][2] = 0 if 0 not in x["slots"] else next(s for s in range(7) if s not in x["slots"])
    path, before = i32([[0, 1], [0, 4], [0, 1], [-1, 1]]), pool.clone()
    status.zero_()
    libkda.kda_tree_commit(args[1], args[3], u, i32(x["cu"]), path, i32([2, 2, 3, 2]), i32(x["slots"]), pool, status=status)
    assert int(status) == libkda.KDA_ERR_INVALID_ARG
    changed = [s for s in range(7) if not torch.equal(pool[s], before[s])]
    assert changed == [x["slots"][0]]
    conv, status = torch.zeros((7, 3, 128), device="cuda"), i32([0])
    flat = q.view(16, 128)
    libkda.kda_tree_conv_commit(flat, i32(x["cu"]), path, i32([2, 2, 3, 2]), i32(x["slots"]), conv, status=status)
    assert int(status) == libkda.KDA_ERR_INVALID_ARG and [s for s in range(7) if conv[s].any()] == [x["slots"][0]]
    y, status = torch.zeros((16, 128), dtype=BF, device="cuda"), i32([0])
    libkda.kda_tree_conv(flat, torch.ones((128, 4), device="cuda"), args[5], i32(x["cu"]), i32(x["slots"]), conv, y, 4, status=status)
    assert int(status) == libkda.KDA_ERR_INVALID_ARG and not y[4:8].any() and bool(y[8:].any())
    v = verify_inputs([2, 2, 2], 10, F32, 1, False)
    v["parent"][3] = 1
    path, length, token, status = run_verify(v, 2)
    assert status == libkda.KDA_ERR_INVALID_ARG and length[1] == 0 and token[1] == -1 and path[1] == [-1, -1] and length[0] > 0
    # a tree above the bound is refused as a whole
    x = step_inputs([3, 5], 1, 64, F32, 2)
    q = x["q"].cuda()
    o, status = torch.zeros_like(q), i32([0])
    libkda.kda_tree_step(q, x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), x["beta"].cuda(), i32(x["parent"]), i32(x["cu"]), None,
                         x["pool"].cuda(), o, None, 4, status=status)
    assert int(status) == libkda.KDA_ERR_INVALID_ARG and not o[3:].any() and bool(o[:3].any())


def test_refusals():
    x = step_inputs([3], 2, 64, F32, 1)
    q, k, v, g, beta, pool = (x[n].cuda() for n in ("q", "k", "v", "g", "beta", "pool"))
    parent, cu, slots, o, u = i32(x["parent"]), i32(x["cu"]), i32(x["slots"]), torch.empty_like(q), torch.empty_like(q)
    ok = [q, k, v, g, beta, parent, cu, slots, pool, o, u, 3]
    libkda.kda_tree_step(*ok)

    def refuses(error, at, value):
        with pytest.raises(error):
            libkda.kda_tree_step(*[value if i == at else a for i, a in enumerate(ok)])
    refuses(ValueError, 1, k[:2])
    refuses(ValueError, 0, q.transpose(0, 1).contiguous().transpose(0, 1))
    refuses(ValueError, 8, pool.cpu())
    refuses(ValueError, 9, torch.empty((3, 2, 63), device="cuda"))
    refuses(TypeError, 2, v.bfloat16())
    refuses(TypeError, 5, parent.long())
    refuses(TypeError, 8, pool.bfloat16())
    refuses(libkda.KdaError, 9, q)
    refuses(libkda.KdaError, 11, 0)
    refuses(libkda.KdaError, 11, 65)
    path, taken = i32([[0, 1]]), i32([2])
    with pytest.raises(ValueError):
        libkda.kda_tree_commit(k, g, u[:2], cu, path, taken, slots, pool)
    with pytest.raises(libkda.KdaError):
        libkda.kda_tree_commit(k, g, u, cu, i32([[0] * 65]), taken, slots, pool)
    xs, w, conv = torch.zeros((3, 8), device="cuda"), torch.zeros((8, 9), device="cuda"), torch.zeros((2, 8, 8), device="cuda")
    with pytest.raises(libkda.KdaError):
        libkda.kda_tree_conv(xs, w, parent, cu, slots, conv, torch.empty_like(xs), 3)
    with pytest.raises(libkda.KdaError):
        libkda.kda_tree_conv(xs, w[:, :3].contiguous(), parent, cu, slots, conv[:, :2].contiguous(), xs, 3)
    l, ut, out = torch.zeros((3, 8), device="cuda"), torch.zeros(3, device="cuda"), i32([0])
    with pytest.raises(TypeError):
        libkda.kda_draft_verify(l.half(), i32([0, 0, 0]), parent, cu, ut, ut[:1], i32([[0] * 3]), out, out.clone())
    with pytest.raises(ValueError):
        libkda.kda_draft_verify(l, i32([0, 0]), parent, cu, ut, ut[:1], i32([[0] * 3]), out, out.clone())


def test_other_streams_and_graphs():
    """Every call runs on the stream it is given and can be captured: a round replayed gives the same bits."""
    x = step_inputs([16, 5], 2, 128, BF, 21)
    q, k, v, g, beta, pool = (x[n].cuda() for n in ("q", "k", "v", "g", "beta", "pool"))
    parent, cu, slots = i32(x["parent"]), i32(x["cu"]), i32(x["slots"])
    o, u = torch.zeros_like(q), torch.zeros(q.shape, device="cuda")
    y = verify_inputs([16, 5], 777, BF, 21, True)
    y = {n: (i32(t) if isinstance(t, list) else t if t is None else t.cuda()) for n, t in y.items()}
    path, taken, token = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 16), (2,), (2,)))

    def round_(stream):
        libkda.kda_tree_step(q, k, v, g, beta, parent, cu, slots, pool, o, u, 16, stream=stream)
        libkda.kda_draft_verify(y["logits"], y["tokens"], parent, cu, y["u"], y["u_next"], path, taken, token, draft_probs=y["probs"], stream=stream)
        libkda.kda_tree_commit(k, g, u, cu, path, taken, slots, pool, stream=stream)
    before = pool.clone()
    y["parent"] = parent
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    round_(side)
    side.synchronize()
    first = [t.clone() for t in (o, u, path, taken, token, pool)]
    pool.copy_(before)
    for t in (o, u, path, taken, token):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        round_(torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (o, u, path, taken, token, pool)))
    assert bool(first[0].any()) and bool(first[3].all())
