"""The draft-tree operators where they can go wrong: addresses, masked logits, long decays, bounds of a batch.

Tolerances (fixed before measuring), max|x - ref| / max|ref|: 1e-4 for fp32 values, 2e-2 for bf16 outputs, as for the
operators' other tests, unless a test says and derives its own.
"""
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from oracle import tree
from tests.gpu_helpers import f64, rel
from tests.test_gpu_tree import BF, F32, check_verify, i32, run_step, step_inputs, verify_inputs

pytestmark = pytest.mark.gpu


def shifted(t, floats=4):
    """The same values, contiguous, 16 bytes behind a 256-byte boundary."""
    room = torch.empty(t.numel() + floats, dtype=t.dtype, device="cuda")
    view = room[floats:].view(t.shape)
    view.copy_(t)
    assert view.data_ptr() % 32 == 16 and view.is_contiguous()
    return view


@pytest.mark.parametrize("d,dtype", [(16, F32), (64, BF), (128, F32), (128, BF)])
@pytest.mark.parametrize("M", [5, 12, 30, 60])
def test_a_pool_at_any_16_byte_boundary(M, d, dtype):
    """A pool's address need not be a multiple of 32 bytes: step and commit give the bits that they give on one that is."""
    x = step_inputs([M, M // 2], 2, d, dtype, seed=M + d)
    o, u, pool = run_step(x, M)
    q, k, v, g, beta = (x[n].cuda() for n in ("q", "k", "v", "g", "beta"))
    at16 = shifted(x["pool"])
    o16, u16, status = torch.zeros_like(q), shifted(torch.zeros_like(u)), i32([0])
    libkda.kda_tree_step(q, k, v, shifted(g), beta, i32(x["parent"]), i32(x["cu"]), i32(x["slots"]), at16, o16, u16, M, status=status)
    assert int(status) == 0 and torch.equal(o16, o) and torch.equal(u16, u)
    path, taken = i32([[0, 1, -1], [0, -1, -1]]), i32([2, 1])
    for S in (pool, at16):
        libkda.kda_tree_commit(k, g, u, i32(x["cu"]), path, taken, i32(x["slots"]), S, status=status)
    assert int(status) == 0 and torch.equal(at16, pool)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("V", [1000, 5000, 50001])
def test_verify_a_nan_among_masked_logits(V, probs, dtype):
    """Rows that are -inf but for 64 tokens and a few NaN, far from those: a NaN weighs nothing, also where a child is
    rejected and the rest of the row is summed and searched."""
    x = verify_inputs([4, 8, 5, 7], V, dtype, V + probs, probs)
    x["logits"][:, 64:] = -float("inf")
    x["logits"][:, [300, 611, V - 1]] = float("nan")
    x["tokens"] = [t % 64 for t in x["tokens"]]
    if probs:  # a draft that is all too sure of one token
        x["tokens"] = [5] * len(x["tokens"])
        x["probs"][:] = 0.0
        x["probs"][:, :64] = 0.1 / 63
        x["probs"][:, 5] = 0.9
    x["u"][:] = 0.9999  # most trials are lost
    paths = check_verify(x, 8)
    assert min(len(p) for p in paths) == 1


@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("C", [130, 2048])
def test_both_commits_refuse_the_same_paths(C, W):
    """A path with a node outside its tree moves neither the state nor the carried inputs, wherever in the path it is."""
    M, N = 9, 4
    path = torch.arange(M, dtype=torch.int32).repeat(N, 1)
    path[1, 0], path[2, 3], path[3, M - 1] = -1, M, -1
    cu, taken, slots = i32([M * n for n in range(N + 1)]), i32([M] * N), i32(list(range(N)))
    g = torch.Generator(device="cuda").manual_seed(C + W)
    conv = torch.randn((N, W - 1, C), generator=g, device="cuda")
    S = torch.randn((N, 1, 64, 64), generator=g, device="cuda")
    x, k = (torch.randn(s, generator=g, device="cuda") for s in ((N * M, C), (N * M, 1, 64)))
    status, before = [i32([0]), i32([0])], (conv.clone(), S.clone())
    libkda.kda_tree_conv_commit(x, cu, path.cuda(), taken, slots, conv, status=status[0])
    libkda.kda_tree_commit(k, -k.abs(), k, cu, path.cuda(), taken, slots, S, status=status[1])
    assert [int(s) for s in status] == [libkda.KDA_ERR_INVALID_ARG] * 2
    assert torch.equal(conv[0], x[M - (W - 1):M]) and torch.equal(conv[1:], before[0][1:])
    assert not torch.equal(S[0], before[1][0]) and torch.equal(S[1:], before[1][1:])


@pytest.mark.parametrize("d,dtype", [(16, F32), (64, F32), (64, BF), (128, F32), (128, BF)])
@pytest.mark.parametrize("back", [1, 3])
@pytest.mark.parametrize("M", [16, 31, 64])
def test_a_steep_start_costs_no_accuracy_below_it(M, back, d, dtype):
    """Half of the channels are cleared by every node of the upper half, and the lower half forgets little: what it adds up
    has small exponents, however far the sums from the root have fallen.

    Tolerance 2e-5.  An exponent whose factor counts (above e^-20) is a sum of up to 64 decays with an error of at most
    64 x 2^-25 of 20, so a factor is off by 4e-5 at e^-20 and 2e-6 at e^-1; the products of two bf16 parts leave 3 x 2^-18 a
    term, 1.1e-5 where all have one sign.
    """
    x = step_inputs([M], 2, d, dtype, seed=M + d, back=back)
    x["g"][: M // 2, :, : d // 2] = -200.0
    x["g"][M // 2:] *= 0.01
    o, u, _ = run_step(x, M)
    o_ref, u_ref, _ = tree.tree_step(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta")), x["parent"], x["cu"], x["slots"], f64(x["pool"]))
    assert rel(u, u_ref) <= 2e-5
    assert rel(o, o_ref) <= (2e-5 if dtype == F32 else 2e-2)


@pytest.mark.parametrize("scale", [1.0, 1e-2, 1e-4])
@pytest.mark.parametrize("nats", [50.0, 78.0, 90.0])
@pytest.mark.parametrize("M", [8, 16, 24, 40])
def test_small_queries_below_a_long_decay(M, nats, scale):
    """The output is linear in q: far down a path, too, where the factors e^b are small, a small q loses no bits.

    Tolerance 2^-8 of a row's largest entry: the output's own rounding is half of that, what the parts of q leave out a
    hundredth.
    """
    x = step_inputs([M], 2, 128, BF, seed=M, back=1)
    x["q"] = (scale * x["q"].float()).to(BF)
    x["g"][:] = -nats / M
    o, _, _ = run_step(x, M)
    o_ref, _, _ = tree.tree_step(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta")), x["parent"], x["cu"], x["slots"], f64(x["pool"]))
    off = abs(f64(o) - o_ref).max(-1) / abs(o_ref).max(-1)
    assert off.max() <= 2.0 ** -8


def alone(x, n):
    """Request n of a batch by itself."""
    rows = slice(x["cu"][n], x["cu"][n + 1])
    return dict(x, cu=[0, rows.stop - rows.start], slots=[x["slots"][n]], parent=x["parent"][rows], **{t: x[t][rows] for t in ("q", "k", "v", "g", "beta")})


@pytest.mark.parametrize("d,dtype,bound,others", [(128, BF, 8, (5, 6)), (128, BF, 16, (9, 12)), (128, BF, 32, (17, 25)), (128, BF, 64, (33, 50)),
                                                  (128, F32, 64, (12, 16, 33)), (64, F32, 64, (12, 16, 33)), (64, BF, 64, (12, 16, 33)), (16, F32, 64, (12, 16, 33))])
def test_bits_do_not_depend_on_the_batch(bound, others, d, dtype):
    """A request gives the bits of o and u alone that it gives among others, and under every bound of its kernel."""
    lengths = [others[0], others[0] - 3, 2]
    x = step_inputs(lengths, 3, d, dtype, seed=bound + d)
    o, u, _ = run_step(x, bound)
    for n in range(3):
        rows = slice(x["cu"][n], x["cu"][n + 1])
        for M in others + (bound,):
            got = run_step(alone(x, n), M)
            assert torch.equal(got[0], o[rows]) and torch.equal(got[1], u[rows])


@pytest.mark.parametrize("low,high", [(8, 9), (16, 17), (32, 33), (8, 64)])
def test_bounds_of_two_kernels_agree(low, high):
    """bf16 at d = 128: the bound picks the kernel.  Each one's products of two bf16 parts are off by at most 3 x 2^-18 a
    term, so two differ by at most twice that in u (2.3e-5 of the largest), and by one rounding (2^-8) more in o."""
    x = step_inputs([low, low - 5, 1], 2, 128, BF, seed=low)
    (o, u, _), (o2, u2, _) = run_step(x, low), run_step(x, high)
    assert rel(u2, f64(u)) <= 2.3e-5 and rel(o2, f64(o)) <= 2.0 ** -8 + 2.3e-5
