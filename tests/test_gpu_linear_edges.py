"""Linear attention where it went wrong once, against fp64 references.  Tolerances as in test_gpu_linear, element by element,
unless a test says otherwise."""
import numpy as np
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from oracle import linear
from tests.gpu_helpers import f64
from tests.test_gpu_linear import BF, F32, HALF, inputs, run_prefill, within

pytestmark = pytest.mark.gpu


def table(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(int).tolist()


def check(x, lengths, q, k, S0=None, **more):
    """A prefill of x against the recurrence over q, k in 64 bits; returns the largest of the sums over absolute values."""
    cu, dtype, d = table(lengths), x["v"].dtype, x["v"].shape[-1]
    o, S = run_prefill(x, cu, S0, **more)
    ref_o, ref_S, m, A = linear.attention(q, k, f64(x["v"]), f64(x["g"]), cu, None if S0 is None else f64(S0))
    T, tensor_cores = max(lengths), dtype == BF and d == 128
    sums = (T + 64) * 2.0 ** -23 + 2.0 ** -20
    within(o, ref_o, (sums + (2.0 ** -8 if tensor_cores else 0)) * m + (HALF[dtype] + 2.0 ** -20) * np.abs(ref_o), "o")
    within(S, ref_S, (sums + (3 * T * 2.0 ** -23 if tensor_cores else 0)) * A, "S")
    return max(m.max(), A.max())


@pytest.mark.parametrize("lengths", [[1], [63], [64], [65], [77], [65, 1, 0, 77, 63], [900]], ids=str)
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_norms_without_an_epsilon(lengths, dtype, d):
    """Rows behind a document have no norm; where the sum of their squares is 0, its inverse root must not reach the state."""
    x = inputs(sum(lengths), 4, 2, d, dtype, 73)
    S0 = 0.1 * torch.randn((len(lengths), 4, d, d), generator=torch.Generator().manual_seed(1))
    check(x, lengths, linear.unit(f64(x["q"]), 0.0), linear.unit(f64(x["k"]), 0.0), S0, qk_l2norm=True, qk_eps=0.0)


def test_calls_on_two_streams_take_memory_of_their_own(monkeypatch):
    """Calls without a workspace, on the current stream and on another, one right behind the other: the second must not be
    given memory that the first one's work, still to come, is to use."""
    lengths, H, d = [4000, 64], 4, 128
    cu = torch.tensor(table(lengths), dtype=torch.int32, device="cuda")
    xs = [inputs(sum(lengths), H, H, d, BF, 79 + i) for i in range(2)]
    refs = [run_prefill(x, table(lengths)) for x in xs]
    on = [{n: t.cuda() for n, t in x.items()} for x in xs]
    outs = [(torch.empty_like(x["v"]), torch.empty((2, H, d, d), device="cuda")) for x in on]
    streams, taken, allocate = [None, torch.cuda.Stream()], [], libkda.new_linear_workspace

    def noted(*args):
        workspace = allocate(*args)
        taken.append(workspace.data_ptr())
        return workspace

    monkeypatch.setattr(libkda, "new_linear_workspace", noted)
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000)
    for _ in range(20):
        for x, (o, S), stream in zip(on, outs, streams):
            libkda.kda_linear_prefill(x["q"], x["k"], x["v"], x["g"], cu, o, S_final=S, stream=stream)
    torch.cuda.synchronize()
    assert not set(taken[0::2]) & set(taken[1::2])
    for out, ref in zip(outs, refs):
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


@pytest.mark.parametrize("kind", ["decays", "grows", "both"])
@pytest.mark.parametrize("dtype,d", [(F32, 16), (F32, 64), (F32, 128), (BF, 16), (BF, 128)])
def test_values_near_the_largest(dtype, d, kind):
    """Twenty bits of decay over 32 tokens, growth, and growth behind decay, of values whose sums stay below fp32's largest even
    if all terms had one sign: nothing on the way may overflow."""
    x = inputs(400, 2, 1, d, dtype, 89)
    g = {"decays": torch.full((400,), -0.4), "grows": torch.full((400,), 0.1), "both": torch.where(torch.arange(400) % 30 < 15, -0.4, 0.4)}[kind]
    x["g"] = g[:, None].expand(400, 2).contiguous()
    x["v"] = (x["v"].float() * 2.0 ** {"decays": 115, "grows": 70, "both": 104}[kind]).to(dtype)
    most = check(x, [150, 250], f64(x["q"]), f64(x["k"]))
    assert most < 2.0 ** 127


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("T,H,d,dtype,factors,tokens", [
    (16384, 608, 128, F32, 1024, 16), (32768, 608, 64, F32, 512, 32), (32768, 608, 16, BF, 512, 32),  # stages of one segment or two
    (65536, 1, 64, F32, 1023, 64), (65536, 2, 128, F32, 255, 256), (38912, 1, 128, BF, 151, 256)])   # links of the chain
def test_one_decay_for_many_factors(T, H, d, dtype, factors, tokens, sign):
    """S0 alone, decayed or grown by one factor for each run of `tokens` tokens: its rounding must not add up.  The mean error of
    S in steps of 2^-24, over its elements: independent roundings, one a factor, 0.3 at most; the product of the factors is
    right to a step of fp32, 2; the log-decay to base 2 has two roundings, times the exponent reached, 0.5; the last run's
    and the chain's products, 2.  A factor that is off by a fifth of 2^-24 adds 30 and more."""
    run = np.float32(sign * 2.0 ** -2 / T) * (1 + np.arange(64, dtype=np.float32) / 64)
    g = next(x for x in run if abs(float(np.float32(np.exp(tokens * float(x)))) / np.exp(tokens * float(x)) - 1) > 0.2 * 2.0 ** -24)
    v, qk = torch.zeros((T, H, d), dtype=dtype, device="cuda"), torch.zeros((T, 1, d), dtype=dtype, device="cuda")
    S0 = torch.randn((1, H, d, d), generator=torch.Generator(device="cuda").manual_seed(97), device="cuda")
    S, cu = torch.empty_like(S0), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    libkda.kda_linear_prefill(qk, qk, v, torch.full((H,), float(g), device="cuda"), cu, torch.empty_like(v), S0=S0, S_final=S)
    some = S0 != 0
    assert (S[~some] == 0).all()
    error = (S[some].double() / (S0[some].double() * np.exp(float(g) * T)) - 1).mean().item()
    assert abs(error) <= 8 * 2.0 ** -24, error * 2 ** 24


STATE = 8e-7  # see test_the_state_keeps_24_bits; test_linear_edges_cpu shows what it tells apart


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("lengths", [[64], [65], [700], [3000, 200], [1, 4097]], ids=str)
def test_the_state_keeps_24_bits(lengths, per_token, norm):
    """The state on the tensor cores in the 2-norm, each document and head by itself.  A chunk's product is twelve sums, each cut off
    below 24 bits, which takes 2^-24 of it on average: 7.2e-7 at most if all were as large as the last; beside that
    the independent errors of single terms (2^-22 at most: exp2, the norm, their products) count for 2e-7, in quadrature.  The
    decayed v in two bf16 parts instead of three, or with a third one that belongs elsewhere, is off by 2e-6."""
    cu = table(lengths)
    x = inputs(cu[-1], 3, 3, 128, BF, 101, per_token)
    q, k = f64(x["q"]), f64(x["k"])
    _, ref, _, _ = linear.attention(linear.unit(q, 1e-6) if norm else q, linear.unit(k, 1e-6) if norm else k, f64(x["v"]), f64(x["g"]), cu)
    _, S = run_prefill(x, cu, qk_l2norm=norm)
    off = np.linalg.norm(f64(S) - ref, axis=(2, 3)) / np.linalg.norm(ref, axis=(2, 3))
    assert (off <= STATE).all(), off
