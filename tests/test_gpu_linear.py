"""Linear attention with one decay per head against fp64 references.

Tolerances, element by element, from the arithmetic (m, A: the reference's sums over absolute values, eps: half a step of
a type, 2^-24 for fp32 and 2^-8 for bf16):
  fp32 sums         of T terms, each with a few roundings:           (T + 64) 2^-23 of m or A
  tensor cores, o   its own rounding, and one of the scores and one of the state, which share m between them:
                    2^-8 (|o| + m)
  tensor cores, S   k v^T's v in three parts, all 24 bits.  A product's sum is cut off, not rounded: each of 3 T products and of the
                    12 sums a chunk carries loses at most 2^-23 of the largest:      (4 T + 64) 2^-23 A
  rsqrt, exp2, 1/x  of the fused steps and the decays, 2^-21 of the value each
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from oracle import linear
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(rows, H, Hqk, d, dtype, seed, per_token=True, decay=-2.5):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k = (torch.nn.functional.normalize(randn(rows, Hqk, d), dim=-1).to(dtype) for _ in range(2))
    gate = -torch.exp(1.2 * randn(rows, H) + decay) if per_token else -torch.exp2(-5 - 7 * torch.arange(H) / max(1, H - 1))
    return dict(q=q, k=k, v=randn(rows, H, d).to(dtype), g=gate.float(), z=randn(rows, H, d).to(dtype), weight=1 + 0.1 * randn(d))


def fused_args(x, fused):
    return dict(qk_l2norm=True, qk_eps=EPS, out_gate=x["z"].cuda(), out_weight=x["weight"].cuda(), out_eps=EPS) if fused else {}


def expected(x, cu, S0, fused, tensor_cores):
    q, k = f64(x["q"]), f64(x["k"])
    if fused:
        q, k = linear.unit(q, EPS), linear.unit(k, EPS)
    o, S, m, A = linear.attention(q, k, f64(x["v"]), f64(x["g"]), cu, None if S0 is None else f64(S0))
    T = max(1, o.shape[0])
    loose_o, loose_S = ((T + 64) * 2.0 ** -23 + 2.0 ** -20) * m, ((T + 64) * 2.0 ** -23 + 2.0 ** -20) * A
    if tensor_cores:
        loose_o, loose_S = loose_o + 2.0 ** -8 * m, loose_S + 3 * T * 2.0 ** -23 * A
    if fused:
        o, loose_o = linear.gated(o, m, x["z"].double().numpy(), x["weight"].double().numpy(), EPS, loose_o)
    loose_o = loose_o + (HALF[x["v"].dtype] + 2.0 ** -20) * np.abs(o)
    return o, S, loose_o, loose_S


def within(x, ref, loose, what):
    d = np.abs(f64(x) - ref)
    assert not np.isnan(d).any(), what
    worst = (d - loose).max() if d.size else 0.0
    assert worst <= 1e-30, (what, worst, (d / np.maximum(loose, 1e-30)).max())


def run_prefill(x, cu, S0=None, fused=False, want_state=True, **more):
    v = x["v"].cuda()
    T, H, d = v.shape
    N = len(cu) - 1
    o = torch.full_like(v, float("nan"))
    S = torch.full((N, H, d, d), float("nan"), device="cuda") if want_state else None
    cu = i32(cu)
    ws = libkda.new_linear_workspace(x["q"].cuda(), v, cu)
    ws.fill_(0xA5)
    libkda.kda_linear_prefill(x["q"].cuda(), x["k"].cuda(), v, x["g"].cuda(), cu, o, S0=None if S0 is None else S0.cuda(), S_final=S, workspace=ws,
                              **fused_args(x, fused), **more)
    assert libkda.kda_prefill_check(ws) == libkda.KDA_OK
    return o, S


def check_prefill(lengths, H, Hqk, d, dtype, seed=0, per_token=True, fused=False, with_S0=False, x=None):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int).tolist()
    x = x or inputs(cu[-1], H, Hqk, d, dtype, seed, per_token)
    S0 = 0.1 * torch.randn((len(lengths), H, d, d), generator=torch.Generator().manual_seed(seed + 99)) if with_S0 else None
    o, S = run_prefill(x, cu, S0, fused)
    ref_o, ref_S, loose_o, loose_S = expected(x, cu, S0, fused, dtype == BF and d == 128)
    within(o, ref_o, loose_o, "o")
    within(S, ref_S, loose_S, "S")
    return x, cu, o, S


LENGTHS = [[1], [63], [64], [65], [0, 5, 0, 0, 130, 64, 1, 0], [200, 3, 321], [1] * 40, [700]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("dtype,d,H,Hqk", [(BF, 128, 3, 3), (BF, 128, 4, 2), (BF, 64, 2, 1), (F32, 128, 2, 2), (F32, 16, 3, 1)])
def test_prefill(lengths, dtype, d, H, Hqk):
    check_prefill(lengths, H, Hqk, d, dtype, with_S0=True)


@pytest.mark.parametrize("lengths", [[1], [64], [0, 77, 300, 0, 64, 1], [900]], ids=str)
@pytest.mark.parametrize("dtype,d,H,Hqk", [(BF, 128, 3, 3), (BF, 128, 4, 1), (F32, 64, 2, 1), (BF, 16, 2, 2)])
def test_prefill_fused(lengths, dtype, d, H, Hqk):
    check_prefill(lengths, H, Hqk, d, dtype, fused=True, seed=3)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("with_S0", [False, True])
def test_one_decay_a_head(dtype, d, with_S0):
    check_prefill([1300, 40], 3, 3, d, dtype, per_token=False, with_S0=with_S0)


def test_parts_of_the_fused_steps():
    """Each fused step by itself, and the output's without a weight."""
    x = inputs(333, 2, 2, 128, BF, 5)
    cu = [0, 100, 333]
    q, k = linear.unit(f64(x["q"]), EPS), linear.unit(f64(x["k"]), EPS)
    v, o = x["v"].cuda(), torch.empty_like(x["v"], device="cuda")
    args = (x["q"].cuda(), x["k"].cuda(), v, x["g"].cuda(), i32(cu), o)
    libkda.kda_linear_prefill(*args, qk_l2norm=True, qk_eps=EPS)
    ref, _, m, _ = linear.attention(q, k, f64(x["v"]), f64(x["g"]), cu)
    within(o, ref, 2.0 ** -8 * (np.abs(ref) + m) + 2.0 ** -14 * m, "normalised q, k")
    libkda.kda_linear_prefill(*args, out_gate=x["z"].cuda(), out_eps=EPS)
    ref, _, m, _ = linear.attention(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["g"]), cu)
    ref, loose = linear.gated(ref, m, f64(x["z"]), None, EPS, (2.0 ** -8 + 2.0 ** -14) * m)
    within(o, ref, loose + (2.0 ** -8 + 2.0 ** -20) * np.abs(ref), "gated o")


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("kind", ["forget all", "keep all", "forget now and then", "grow"])
def test_extreme_decays(dtype, d, kind):
    """exp(-inf) = 0 at every token or some, log-decays of zero, and states that grow."""
    x = inputs(400, 2, 2, d, dtype, 7)
    r = torch.Generator().manual_seed(1)
    shape = x["g"].shape
    if kind == "forget all":
        x["g"] = torch.full(shape, float("-inf"))
    elif kind == "keep all":
        x["g"] = torch.zeros(shape)
    elif kind == "forget now and then":
        far = torch.tensor([float("-inf"), -1e30, -300.0, -90.0])[torch.randint(0, 4, shape, generator=r)]
        x["g"] = torch.where(torch.rand(shape, generator=r) < 0.1, far, torch.tensor(-1e-3))
    else:
        x["g"] = 0.05 * torch.rand(shape, generator=r)
    check_prefill([150, 250], 2, 2, d, dtype, with_S0=True, x=x)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_many_tokens_behind_one_another(dtype, d):
    """Sums over thousands of tokens that nothing is forgotten of, in several segments."""
    x = inputs(5000, 2, 1, d, dtype, 11)
    x["g"] = torch.full((2,), -1e-4)
    check_prefill([5000], 2, 1, d, dtype, x=x)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_a_document_of_nan_leaves_the_others_alone(dtype, d):
    lengths, H = [70, 30, 500, 64, 10], 2
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    x = inputs(cu[-1], H, H, d, dtype, 13)
    clean_o, clean_S = run_prefill(x, cu, fused=True)
    for name in ("q", "k", "v"):
        for n in (1, 3):
            x[name][cu[n]:cu[n + 1]] = float("nan") if n == 1 else float("inf")
    o, S = run_prefill(x, cu, fused=True)
    for n in (0, 2, 4):
        assert torch.equal(o[cu[n]:cu[n + 1]], clean_o[cu[n]:cu[n + 1]]) and torch.equal(S[n], clean_S[n])
    assert torch.isnan(S[1]).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_a_nan_decay_shows(dtype, d):
    x = inputs(300, 1, 1, d, dtype, 17)
    clean_o, _ = run_prefill(x, [0, 300])
    x["g"][100] = float("nan")
    o, S = run_prefill(x, [0, 300])
    assert torch.isnan(S).all() and torch.isnan(o[100:]).all()
    assert torch.equal(o[:64], clean_o[:64])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_same_inputs_same_bits(dtype, d):
    x = inputs(3000, 4, 4, d, dtype, 19)
    cu = [0, 1000, 1000, 3000]
    first = run_prefill(x, cu, fused=True)
    for _ in range(3):
        again = run_prefill(x, cu, fused=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_states_in_place_and_continued(dtype, d):
    """S_final in S0's place, over documents of several segments; and two calls that continue one another."""
    lengths, H = [2000, 0, 100], 2
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    x = inputs(cu[-1], H, H, d, dtype, 23)
    S0 = 0.1 * torch.randn((3, H, d, d), generator=torch.Generator().manual_seed(2))
    ref_o, ref_S = run_prefill(x, cu, S0)
    S = S0.cuda()
    o = torch.empty_like(x["v"], device="cuda")
    libkda.kda_linear_prefill(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), i32(cu), o, S0=S, S_final=S)
    assert torch.equal(o, ref_o) and torch.equal(S, ref_S)
    assert torch.equal(S[1].cpu(), S0[1])  # the empty document's is its incoming one
    one = inputs(1500, H, H, d, dtype, 29)
    whole, end = run_prefill(one, [0, 1500])
    part = lambda a, b: {n: t[a:b] if n != "weight" else t for n, t in one.items()}  # noqa: E731
    o1, S1 = run_prefill(part(0, 777), [0, 777])
    o2, S2 = run_prefill(part(777, 1500), [0, 723], S0=S1)
    ref_o, ref_S, loose_o, loose_S = expected(one, [0, 1500], None, False, dtype == BF and d == 128)
    within(torch.cat([o1, o2]), ref_o, loose_o, "continued o")
    within(S2, ref_S, loose_S, "continued S")


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("cu", [[0, 100, 50, 400], [0, 100, 401], [1, 100, 400], [0, -5, 400], [0, 100, 399], [0, 500, 400]], ids=str)
def test_invalid_tables_write_nothing(dtype, d, cu):
    x = inputs(400, 2, 2, d, dtype, 31)
    o = torch.full_like(x["v"], 3.0, device="cuda")
    S = torch.full((len(cu) - 1, 2, d, d), 5.0, device="cuda")
    ws = libkda.new_linear_workspace(x["q"].cuda(), x["v"].cuda(), i32(cu))
    libkda.kda_linear_prefill(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), i32(cu), o, S_final=S, workspace=ws)
    assert libkda.kda_prefill_check(ws) == libkda.KDA_ERR_INVALID_ARG
    assert (o == 3).all() and (S == 5).all()


def test_no_tokens_and_no_sequences():
    for dtype, d in ((BF, 128), (F32, 16)):
        x = inputs(0, 2, 2, d, dtype, 37)
        S0 = torch.randn(3, 2, d, d)
        o, S = run_prefill(x, [0, 0, 0, 0], S0)
        assert torch.equal(S.cpu(), S0)
        _, S = run_prefill(x, [0, 0, 0, 0])
        assert (S == 0).all()
        libkda.kda_linear_prefill(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), i32([0]), o)
        libkda.kda_linear_decode_step(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), S, o)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_streams_and_graphs(dtype, d):
    """Two calls on two streams at once, and a captured call replayed on new inputs."""
    lengths = [900, 64, 300]
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    xs = [inputs(cu[-1], 4, 4, d, dtype, 41 + i) for i in range(2)]
    refs = [run_prefill(x, cu, fused=True) for x in xs]
    on = [{n: t.cuda() for n, t in x.items()} for x in xs]
    outs = [(torch.empty_like(x["v"]), torch.empty((3, 4, d, d), device="cuda")) for x in on]
    works = [libkda.new_linear_workspace(x["q"], x["v"], i32(cu)) for x in on]
    table = i32(cu)

    def call(i, stream=None):
        x = on[i]
        libkda.kda_linear_prefill(x["q"], x["k"], x["v"], x["g"], table, outs[i][0], S_final=outs[i][1], workspace=works[i], stream=stream,
                                  qk_l2norm=True, qk_eps=EPS, out_gate=x["z"], out_weight=x["weight"], out_eps=EPS)

    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], refs[i][0]) and torch.equal(outs[i][1], refs[i][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for n, t in on[0].items():
        t.copy_(xs[1][n])
    for t in outs[0]:
        t.fill_(float("nan"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], refs[1][0]) and torch.equal(outs[0][1], refs[1][1])


def test_one_decay_for_many_chunks():
    """S0 alone, decayed by one factor chunk after chunk: its rounding must not add up.  The mean error of S over 2.5 million
    elements: each chunk's rounding of S, within 2^-24 either way and independent, stays below 256 x 2^-24 x sqrt(28 / 5e6),
    1 part of 2^-24, but for one time in 10^12; one factor's rounding, the log-decay's to base 2 (times the exponent reached,
    0.4) and the last product add 3.  A factor that is off by a fifth of 2^-24 would add 50 in 256 chunks."""
    T, H, d = 16384, 152, 128
    g = next(x for x in np.float32(-2.0 ** -16) * (1 + np.arange(64, dtype=np.float32) / 64)
             if abs(float(np.float32(np.exp(64.0 * x))) / np.exp(64.0 * float(x)) - 1) > 0.2 * 2.0 ** -24)
    zeros = torch.zeros((T, H, d), dtype=BF, device="cuda")
    S0 = torch.randn((1, H, d, d), device="cuda")
    S = torch.empty_like(S0)
    libkda.kda_linear_prefill(zeros[:, :1].contiguous(), zeros[:, :1].contiguous(), zeros, torch.full((H,), float(g), device="cuda"), i32([0, T]),
                              torch.empty_like(zeros), S0=S0, S_final=S)
    some = S0 != 0  # (a zero stays one; 0 / 0 is no error of S)
    assert (S[~some] == 0).all()
    error = (S[some].double() / (S0[some].double() * np.exp(float(g) * T)) - 1).mean().item()
    assert abs(error) <= 8 * 2.0 ** -24


def test_a_workspace_of_its_own_on_another_stream():
    """Memory that the call takes for itself is not given out again before the other stream's work is done."""
    x, cu, stream = inputs(4000, 4, 4, 128, BF, 47), [0, 4000], torch.cuda.Stream()
    ref = run_prefill(x, cu)
    on, table = {n: t.cuda() for n, t in x.items()}, i32(cu)
    o, S = torch.empty_like(on["v"]), torch.empty((1, 4, 128, 128), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
    libkda.kda_linear_prefill(on["q"], on["k"], on["v"], on["g"], table, o, S_final=S, stream=stream)
    others = [libkda.new_linear_workspace(on["q"], on["v"], table).fill_(255) for _ in range(3)]
    torch.cuda.synchronize()
    assert others and torch.equal(o, ref[0]) and torch.equal(S, ref[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_past_32_bits(dtype):
    """The last document of a batch whose v, o and states lie past 2^31 elements gives what it gives alone."""
    d, H, T = 128, 128, 133000
    N = 1100 if dtype == F32 else 2  # states past 2^31 elements too
    g = torch.Generator(device="cuda").manual_seed(43)
    last = 300
    cu = torch.cat([torch.linspace(0, T - last, N, device="cuda").to(torch.int32), torch.tensor([T], dtype=torch.int32, device="cuda")])
    q, k = (torch.randn((T, 1, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    v = torch.empty((T, H, d), dtype=dtype, device="cuda")
    v[:-last] = 1
    v[-last:] = torch.randn((last, H, d), generator=g, device="cuda").to(dtype)
    decay = -torch.rand(H, generator=g, device="cuda")
    o, S = torch.empty_like(v), torch.empty((N, H, d, d), device="cuda")
    assert v.numel() > 2 ** 31 and (dtype == BF or S.numel() > 2 ** 31)
    libkda.kda_linear_prefill(q, k, v, decay, cu, o, S_final=S)
    alone, end = torch.empty_like(v[-last:]), torch.empty((1, H, d, d), device="cuda")
    libkda.kda_linear_prefill(q[-last:], k[-last:], v[-last:], decay, i32([0, last]), alone, S_final=end)
    tight = 2.0 ** -6 if dtype == BF else 2.0 ** -12  # another split of the document: rounded at other places
    assert (o[-last:].float() - alone.float()).norm() <= tight * alone.float().norm()
    assert (S[-1] - end[0]).norm() <= 2.0 ** -12 * end.norm()
    del q, k, v, o, S
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------------------------------------------
# one token
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("dtype,d,H,Hqk,N", [(BF, 128, 3, 3, 5), (BF, 128, 16, 4, 1), (F32, 64, 4, 1, 7), (BF, 16, 5, 5, 33), (F32, 128, 2, 2, 40),
                                             (F32, 16, 1, 1, 1)])
def test_decode(dtype, d, H, Hqk, N, per_token, fused):
    x = inputs(N, H, Hqk, d, dtype, 47, per_token)
    slots = torch.randperm(N + 3, generator=torch.Generator().manual_seed(3))[:N].tolist()
    pool = 0.1 * torch.randn((N + 3, H, d, d), generator=torch.Generator().manual_seed(4))
    S, o, status = pool.cuda(), torch.full_like(x["v"], float("nan"), device="cuda"), i32([0])
    libkda.kda_linear_decode_step(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), S, o, seq_idx=i32(slots), status=status,
                                  **fused_args(x, fused))
    ref_o, ref_S, loose_o, loose_S = expected(x, list(range(N + 1)), pool[slots], fused, False)
    within(o, ref_o, loose_o, "o")
    within(S[slots], ref_S, loose_S, "S")
    rest = [i for i in range(N + 3) if i not in slots]
    assert int(status) == 0 and torch.equal(S[rest].cpu(), pool[rest])


def test_decode_without_an_index():
    x = inputs(4, 2, 2, 128, BF, 53)
    pool = torch.randn(6, 2, 128, 128)
    S, o = pool.cuda(), torch.empty_like(x["v"], device="cuda")
    libkda.kda_linear_decode_step(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), S, o)
    ref_o, ref_S, loose_o, loose_S = expected(x, list(range(5)), pool[:4], False, False)
    within(o, ref_o, loose_o, "o")
    within(S[:4], ref_S, loose_S, "S")
    assert torch.equal(S[4:].cpu(), pool[4:])


def test_decode_skips_slots_outside_the_pool():
    x = inputs(5, 2, 2, 128, BF, 59)
    pool = torch.randn(4, 2, 128, 128)
    S, o, status = pool.cuda(), torch.full_like(x["v"], 7.0, device="cuda"), i32([0])
    libkda.kda_linear_decode_step(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), S, o, seq_idx=i32([2, -1, 0, 4, 1 << 30]), status=status)
    assert int(status) == libkda.KDA_ERR_INVALID_ARG
    assert (o[[1, 3, 4]] == 7).all() and not (o[[0, 2]] == 7).all()
    assert torch.equal(S[[1, 3]].cpu(), pool[[1, 3]]) and not torch.equal(S[0].cpu(), pool[0])


def test_decode_pool_past_32_bits():
    slots, H, d = 4200, 32, 128
    S = torch.zeros((slots, H, d, d), device="cuda")
    assert S.numel() > 2 ** 31
    x = {n: t.cuda() for n, t in inputs(1, H, H, d, BF, 61).items()}
    o = torch.empty_like(x["v"])
    libkda.kda_linear_decode_step(x["q"], x["k"], x["v"], x["g"], S, o, seq_idx=i32([slots - 1]))
    ref = x["k"][0].float()[:, :, None] * x["v"][0].float()[:, None, :]
    assert (S[-1] - ref).abs().max() <= 2.0 ** -23 * ref.abs().max() and (S[-2] == 0).all()
    del S
    torch.cuda.empty_cache()


def test_decode_graph_replay_and_stream():
    x = {n: t.cuda() for n, t in inputs(9, 4, 4, 128, BF, 67).items()}
    pool = torch.randn((9, 4, 128, 128), device="cuda")
    want, got, o1, o2 = pool.clone(), pool.clone(), torch.empty_like(x["v"]), torch.empty_like(x["v"])
    for _ in range(3):
        libkda.kda_linear_decode_step(x["q"], x["k"], x["v"], x["g"], want, o1)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        libkda.kda_linear_decode_step(x["q"], x["k"], x["v"], x["g"], got, o2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(o1, o2)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_serving_a_layer(dtype, d):
    """Prompts of several requests, their states to a pool, tokens one after another: positions rotated, as one long
    sequence gives it."""
    H, lengths, steps = 2, [70, 1, 200], 4
    N = len(lengths)
    total = [n + steps for n in lengths]
    cu_all = np.concatenate([[0], np.cumsum(total)]).tolist()
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    x = inputs(cu_all[-1], H, H, d, dtype, 71)
    positions = np.concatenate([np.arange(n) for n in total])
    freq, _ = libkda.rope_frequencies(d)
    table = libkda.rope_steps(freq).cuda()
    prompt = np.concatenate([np.arange(cu_all[n], cu_all[n] + lengths[n]) for n in range(N)])
    pool, slots = torch.full((N + 2, H, d, d), float("nan"), device="cuda"), i32([3, 0, 4])

    def layer(rows, run):
        q, k, v, g = (x[n][rows].cuda() for n in ("q", "k", "v", "g"))
        libkda.kda_rope(q, k, i32(positions[rows].tolist()), table, q, k)
        o = torch.empty_like(v)
        run(q, k, v, g, o)
        return q, k, o

    S = torch.empty((N, H, d, d), device="cuda")
    q, k, o = layer(prompt, lambda q, k, v, g, o: libkda.kda_linear_prefill(q, k, v, g, i32(cu), o, S_final=S))
    libkda.kda_state_restore(S, slots, pool)
    rq, rk, ro = x["q"].clone(), x["k"].clone(), torch.empty_like(x["v"])
    rq[prompt], rk[prompt], ro[prompt] = q.cpu(), k.cpu(), o.cpu()
    for t in range(steps):
        rows = np.array([cu_all[n] + lengths[n] + t for n in range(N)])
        q, k, o = layer(rows, lambda q, k, v, g, o: libkda.kda_linear_decode_step(q, k, v, g, pool, o, seq_idx=slots))
        rq[rows], rk[rows], ro[rows] = q.cpu(), k.cpu(), o.cpu()
    turned = linear.rope(f64(x["q"]), positions, freq.numpy(), 1.0, False)
    within(rq, turned.astype(np.float64), 2 * HALF[dtype] * np.abs(turned).max() + 0 * f64(rq), "rotated q")
    ref_o, ref_S, loose_o, loose_S = expected({**x, "q": rq, "k": rk}, cu_all, None, False, dtype == BF and d == 128)
    within(ro, ref_o, loose_o, "o")
    within(pool[slots.long()], ref_S, loose_S, "S")
