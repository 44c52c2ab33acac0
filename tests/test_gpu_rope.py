"""Rotary positions against references in extended precision.

Tolerances: a value's rounding (half a step: 2^-24, 2^-8), and |x| + |y| times the errors of the angle -- fp32's rounding of
a part of half a turn (2^-24 of pi), sincospi's 2^-23, the frequency's own rounding to fp64 times the position -- with the
two products' roundings: 2^-21 + 2^-51 |position x frequency| in all.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from oracle import linear
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def check(q, q_out, positions, freq, scale, interleaved):
    ref = linear.rope(f64(q), positions, freq.numpy(), scale, interleaved)
    x = np.abs(f64(q))
    half, d = freq.numel(), q.shape[-1]
    pair = np.zeros_like(x)
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    far = np.abs(np.asarray(positions, dtype=np.float64))[:, None, None] * freq.numpy()
    pair[..., lo] = pair[..., hi] = scale * (x[..., lo] + x[..., hi]) * (2.0 ** -21 + 2.0 ** -51 * far)
    off = np.abs(f64(q_out) - ref.astype(np.float64)) - pair - HALF[q.dtype] * np.abs(ref.astype(np.float64))
    assert not np.isnan(off).any() and off.max(initial=0.0) <= 1e-30
    assert torch.equal(q_out[..., 2 * half:].cpu(), q[..., 2 * half:].cpu()) or d == 2 * half


SIZES = [(1, 1, 1, 16, 16), (7, 3, 1, 128, 128), (7, 3, 1, 128, 64), (5, 2, 2, 80, 20), (3, 4, 0, 64, 6), (2, 1, 1, 2, 2), (300, 5, 3, 96, 96),
         (9, 2, 1, 257, 130), (2000, 4, 4, 128, 128), (1, 64, 8, 1024, 1024), (70, 2, 1, 24, 8)]


@pytest.mark.parametrize("T,Hq,Hk,d,rot", SIZES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope(T, Hq, Hk, d, rot, interleaved, dtype, in_place):
    g = torch.Generator().manual_seed(T + d)
    q, k = torch.randn((T, Hq, d), generator=g).to(dtype), torch.randn((T, Hk, d), generator=g).to(dtype)
    positions = torch.randint(-5, 40000, (T,), generator=g)
    freq, _ = libkda.rope_frequencies(rot)
    dq, dk = q.cuda(), k.cuda() if Hk else None
    oq = dq if in_place else torch.full_like(dq, float("nan"))
    ok = None if dk is None else dk if in_place else torch.full_like(dk, float("nan"))
    libkda.kda_rope(dq, dk, positions.to(torch.int32).cuda(), libkda.rope_steps(freq).cuda(), oq, ok, interleaved=interleaved, scale=1.25)
    check(q, oq, positions.numpy(), freq, 1.25, interleaved)
    if Hk:
        check(k, ok, positions.numpy(), freq, 1.25, interleaved)
    if not in_place:
        assert torch.equal(dq.cpu(), q)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Positions up to the ends of 32 bits lose nothing; the fastest pair turns a radian a position."""
    positions = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 10 ** 6, -10 ** 9])
    q = torch.randn((8, 2, 64), generator=torch.Generator().manual_seed(1))
    freq, _ = libkda.rope_frequencies(64)
    out = torch.empty_like(q, device="cuda")
    libkda.kda_rope(q.cuda(), None, torch.tensor(positions, dtype=torch.int32, device="cuda"), libkda.rope_steps(freq).cuda(), out, None,
                    interleaved=interleaved)
    check(q, out, positions, freq, 1.0, interleaved)


def test_turning_back():
    """Negative frequencies undo a rotation, and the rotation's gradient is that."""
    g = torch.Generator().manual_seed(2)
    q = torch.randn((50, 3, 64), generator=g, dtype=torch.float64).float().cuda()
    positions = torch.randint(0, 10 ** 6, (50,), generator=g).to(torch.int32).cuda()
    freq, _ = libkda.rope_frequencies(48)
    there, back = torch.empty_like(q), torch.empty_like(q)
    libkda.kda_rope(q, None, positions, libkda.rope_steps(freq).cuda(), there, None)
    libkda.kda_rope(there, None, positions, libkda.rope_steps(-freq).cuda(), back, None)
    assert (back - q).abs().max() <= 2.0 ** -19 * q.abs().max()
    assert not torch.allclose(there, q)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned_tensors(dtype):
    """Tensors that start between 16-byte boundaries, and outputs beside them that stay as they were."""
    T, H, d = 11, 3, 64
    freq, _ = libkda.rope_frequencies(d)
    store = torch.randn(2 * T * H * d + 8, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    before = store.clone()
    q, out = store[1:1 + T * H * d].view(T, H, d), store[3 + T * H * d:3 + 2 * T * H * d].view(T, H, d)
    q0 = q.clone()
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    libkda.kda_rope(q, None, positions, libkda.rope_steps(freq).cuda(), out, None)
    check(q0.cpu(), out, np.arange(T), freq, 1.0, False)
    out.copy_(before[3 + T * H * d:3 + 2 * T * H * d].view(T, H, d))
    assert torch.equal(store, before)


def test_offsets_past_32_bits():
    T, H, d = 140000, 120, 128
    q = torch.zeros((T, H, d), dtype=BF, device="cuda")
    assert q.numel() > 2 ** 31
    q[-1] = torch.randn((H, d), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(BF)
    last = q[-1:].cpu()
    freq, _ = libkda.rope_frequencies(d)
    libkda.kda_rope(q, None, torch.arange(T, dtype=torch.int32, device="cuda"), libkda.rope_steps(freq).cuda(), q, None)
    check(last, q[-1:], np.array([T - 1]), freq, 1.0, False)
    assert (q[:-1] == 0).all()
    del q
    torch.cuda.empty_cache()


def test_graph_replay():
    q = torch.randn((33, 4, 128), generator=torch.Generator().manual_seed(6)).to(BF).cuda()
    freq, _ = libkda.rope_frequencies(128)
    table, positions, out = libkda.rope_steps(freq).cuda(), torch.zeros(33, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        libkda.kda_rope(q, None, positions, table, out, None)
    positions.copy_(torch.arange(33))
    graph.replay()
    check(q, out, np.arange(33), freq, 1.0, False)


def test_as_many_tokens_as_an_int_counts():
    T = 2 ** 31 - 1
    q, positions = torch.zeros((T, 1, 2), dtype=BF, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    q[-1, 0], positions[-1] = torch.tensor([1.0, 2.0]), 5
    last = q[-1:].cpu()
    freq, _ = libkda.rope_frequencies(2)
    libkda.kda_rope(q, None, positions, libkda.rope_steps(freq).cuda(), q, None)
    check(last, q[-1:], np.array([5]), freq, 1.0, False)
    assert not q[:-1].any()
    del q, positions
    torch.cuda.empty_cache()
