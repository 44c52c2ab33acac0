"""The binding and its limits where they went wrong once, without a GPU."""
import contextlib
import ctypes
import types

import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from tests.test_linear_cpu import GIVEN, PREFILL, call


Q = torch.zeros(3, 4, 64)
DELTA = dict(q=Q, k=Q, v=Q, g=Q, beta=torch.zeros(3, 4), cu_seqlens=torch.zeros(2, dtype=torch.int32), o=Q)
CALLS = {"kda_linear_prefill": ("new_linear_workspace", {**GIVEN["kda_linear_prefill"], "workspace": None}),
         "kda_prefill_chunked": ("new_workspace", DELTA), "kda_prefill_chunked_ex": ("new_workspace", DELTA),
         "kda_prefill_chunked_profiled": ("new_workspace", {**DELTA, "events": []})}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [False, True])
def test_a_workspace_is_the_stream_s_own(monkeypatch, name, given):
    """Scratch that a call takes for itself is allocated with the call's stream as the current one."""
    current, taken, stream = [], [], types.SimpleNamespace(cuda_stream=1)

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def allocate(*args):
        taken.append(current[-1] if current else None)
        return torch.zeros(256, dtype=torch.uint8)

    monkeypatch.setattr(torch.cuda, "stream", on)
    allocator, args = CALLS[name]
    monkeypatch.setattr(libkda, allocator, allocate)
    with pytest.raises((ValueError, IndexError)):  # (the binding's answers to tensors on the host, and to no events)
        getattr(libkda, name)(**args, stream=stream if given else None)
    assert taken == [stream if given else None] and not current


@pytest.mark.parametrize("name,outputs", [("prefill", 2), ("decode_step", 1)])
def test_outputs_are_the_stream_s_own(monkeypatch, name, outputs):
    """Allocated as the call's stream's, and kept until the work that the current stream then has with them is done."""
    current, taken, kept = [], [], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def noted(allocate):
        return lambda *args, **kw: (taken.append(current[-1] if current else None), allocate(*args, **kw))[1]

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(libkda, "kda_prefill_chunked", lambda *args, **kw: None)
    monkeypatch.setattr(libkda, "kda_decode_step", lambda *args, **kw: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: kept.append(s))
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, noted(getattr(torch, f)))
    getattr(libkda, name)(Q, Q, Q, Q, torch.zeros(3, 4), torch.zeros(2, dtype=torch.int32), stream="one")
    assert taken == ["one"] * outputs and kept == ["current"] * outputs


@pytest.mark.parametrize("T", [64, 700])
@pytest.mark.parametrize("third", ["there", "missing", "another row's", "another token's"])
def test_what_the_state_s_tolerance_tells_apart(third, T):
    """The decayed v in three bf16 parts, as the tensor cores take it, in 64-bit sums: all 24 bits are well within the
    tolerance of the state's test on the GPU, and a third part that is missing or out of place is well outside."""
    from tests.test_gpu_linear_edges import STATE, inputs

    x = inputs(T, 1, 1, 128, torch.bfloat16, 103)
    k, v, g = x["k"][:, 0].double(), x["v"][:, 0].float(), x["g"][:, 0].double()
    w = torch.exp(g.sum() - g.cumsum(0))
    y = v * w.float()[:, None]
    bf16 = lambda t: t.to(torch.bfloat16).float()  # noqa: E731
    high = bf16(y)
    middle = bf16(y - high)
    low = bf16(y - high - middle)
    low = {"there": low, "missing": 0 * low, "another row's": low.roll(8, 1), "another token's": low.roll(1, 0)}[third]
    ref = k.T @ (v.double() * w[:, None])
    off = (k.T @ (high.double() + middle.double() + low.double()) - ref).norm() / ref.norm()
    assert off < STATE / 4 if third == "there" else off > 2 * STATE, off


def test_the_final_state_in_the_gate_s_place_is_refused():
    gated = lambda gate: ctypes.byref(libkda.FusionOpts(0, 0.0, gate, None, 1e-6))  # noqa: E731
    assert call("kda_linear_prefill", opts=gated(PREFILL["S"].value)) == libkda.KDA_ERR_INVALID_ARG


def test_token_counts_that_leave_an_int_when_rounded_up_are_refused():
    for d, dtype in ((16, libkda.KDA_BF16), (64, libkda.KDA_F32), (128, libkda.KDA_BF16)):
        most = 2 ** 31 - 1
        assert call("kda_linear_prefill", T=most, N=1, H=1, Hqk=1, dk=d, dv=d, dt=dtype) == libkda.KDA_ERR_UNSUPPORTED
        assert libkda.kda_linear_workspace_size(most, 1, 1, d, d, dtype) == 0
        assert libkda.kda_linear_workspace_size(most - 2 ** 24, 1, 1, d, d, dtype) > 0
