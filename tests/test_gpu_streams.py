"""Calls that allocate for themselves, on a stream that is not the current one."""
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda, workloads
from tests.gpu_helpers import to_device

pytestmark = pytest.mark.gpu


def test_outputs_of_a_call_on_another_stream_used_on_the_current_one():
    """Prefill and decode on a stream, their outputs read on the current one after a wait and let go while that is still to
    come: the next call's outputs must not be given their memory, nor memory that the current stream still uses."""
    inp = workloads.prefill_inputs([300, 77], H=4, d=128, dtype=torch.bfloat16, seed=11, s0_std=0.1)
    x, S0 = to_device(inp), inp.S0.cuda()
    dec = workloads.decode_inputs(1, 2, 4, 128, torch.bfloat16, seed=12)
    step = [t[0].cuda() for t in (dec.q, dec.k, dec.v, dec.g, dec.beta)]
    ref_o, ref_S = libkda.prefill(*x, S0=S0)
    ref_step = libkda.decode_step(*step, ref_S.clone())
    stream, seen = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for _ in range(6):
        before = torch.empty_like(ref_o)
        torch.cuda._sleep(2_000_000)
        before.fill_(1.0)
        del before  # its memory is free in the current stream's order, its work is still to come
        o, S = libkda.prefill(*x, S0=S0, stream=stream)
        with torch.cuda.stream(stream):
            state = S.clone()
        first = libkda.decode_step(*step, state, stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
        torch.cuda._sleep(2_000_000)
        seen.append((o.clone(), S.clone(), first.clone()))
        state.record_stream(torch.cuda.current_stream())
        del o, S, first, state
    torch.cuda.synchronize()
    for o, S, first in seen:
        assert torch.equal(o, ref_o) and torch.equal(S, ref_S) and torch.equal(first, ref_step)
