"""A linear prefill whose warps do not hear from one another ends by itself, says so and leaves the context usable.

The test hook kda_testing_set_fault keeps the warp that sums a chunk's decays from telling the others, whose waits, a second
each, run out: nothing hangs, nothing faults.
"""
import time

import numpy as np
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from tests.test_gpu_linear import BF, check_prefill, fused_args, i32, inputs, run_prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("lengths", [[77], [1, 0, 900]], ids=str)  # the outputs' kernel alone, and behind the segments'
def test_decays_that_never_come_are_reported(lengths, fused):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(int).tolist()
    x = inputs(cu[-1], 3, 3, 128, BF, 83)
    on = {n: t.cuda() for n, t in x.items()}
    o, S = torch.empty_like(on["v"]), torch.empty((len(lengths), 3, 128, 128), device="cuda")
    ws = libkda.new_linear_workspace(on["q"], on["v"], i32(cu))
    args, more = (on["q"], on["k"], on["v"], on["g"], i32(cu), o), dict(S_final=S, workspace=ws, **fused_args(x, fused))
    torch.cuda.synchronize()
    libkda.testing_set_fault(libkda.FAULT_NO_PUBLISH, 20_000_000)
    try:
        t0 = time.perf_counter()
        libkda.kda_linear_prefill(*args, **more)
        status = libkda.kda_prefill_check(ws)
        elapsed = time.perf_counter() - t0
    finally:
        libkda.testing_set_fault(libkda.FAULT_NONE, 0)
    assert status == libkda.KDA_ERR_TIMEOUT and elapsed < 15.0
    # the same memory takes a call afterwards, and its results are right
    libkda.kda_linear_prefill(*args, **more)
    assert libkda.kda_prefill_check(ws) == libkda.KDA_OK
    ref = run_prefill(x, cu, fused=fused)
    assert torch.equal(o, ref[0]) and torch.equal(S, ref[1])
    check_prefill(lengths, 3, 3, 128, BF, x=x, fused=fused)
