"""A verification whose CTAs do not hear from one another ends by itself, says so and leaves the context usable.

The test hook kda_testing_set_fault keeps the last CTA of each request from sending anything, with a short (20 ms) bound
on the others' waits for it: nothing hangs, nothing faults, the waits simply run out.
"""
import time

import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from tests.test_gpu_tree import BF, F32, check_verify, run_verify, verify_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,dtype", [(20000, BF), (50001, BF), (9000, F32)])  # eight CTAs a request
def test_an_exchange_that_never_comes_is_reported(V, dtype):
    x = verify_inputs([6, 3, 0, 9], V, dtype, 7, True)
    libkda.testing_set_fault(libkda.FAULT_NO_PUBLISH, 20_000_000)
    try:
        t0 = time.perf_counter()
        path, length, token, status = run_verify(x, 9)
        elapsed = time.perf_counter() - t0
    finally:
        libkda.testing_set_fault(libkda.FAULT_NONE, 0)
    assert status == libkda.KDA_ERR_TIMEOUT and elapsed < 10.0
    assert length == [0] * 4 and token == [-1] * 4 and path == [[-1] * 9] * 4
    check_verify(x, 9)  # the next call is right
