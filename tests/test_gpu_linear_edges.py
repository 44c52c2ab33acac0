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
    """A prefill of x against the recurrence over q, k in 64 bits."""
    cu, dtype, d = table(lengths), x["v"].dtype, x["v"].shape[-1]
    o, S = run_prefill(x, cu, S0, **more)
    ref_o, ref_S, m, A = linear.attention(q, k, f64(x["v"]), f64(x["g"]), cu, None if S0 is None else f64(S0))
    T, tensor_cores = max(lengths), dtype == BF and d == 128
    sums = (T + 64) * 2.0 ** -23 + 2.0 ** -20
    within(o, ref_o, (sums + (2.0 ** -8 if tensor_cores else 0)) * m + (HALF[dtype] + 2.0 ** -20) * np.abs(ref_o), "o")
    within(S, ref_S, (sums + (3 * T * 2.0 ** -23 if tensor_cores else 0)) * A, "S")


@pytest.mark.parametrize("lengths", [[1], [63], [64], [65], [77], [65, 1, 0, 77, 63], [900]], ids=str)
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_norms_without_an_epsilon(lengths, dtype, d):
    """Rows behind a document have no norm; where the sum of their squares is 0, its inverse root must not reach the state."""
    x = inputs(sum(lengths), 4, 2, d, dtype, 73)
    S0 = 0.1 * torch.randn((len(lengths), 4, d, d), generator=torch.Generator().manual_seed(1))
    check(x, lengths, linear.unit(f64(x["q"]), 0.0), linear.unit(f64(x["k"]), 0.0), S0, qk_l2norm=True, qk_eps=0.0)
