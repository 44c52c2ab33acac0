"""The linear-attention sublayer at its ends: batches without a token, and what the normalisation leaves of the rotary scale."""
import pytest
import torch

from gated_delta_rule_27_gb300 import sublayer

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_no_tokens():
    D, H, d = 256, 2, 128
    w = sublayer.synthetic_linear_weights(D, H, 1, d, 5, "cuda")
    x = torch.zeros((0, D), dtype=torch.bfloat16, device="cuda")
    S0 = torch.randn((2, H, d, d), device="cuda")
    y, S = sublayer.linear_prefill_forward(x, i32([0, 0, 0]), i32([]), w, d, S0=S0)
    assert y.shape == (0, D) and torch.equal(S, S0)
    pool = S0.clone()
    assert sublayer.linear_decode_forward(x, i32([]), pool, i32([]), w, d).shape == (0, D)
    assert torch.equal(pool, S0)
