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


def test_the_normalisation_takes_a_whole_head_s_scale_out():
    """With all of a head turned, a scale of 2 (which no rounding sees) changes no bit; with half of it, the states."""
    D, H, d, T = 256, 2, 128, 100
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    for rot in (d, d // 2):
        w = sublayer.synthetic_linear_weights(D, H, H, d, 5, "cuda", rot=rot)
        y, S = sublayer.linear_prefill_forward(x, i32([0, T]), i32(list(range(T))), w, d, qk_eps=0.0)
        w.rope_scale = 2.0
        y2, S2 = sublayer.linear_prefill_forward(x, i32([0, T]), i32(list(range(T))), w, d, qk_eps=0.0)
        assert torch.equal(S, S2) == torch.equal(y, y2) == (rot == d)
