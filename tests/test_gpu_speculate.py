"""The speculative rounds (gated_delta_rule_27_gb300/speculate.py) against the same tokens decoded one by one.

The two run their bf16 projections as GEMMs of different sizes, so they agree to the bf16 contract
(max|x - ref| / max|ref| <= 2e-2 on states), not bit for bit.
"""
import pytest
import torch

from gated_delta_rule_27_gb300 import speculate, sublayer
from tests.gpu_helpers import dev, f64, rel

pytestmark = pytest.mark.gpu


def _replay(model, tokens):
    """Decodes one request's tokens in order: the logits after each, and the states at the end."""
    H, d = model.H, model.d
    S = torch.zeros((1, H, d, d), device=dev())
    conv = [torch.zeros((1, sublayer.CONV_W - 1, H * d), device=dev()) for _ in range(3)]
    logits = []
    for t in tokens:
        token = torch.tensor([t], device=dev())
        y = sublayer.decode_forward(model.embed[token], S, conv, model.weights, H, d)
        logits.append(model.target_logits(token, y)[0].float())
    return logits, S, conv


@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_rounds_equal_decoding_token_by_token(temperature):
    model = speculate.Model.random(V=600, H=2, d=128, seed=3, device=dev())
    pools = speculate.Pools(6, model.H, model.d, dev())
    last = torch.tensor([5, 17, 300], dtype=torch.int32, device=dev())
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=dev())
    new, rate = speculate.generate(model, last, slots, pools, rounds=6, temperature=temperature, seed=1)
    assert rate > 1.2  # some drafts are kept
    for n, slot in enumerate(slots.tolist()):
        tokens = [int(last[n])] + new[n]
        logits, S, conv = _replay(model, tokens[:-1])  # the last token is not in the states yet
        assert rel(pools.S[slot], f64(S[0])) <= 2e-2
        for pool, c in zip(pools.conv, conv):
            assert rel(pool[slot], f64(c[0])) <= 2e-2
        if temperature == 0.0:
            for after, token in zip(logits, tokens[1:]):
                assert float(after.max() - after[token]) <= 0.05 * float(after.std())
    untouched = [s for s in range(6) if s not in slots.tolist()]
    assert not pools.S[untouched].any()


def test_the_draft_of_a_deterministic_model_is_always_kept():
    """Without the sublayer's contribution the target is the draft: every round keeps a path to a leaf."""
    model = speculate.Model.random(V=200, H=1, d=128, seed=4, device=dev())
    model.weights.W_o.zero_()
    pools = speculate.Pools(2, 1, 128, dev())
    last = torch.tensor([7, 9], dtype=torch.int32, device=dev())
    _, rate = speculate.generate(model, last, torch.tensor([0, 1], dtype=torch.int32, device=dev()), pools, rounds=8,
                                 shape=(-1, 0, 1, 2), seed=2)
    assert rate > 3.9
