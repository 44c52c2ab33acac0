"""Speculative rounds that have nothing to go on with."""
import pytest
import torch

from gated_delta_rule_27_gb300 import speculate
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def test_a_model_without_a_distribution_is_reported():
    """Logits that are all NaN give no next token; the rounds stop there instead of going on from row -1 of the embedding."""
    model = speculate.Model.random(V=100, H=1, d=128, seed=4, device=dev())
    pools = speculate.Pools(2, 1, 128, dev())
    model.weights.W_o[:] = float("nan")  # the draft, which has no sublayer, is sound
    last, slots = (torch.tensor(x, dtype=torch.int32, device=dev()) for x in ([7, 9], [0, 1]))
    with pytest.raises(ValueError, match="request 0: no token"):
        speculate.generate(model, last, slots, pools, rounds=2, seed=2)


@pytest.mark.parametrize("requests,rounds", [(2, 0), (0, 2), (0, 0)])
def test_nothing_to_do(requests, rounds):
    """No rounds, or no requests: no tokens, at a rate of zero."""
    model = speculate.Model.random(V=100, H=1, d=128, seed=4, device=dev())
    pools = speculate.Pools(2, 1, 128, dev())
    ids = torch.arange(requests, dtype=torch.int32, device=dev())
    assert speculate.generate(model, ids, ids, pools, rounds=rounds, seed=2) == ([[]] * requests, 0.0)
    assert not pools.S.any()
