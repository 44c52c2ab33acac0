"""The Python binding of the draft-tree calls without a GPU: wrong types, shapes and devices raise before the library is
called."""
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


T, H, D, N, V, C, W = 3, 2, 64, 1, 10, 8, 4
ROWS, POOL = torch.zeros(T, H, D), torch.zeros(2, H, D, D)
CALLS = {
    "kda_tree_step": dict(q=ROWS, k=ROWS, v=ROWS, g=ROWS, beta=torch.zeros(T, H), parent=ints(T), cu_nodes=ints(N + 1),
                          seq_idx=ints(N), S_pool=POOL, o=ROWS, u=ROWS, max_nodes=3),
    "kda_tree_commit": dict(k=ROWS, g=ROWS, u=ROWS, cu_nodes=ints(N + 1), path=ints(N, 3), path_len=ints(N), seq_idx=ints(N),
                            S_pool=POOL),
    "kda_tree_conv": dict(x=torch.zeros(T, C), w=torch.zeros(C, W), parent=ints(T), cu_nodes=ints(N + 1), seq_idx=ints(N),
                          conv_pool=torch.zeros(2, W - 1, C), y=torch.zeros(T, C), max_nodes=3),
    "kda_tree_conv_commit": dict(x=torch.zeros(T, C), cu_nodes=ints(N + 1), path=ints(N, 3), path_len=ints(N), seq_idx=ints(N),
                                 conv_pool=torch.zeros(2, W - 1, C)),
    "kda_draft_verify": dict(logits=torch.zeros(T, V), tokens=ints(T), parent=ints(T), cu_nodes=ints(N + 1),
                             u_accept=torch.zeros(T), u_next=torch.zeros(N), path=ints(N, 3), path_len=ints(N),
                             next_token=ints(N)),
}


@pytest.mark.parametrize("name", CALLS)
def test_refusals(name):
    f, given = getattr(libkda, name), CALLS[name]
    lead = next(iter(given))
    with pytest.raises(ValueError, match="device tensors"):
        f(**given)
    with pytest.raises(TypeError, match="not a tensor"):
        f(**{**given, lead: None})
    with pytest.raises(TypeError, match="bf16 or fp32"):
        f(**{**given, lead: given[lead].double()})
    with pytest.raises(ValueError, match="dimensions"):
        f(**{**given, lead: given[lead].reshape(-1)})
    with pytest.raises(TypeError):
        f()
    # which of several faults is reported is not promised: that every tensor is on the host is one in these calls
    for key, x in given.items():
        for wrong in ([x.tolist(), x.unsqueeze(0)] if torch.is_tensor(x) else ["3", 1 << 40]):
            with pytest.raises((TypeError, ValueError, OverflowError)):
                f(**{**given, key: wrong})
