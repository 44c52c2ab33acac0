"""Linear attention's binding and limits where they went wrong once, without a GPU."""
import contextlib
import types

import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from tests.test_linear_cpu import GIVEN


@pytest.mark.parametrize("given", [False, True])
def test_a_workspace_is_the_stream_s_own(monkeypatch, given):
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
    monkeypatch.setattr(libkda, "new_linear_workspace", allocate)
    args = {**GIVEN["kda_linear_prefill"], "workspace": None}
    with pytest.raises(ValueError, match="device tensors"):  # (the binding's answer to tensors on the host)
        libkda.kda_linear_prefill(**args, stream=stream if given else None)
    assert taken == [stream if given else None] and not current
