"""Draft-tree calls on tensors of several devices are refused on the host (tensors without data stand for a second GPU's)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from gated_delta_rule_27_gb300 import libkda
from tests.test_tree_binding_cpu import CALLS


def on(device, x):
    with FakeTensorMode():
        return torch.empty(x.shape, dtype=x.dtype, device=device)


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2, reason="beside a GPU the stand-ins ask for the second one")
@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_two_devices_are_refused(name):
    given = {key: on("cuda:0", x) if torch.is_tensor(x) else x for key, x in CALLS[name].items()}
    for key, x in given.items():
        if torch.is_tensor(x):
            with pytest.raises(ValueError, match="one device; got cuda:"):
                getattr(libkda, name)(**{**given, key: on("cuda:1", x)})
