"""The draft-tree entry points without a GPU: every bad argument is refused on the host, before the device is touched."""
import ctypes

import pytest

from gated_delta_rule_27_gb300 import libkda

OK, INVALID, UNSUPPORTED = libkda.KDA_OK, libkda.KDA_ERR_INVALID_ARG, libkda.KDA_ERR_UNSUPPORTED
BF16 = libkda.KDA_BF16


def at(i):
    return ctypes.c_void_p(i << 20)  # never dereferenced: every call below fails its checks first, or has no work


STEP = dict(q=at(1), k=at(2), v=at(3), g=at(4), beta=at(5), parent=at(6), cu=at(7), idx=at(8), N=2, T=5, max_nodes=4, slots=3, H=2,
            dk=128, dv=128, dt=BF16, S=at(9), o=at(10), u=at(11), status=None, stream=None, opts=None)
COMMIT = dict(k=at(1), g=at(2), u=at(3), cu=at(4), path=at(5), len=at(6), idx=at(7), N=2, T=5, stride=4, slots=3, H=2, dk=128, dv=128,
              dt=BF16, S=at(8), status=None, stream=None, opts=None)
CONV = dict(x=at(1), w=at(2), parent=at(3), cu=at(4), idx=at(5), N=2, T=5, max_nodes=4, slots=3, C=8, W=4, dt=BF16, pool=at(6), y=at(7),
            status=None, stream=None)
CONV_COMMIT = dict(x=at(1), cu=at(2), path=at(3), len=at(4), idx=at(5), N=2, T=5, stride=4, slots=3, C=8, W=4, dt=BF16, pool=at(6),
                   status=None, stream=None)
VERIFY = dict(logits=at(1), probs=at(2), tokens=at(3), parent=at(4), cu=at(5), temperature=at(6), u=at(7), u_next=at(8), N=2, T=5, V=100,
              dt=BF16, stride=4, path=at(9), len=at(10), next=at(11), status=None, stream=None)
CALLS = {"kda_tree_step": STEP, "kda_tree_commit": COMMIT, "kda_tree_conv": CONV, "kda_tree_conv_commit": CONV_COMMIT,
         "kda_draft_verify": VERIFY}


def call(name, **changed):
    assert set(changed) <= set(CALLS[name])
    return getattr(libkda.load(), name)(*{**CALLS[name], **changed}.values())


@pytest.mark.parametrize("name", CALLS)
def test_sizes(name):
    bound = "max_nodes" if "max_nodes" in CALLS[name] else "stride"
    assert call(name, N=-1) == INVALID
    assert call(name, T=-1) == INVALID
    assert call(name, dt=7) == INVALID
    assert call(name, **{bound: 0}) == INVALID
    assert call(name, **{bound: libkda.TREE_MAX_NODES + 1}) == UNSUPPORTED
    assert call(name, N=0) == OK  # nothing to do: no pointer is looked at
    if "H" in CALLS[name]:
        assert call(name, H=0) == INVALID
        assert call(name, dk=96, dv=96) == UNSUPPORTED
        assert call(name, dk=64) == UNSUPPORTED
        assert call(name, T=1 << 30, H=4) == UNSUPPORTED
        assert call(name, slots=1 << 30, H=4) == UNSUPPORTED
    if "C" in CALLS[name]:
        assert call(name, C=0) == INVALID
        assert call(name, W=0) == UNSUPPORTED and call(name, W=9) == UNSUPPORTED
        assert call(name, N=65536) == UNSUPPORTED
    if "V" in CALLS[name]:
        assert call(name, V=0) == INVALID
        assert call(name, V=(1 << 22) + 1) == UNSUPPORTED
        assert call(name, N=1 << 29) == UNSUPPORTED


@pytest.mark.parametrize("name", CALLS)
def test_pointers(name):
    optional = {"kda_tree_step": {"idx", "u"}, "kda_tree_commit": {"idx"}, "kda_tree_conv": {"idx"}, "kda_tree_conv_commit": {"idx"},
                "kda_draft_verify": {"probs", "temperature"}}[name]
    for arg, value in CALLS[name].items():
        if isinstance(value, ctypes.c_void_p):
            if arg not in optional:
                assert call(name, **{arg: None}) == INVALID, arg
            assert call(name, **{arg: ctypes.c_void_p(value.value + 1)}) == INVALID, arg  # misaligned
    assert call(name, status=ctypes.c_void_p(0x1002)) == INVALID


def test_aliases_and_options():
    for out in ("o", "u"):
        for source in ("q", "k", "v", "g", "beta", "S"):
            assert call("kda_tree_step", **{out: STEP[source]}) == INVALID
    assert call("kda_tree_step", o=at(11)) == INVALID  # o = u
    assert call("kda_tree_commit", S=COMMIT["u"]) == INVALID
    assert call("kda_tree_conv", y=CONV["x"]) == INVALID
    assert call("kda_tree_conv", y=CONV["pool"]) == INVALID
    opts = lambda *a: ctypes.byref(libkda.FusionOpts(*a))
    assert call("kda_tree_step", opts=opts(1, -1.0, None, None, 0.0)) == INVALID
    assert call("kda_tree_step", opts=opts(0, 0.0, 16 << 20, None, 0.0)) == INVALID      # out_eps must be positive
    assert call("kda_tree_step", opts=opts(0, 0.0, 10 << 20, None, 1e-6)) == INVALID     # the gate is o
    assert call("kda_tree_commit", opts=opts(1, float("nan"), None, None, 0.0)) == INVALID


def test_the_binding_knows_the_header():
    with open(libkda._build.INCLUDE + "/kda.h") as f:
        assert "#define KDA_TREE_MAX_NODES %d\n" % libkda.TREE_MAX_NODES in f.read()
