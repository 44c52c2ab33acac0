"""Linear attention and rotary positions without a GPU: refusals of the C ABI and of the binding, frequencies, and the
numbering of segments that the kernels go by."""
import ctypes
import math

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from gated_delta_rule_27_gb300 import libkda

OK, INVALID, UNSUPPORTED = libkda.KDA_OK, libkda.KDA_ERR_INVALID_ARG, libkda.KDA_ERR_UNSUPPORTED
BF16, F32 = libkda.KDA_BF16, libkda.KDA_F32


def at(i, off=0):
    return ctypes.c_void_p((i << 20) + off)  # never dereferenced: every call below fails its checks first, or has no work


PREFILL = dict(q=at(1), k=at(2), v=at(3), g=at(4), per_token=1, cu=at(5), N=2, T=100, H=4, Hqk=2, dk=128, dv=128, dt=BF16, S0=at(6), o=at(7),
               S=at(8), ws=at(9), wsb=1 << 30, stream=None, opts=None)
DECODE = dict(q=at(1), k=at(2), v=at(3), g=at(4), per_token=1, idx=at(5), N=3, slots=5, H=4, Hqk=2, dk=128, dv=128, dt=BF16, S=at(6), o=at(7),
              status=None, stream=None, opts=None)
ROPE = dict(q=at(1), k=at(2), positions=at(3), steps=at(4), T=10, Hq=4, Hk=2, d=64, rot=32, interleaved=0, scale=1.0, dt=BF16, q_out=at(5), k_out=at(6),
            stream=None)
CALLS = {"kda_linear_prefill": PREFILL, "kda_linear_decode_step": DECODE, "kda_rope": ROPE}


def call(name, **changed):
    assert set(changed) <= set(CALLS[name])
    return getattr(libkda.load(), name)(*{**CALLS[name], **changed}.values())


@pytest.mark.parametrize("name", ["kda_linear_prefill", "kda_linear_decode_step"])
def test_attention_sizes(name):
    rows = "T" if name == "kda_linear_prefill" else "N"
    for bad in (dict(H=0), dict(H=-1), dict(H=65536), dict(Hqk=0), dict(Hqk=3), dict(Hqk=8), dict(dt=7), {rows: -1}, dict(N=-1)):
        assert call(name, **bad) == INVALID, bad
    for bad in (dict(dk=32, dv=32), dict(dk=64), dict(dk=256, dv=256), {rows: 1 << 30, "H": 4, "Hqk": 2}):
        assert call(name, **bad) == UNSUPPORTED, bad
    if name == "kda_linear_prefill":
        assert call(name, N=2 ** 31 - 1, T=0, H=1, Hqk=1) == UNSUPPORTED


@pytest.mark.parametrize("name", CALLS)
def test_pointers(name):
    need = dict(kda_linear_prefill=["q", "k", "v", "g", "cu", "o", "ws"], kda_linear_decode_step=["q", "k", "v", "g", "S", "o"],
                kda_rope=["q", "k", "positions", "steps", "q_out", "k_out"])[name]
    for p in need:
        assert call(name, **{p: None}) == INVALID, p
    for p, x in CALLS[name].items():
        if isinstance(x, ctypes.c_void_p):
            assert call(name, **{p: ctypes.c_void_p(x.value + 1)}) == INVALID, p
    if name == "kda_linear_decode_step":
        assert call(name, status=at(8, 2)) == INVALID


def test_aliases():
    for p in ("q", "k", "v", "g"):
        assert call("kda_linear_prefill", o=PREFILL[p]) == INVALID
        assert call("kda_linear_prefill", S=PREFILL[p]) == INVALID
        assert call("kda_linear_decode_step", o=DECODE[p]) == INVALID
        assert call("kda_linear_decode_step", S=DECODE[p]) == INVALID
    assert call("kda_linear_prefill", S=PREFILL["o"]) == INVALID
    assert call("kda_linear_prefill", o=PREFILL["S0"]) == INVALID
    assert call("kda_linear_decode_step", S=DECODE["o"]) == INVALID
    for wrong in (dict(q_out=ROPE["k"]), dict(k_out=ROPE["q"]), dict(k_out=ROPE["q_out"]), dict(k=ROPE["q"])):
        assert call("kda_rope", **wrong) == INVALID, wrong


def test_fusion_options():
    opts = lambda *a: ctypes.byref(libkda.FusionOpts(*a))  # noqa: E731
    for name in ("kda_linear_prefill", "kda_linear_decode_step"):
        assert call(name, opts=opts(1, -1.0, None, None, 0.0)) == INVALID
        assert call(name, opts=opts(1, float("nan"), None, None, 0.0)) == INVALID
        assert call(name, opts=opts(0, 0.0, 10 << 20, None, 0.0)) == INVALID  # no out_eps
        assert call(name, opts=opts(0, 0.0, (10 << 20) + 8, None, 1e-6)) == INVALID
        assert call(name, opts=opts(0, 0.0, 10 << 20, (11 << 20) + 4, 1e-6)) == INVALID
        assert call(name, opts=opts(0, 0.0, 7 << 20, None, 1e-6)) == INVALID  # the gate in o's place


def test_no_work():
    none = dict(q=None, k=None, v=None, g=None, o=None)
    assert call("kda_linear_prefill", **none, cu=None, N=0, T=0, S0=None, S=None) == OK
    assert call("kda_linear_prefill", N=0) == INVALID  # tokens of no sequence
    assert call("kda_linear_decode_step", **none, N=0) == OK
    assert call("kda_rope", T=0, q=None, k=None, positions=None, steps=None, q_out=None, k_out=None) == OK


def test_rope_sizes():
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hk=-1), dict(Hq=0, Hk=0), dict(d=0), dict(rot=0), dict(rot=3), dict(rot=66), dict(dt=5), dict(Hq=70000)):
        assert call("kda_rope", **bad) == INVALID, bad
    for bad in (dict(d=1026, rot=2), dict(T=1 << 30)):
        assert call("kda_rope", **bad) == UNSUPPORTED, bad


def test_workspace():
    size = libkda.kda_linear_workspace_size
    assert size(100, 2, 16, 128, 128, BF16) >= 256
    assert size(65536, 1, 16, 128, 128, BF16) >= 9 * 16 * 128 * 128 * 4
    assert size(0, 0, 1, 16, 16, F32) > 0
    assert size(100, 2, 16, 32, 32, BF16) == size(100, 2, 16, 128, 64, BF16) == size(-1, 2, 16, 128, 128, BF16) == size(1, -1, 1, 64, 64, F32) == 0
    need = size(65536, 3, 16, 128, 128, BF16)
    big = dict(T=65536, N=3, H=16, Hqk=16)
    assert call("kda_linear_prefill", **big, wsb=need - 1) == INVALID


# ---------------------------------------------------------------------------------------------------------------
# the Python binding
# ---------------------------------------------------------------------------------------------------------------
def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


ROWS, QK = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
GIVEN = {
    "kda_linear_prefill": dict(q=QK, k=QK, v=ROWS, g=torch.zeros(3, 4), cu_seqlens=ints(2), o=ROWS, S0=torch.zeros(1, 4, 64, 64),
                               S_final=torch.zeros(1, 4, 64, 64), workspace=torch.zeros(4096, dtype=torch.uint8)),
    "kda_linear_decode_step": dict(q=QK, k=QK, v=ROWS, g=torch.zeros(4), S_pool=torch.zeros(5, 4, 64, 64), o=ROWS, seq_idx=ints(3), status=ints(1)),
    "kda_rope": dict(q=ROWS, k=QK, positions=ints(3), steps=torch.zeros(16, dtype=torch.int64), q_out=ROWS, k_out=QK),
}


@pytest.mark.parametrize("name", GIVEN)
def test_binding_refuses(name):
    f, given = getattr(libkda, name), GIVEN[name]
    with pytest.raises(ValueError, match="device tensors"):
        f(**given)
    with pytest.raises(TypeError, match="bf16 or fp32"):
        f(**{**given, "q": given["q"].double()})
    with pytest.raises(TypeError):
        f()
    for key, x in given.items():
        for wrong in (x.tolist(), x.unsqueeze(0), x.to(torch.float16)):
            with pytest.raises((TypeError, ValueError)):
                f(**{**given, key: wrong})


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2, reason="beside a GPU the stand-ins ask for the second one")
@pytest.mark.parametrize("name", GIVEN)
def test_tensors_of_two_devices_are_refused(name):
    def on(device, x):
        with FakeTensorMode():
            return torch.empty(x.shape, dtype=x.dtype, device=device)

    given = {key: on("cuda:0", x) for key, x in GIVEN[name].items()}
    for key, x in given.items():
        with pytest.raises(ValueError, match="one device; got cuda:"):
            getattr(libkda, name)(**{**given, key: on("cuda:1", x)})


# ---------------------------------------------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------------------------------------------
def test_steps_are_parts_of_a_turn():
    freq = torch.tensor([0.0, 1.0, -1.0, 2 * math.pi * 0.25, 1e-9, 7.0, 2 * math.pi], dtype=torch.float64)
    steps = [int(s) % 2 ** 64 for s in libkda.rope_steps(freq)]
    for f, s in zip(freq.tolist(), steps):
        turn = (f / (2 * math.pi)) % 1.0
        assert abs(s / 2.0 ** 64 - turn) < 2.0 ** -52 or abs(s / 2.0 ** 64 - turn) > 1 - 2.0 ** -52
    assert steps[0] == 0 and steps[3] == 2 ** 62
    assert (steps[1] + steps[2]) % 2 ** 64 < 4096 or (steps[1] + steps[2]) % 2 ** 64 > 2 ** 64 - 4096
    with pytest.raises(TypeError):
        libkda.rope_steps(freq.float())
    with pytest.raises(TypeError):
        libkda.rope_steps(freq[None])


def test_frequencies():
    plain, scale = libkda.rope_frequencies(128, base=10000.0)
    assert scale == 1.0 and plain[0] == 1.0 and torch.allclose(plain[-1], torch.tensor(10000.0 ** (-126 / 128), dtype=torch.float64))
    linear, _ = libkda.rope_frequencies(128, scaling={"type": "linear", "factor": 4})
    assert torch.allclose(linear * 4, plain)
    ntk, _ = libkda.rope_frequencies(128, scaling={"type": "ntk", "factor": 8})
    assert ntk[0] == 1.0 and math.isclose(plain[-1] / ntk[-1], 8.0)
    yarn, scale = libkda.rope_frequencies(64, scaling={"type": "yarn", "factor": 16, "original_max_position": 4096})
    plain, _ = libkda.rope_frequencies(64)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], plain[turns > 40]) and torch.allclose(yarn[turns < 0.7] * 16, plain[turns < 0.7])
    assert (yarn <= plain).all() and (yarn >= plain / 16).all() and (yarn[1:] < yarn[:-1]).all()
    assert math.isclose(scale, 0.1 * math.log(16) + 1)
    assert libkda.rope_frequencies(2, scaling={"type": "ntk", "factor": 3})[0].tolist() == [1.0]
    for bad in (0, 3, -2):
        with pytest.raises(ValueError):
            libkda.rope_frequencies(bad)
    for bad in ({"type": "other", "factor": 2}, {"type": "linear", "factor": 0.5}):
        with pytest.raises(ValueError):
            libkda.rope_frequencies(8, scaling=bad)


# ---------------------------------------------------------------------------------------------------------------
# segments are numbered without a table
# ---------------------------------------------------------------------------------------------------------------
def find_segment(cu, seg, slot):
    """As the kernels do it: the last document whose first slot is not above it, 32 documents looked at at once."""
    lo, n = 0, len(cu) - 1
    while n > 1:
        step = (n + 31) // 32
        hit = sum(lane * step < n and cu[lo + lane * step] // seg + lo + lane * step <= slot for lane in range(32)) - 1
        lo, n = lo + hit * step, min(step, n - hit * step)
    begin, length = cu[lo], cu[lo + 1] - cu[lo]
    i, count = slot - (begin // seg + lo), (length + seg - 1) // seg if length > seg else 1
    return (lo, begin + i * seg, min(seg, length - i * seg)) if i < count else None


@pytest.mark.parametrize("seed", range(30))
def test_every_segment_has_a_slot(seed):
    r = np.random.default_rng(seed)
    seg = int(r.choice([64, 128, 256]))
    lengths = r.integers(0, r.choice([2, 70, 1000]), size=int(r.choice([1, 2, 31, 32, 33, 100, 1025])))
    lengths[r.random(len(lengths)) < 0.2] = 0
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    slots = cu[-1] // seg + len(lengths)
    got = [find_segment(cu, seg, s) for s in range(slots)]
    want = [(n, cu[n] + i, min(seg, lengths[n] - i)) for n in range(len(lengths)) for i in range(0, max(1, lengths[n]), seg)]
    assert [s for s in got if s] == want
