"""The linear-attention sublayer: prompts packed together, then tokens one by one from a pool, against the fp64 operators on
the same projections.

Tolerance (2-norm over a document's outputs): q and k are rounded to bf16 after their rotation, o before its projection,
whose own result is bf16; the scores and the state that form o add two roundings: five of 2^-8 at most, 2^-8 x 5 < 2^-5.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda, sublayer
from oracle import linear
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hqk,rot,scaling", [(4, 4, None, None), (4, 2, 64, {"type": "yarn", "factor": 8, "original_max_position": 256})])
def test_prompts_then_tokens(H, Hqk, rot, scaling):
    D, d, lengths, steps = 256, 128, [100, 1, 333], 3
    w = sublayer.synthetic_linear_weights(D, H, Hqk, d, 5, "cuda", rot=rot, scaling=scaling)
    N, total = len(lengths), [n + steps for n in lengths]
    cu_all = np.concatenate([[0], np.cumsum(total)]).tolist()
    x = torch.randn((cu_all[-1], D), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).cuda()
    positions = torch.tensor(np.concatenate([np.arange(n) for n in total]), dtype=torch.int32, device="cuda")
    prompt = torch.tensor(np.concatenate([np.arange(cu_all[n], cu_all[n] + lengths[n]) for n in range(N)]), device="cuda")
    cu = torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    y[prompt], S = sublayer.linear_prefill_forward(x[prompt], cu, positions[prompt], w, d)
    pool, slots = torch.full((N + 2, H, d, d), float("nan"), device="cuda"), torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    libkda.kda_state_restore(S, slots, pool)
    for t in range(steps):
        rows = torch.tensor([cu_all[n] + lengths[n] + t for n in range(N)], device="cuda")
        y[rows] = sublayer.linear_decode_forward(x[rows], positions[rows], pool, slots, w, d)
    freq, scale = libkda.rope_frequencies(rot or d, scaling=scaling)
    project = lambda m: f64(x @ m).reshape(x.shape[0], -1, d)  # noqa: E731
    q, k = (linear.unit(linear.rope(project(m), positions.cpu().numpy(), freq.numpy(), scale, False).astype(np.float64), 1e-6) for m in (w.W_q, w.W_k))
    g = -np.logaddexp(0, f64(x @ w.W_a))
    o, end, m, _ = linear.attention(q, k, project(w.W_v), g, cu_all)
    o, _ = linear.gated(o, m, project(w.W_z), f64(w.out_weight), 1e-6, 0 * o)
    ref = o.reshape(x.shape[0], -1) @ f64(w.W_o)
    for n in range(N):
        a, b = f64(y)[cu_all[n]:cu_all[n + 1]], ref[cu_all[n]:cu_all[n + 1]]
        assert np.linalg.norm(a - b) <= 2.0 ** -5 * np.linalg.norm(b)
    assert np.linalg.norm(f64(pool[slots.long()]) - end) <= 2.0 ** -5 * np.linalg.norm(end)
