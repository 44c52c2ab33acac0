"""fp64 references of linear attention with one decay per head, and of rotary positions.

TEST INFRASTRUCTURE ONLY: tests may use this module; the library path never does, and nothing here is shared with
the CUDA code.  Each function goes by its operator's definition, token by token:

  attention  S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t
  rope       pair (x, y) of a token at position p turned by p x frequency

`attention` also gives, for every output and state element, the same sums over absolute values: what a rounding of
the terms can change is a multiple of those.
"""
from __future__ import annotations

import numpy as np


def unit(x, eps):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + eps)


def attention(q, k, v, g, cu, S0=None):
    """q, k [T, Hqk, d], v [T, H, d], g [T, H] or [H] -> o [T, H, d], S [N, H, d, d], and both over absolute values."""
    q, k, v, g = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g))
    T, H, d = v.shape
    N = len(cu) - 1
    of = np.arange(H) // (H // q.shape[1])
    q, k = q[:, of], k[:, of]
    decay = np.broadcast_to(np.exp(g), (T, H))
    S = np.zeros((N, H, d, d)) if S0 is None else np.array(S0, dtype=np.float64)
    A = np.abs(S)
    o, m = np.zeros((T, H, d)), np.zeros((T, H, d))
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            S[n] = decay[t][:, None, None] * S[n] + k[t][:, :, None] * v[t][:, None, :]
            A[n] = decay[t][:, None, None] * A[n] + np.abs(k[t])[:, :, None] * np.abs(v[t])[:, None, :]
            o[t] = (q[t][:, None] @ S[n])[:, 0]
            m[t] = (np.abs(q[t])[:, None] @ A[n])[:, 0]
    return o, S, m, A


def gated(o, m, z, weight, eps, loose):
    """The gated normalisation of o, and how far it may be off where o may be by `loose` (an array)."""
    z = np.asarray(z, dtype=np.float64)
    rms = np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    scale = (1.0 if weight is None else np.asarray(weight, dtype=np.float64)) / (1 + np.exp(-z)) / rms
    off_rms = np.sqrt((loose * loose).mean(-1, keepdims=True)) / rms
    return o * scale, (loose + np.abs(o) * off_rms) * np.abs(scale)


def rope(x, positions, freq, scale, interleaved):
    """x [T, H, d] turned by positions [T] and frequencies [rot / 2], in the widest floats there are."""
    x, freq = np.asarray(x, dtype=np.longdouble), np.asarray(freq, dtype=np.longdouble)
    angle = np.asarray(positions, dtype=np.longdouble)[:, None] * freq
    cos, sin = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
    half = freq.shape[0]
    y = x.copy()
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
    y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
    return y
