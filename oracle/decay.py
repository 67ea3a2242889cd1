"""Float64 oracles of the decayed linear attention and of the rotary embedding (test infrastructure).

Plain numpy, straight from the definitions and sharing nothing with the CUDA path:

    S_n = g_h S_{n-1} + k_n^T v_n,   o_n = scale * q_n S_n,   g_h = exp(log_decay[h])

one token at a time; a pair (2j, 2j+1) of an axis section of `d_a` features turns by
p_a * theta^(-2j/d_a).
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import numpy as np


def decay_attention(q, k, v, log_decay, scale: float = 1.0, S: Optional[np.ndarray] = None,
                    lengths: Optional[Sequence[int]] = None) -> Tuple[np.ndarray, np.ndarray]:
    """(o, final states) of q, k, v [B, H, N, d] and entering states S [B, H, d, d] (None: zeros);
    rows of o from a batch row's length on are zeros, and its state stops there."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, H, N, d = q.shape
    g = np.exp(np.asarray(log_decay, np.float64)).reshape(1, H, 1, 1)
    S = np.zeros((B, H, d, d)) if S is None else np.array(S, np.float64)
    L = np.full(B, N) if lengths is None else np.asarray(lengths)
    o = np.zeros_like(q)
    for n in range(N):
        on = n < L
        if not on.any():
            break
        S[on] = g * S[on] + k[on, :, n, :, None] * v[on, :, n, None, :]
        o[on, :, n] = scale * np.einsum("bhi,bhij->bhj", q[on, :, n], S[on])
    return o, S


def rope_positions(T: int, Hg: int, Wg: int, t0: int = 0) -> np.ndarray:
    """(t, y, x) of the tokens of a latent grid, t-major, then y, then x: [N, 3]."""
    return np.array([(t0 + t, y, x) for t in range(T) for y in range(Hg) for x in range(Wg)], np.int64).reshape(-1, 3)


def rope(x, positions, split: Sequence[int], theta: float = 1e4, inverse: bool = False) -> np.ndarray:
    """x [B, H, N, d] rotated; positions [N, 3] or [B, N, 3]."""
    y = np.array(x, np.float64)
    pos = np.asarray(positions, np.float64)
    pos = pos[None] if pos.ndim == 2 else pos
    at = 0
    for axis, n in enumerate(split):
        for j in range(n // 2):
            w = pos[:, None, :, axis] * float(theta) ** (-2.0 * j / n)
            c, s = np.cos(w), -np.sin(w) if inverse else np.sin(w)
            a, b = y[..., at].copy(), y[..., at + 1].copy()
            y[..., at], y[..., at + 1] = a * c - b * s, a * s + b * c
            at += 2
    return y
