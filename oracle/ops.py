"""float64 statements of the context-free operators, from their definitions.

linattn: the recurrence S_t = g S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t, one
position at a time. linear: y = act(x W^T + bias) + residual.
"""
from __future__ import annotations

import math

import numpy as np


def linattn(q, k, v, log_decay, scale=1.0, state=None, lengths=None):
    """q, k [n][B][H][dk], v [n][B][H][dv] -> (o [n][B][H][dv], zero behind a
    sequence's length; state [B][H][dk][dv] after its last position)."""
    n, B, H, dk = q.shape
    dv = v.shape[-1]
    S = np.zeros((B, H, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    o = np.zeros((n, B, H, dv))
    lens = [n] * B if lengths is None else [min(max(int(x), 0), n) for x in lengths]
    g = np.exp(np.minimum(np.asarray(log_decay, dtype=np.float64), 0.0))
    for b in range(B):
        for h in range(H):
            s = S[b, h]
            for t in range(lens[b]):
                # a decay of 0 drops the past whatever it holds
                s = (g[h] * s if g[h] > 0 else np.zeros_like(s)) + np.outer(k[t, b, h], v[t, b, h])
                o[t, b, h] = scale * (q[t, b, h] @ s)
            S[b, h] = s
    return o, S


def gelu(u):
    return u * 0.5 * (1.0 + np.vectorize(math.erf)(u / math.sqrt(2.0)))


ACTIVATIONS = {
    "none": lambda u: u,
    "gelu": gelu,
    "silu": lambda u: u / (1.0 + np.exp(-u)),
    "relu": lambda u: np.maximum(u, 0.0),
    "tanh": np.tanh,
}


def linear(x, w, bias=None, residual=None, act="none"):
    """y [n][out] = act(x [n][in] @ w [out][in]^T + bias) + residual."""
    u = x @ w.T
    if bias is not None:
        u = u + bias
    u = ACTIVATIONS[act](u)
    return u if residual is None else u + residual
