"""fp64 CPU oracle of the label log-probabilities at the LM head.

TEST INFRASTRUCTURE ONLY (like ``kd_oracle``): used by ``tests/`` alone; the
CUDA library never imports it and shares no code with it.  The tests hold the
gradient against central differences.
"""

from __future__ import annotations

import numpy as np

from .kd_oracle import as_f64

__all__ = ["token_logprobs", "token_logprobs_grad"]


def _logq(H, W, T):
    z = as_f64(H) @ as_f64(W).T / T
    m = z.max(axis=1, keepdims=True)
    return z, z - (m + np.log(np.exp(z - m).sum(axis=1, keepdims=True)))


def token_logprobs(H, W, labels, T=1.0):
    """(logp, lse, entropy) per token, 0 where the label is negative."""
    y = np.asarray(labels)
    z, logq = _logq(H, W, T)
    live = y >= 0
    rows = np.arange(len(y))
    col = np.where(live, y, 0)
    lse = (z - logq)[:, 0]
    return (np.where(live, logq[rows, col], 0.0), np.where(live, lse, 0.0),
            np.where(live, -(np.exp(logq) * logq).sum(axis=1), 0.0))


def token_logprobs_grad(H, W, labels, dlogp, dent=None, T=1.0):
    """(dH, dW, dZ) of sum_n dlogp_n logp_n + dent_n entropy_n."""
    y = np.asarray(labels)
    _, logq = _logq(H, W, T)
    live = y >= 0
    p = np.exp(logq)
    g = np.where(live, np.asarray(dlogp, np.float64), 0.0)[:, None]
    dz = -g * p
    if dent is not None:
        h = np.where(live, np.asarray(dent, np.float64), 0.0)[:, None]
        dz -= h * p * (logq - (p * logq).sum(axis=1, keepdims=True))
    dz[np.arange(len(y)), np.where(live, y, 0)] += g[:, 0]
    dz /= T
    return dz @ as_f64(W), dz.T @ as_f64(H), dz
