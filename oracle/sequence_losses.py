"""fp64 CPU oracle of the losses over token log-probabilities.

TEST INFRASTRUCTURE ONLY (like ``kd_oracle``): used by ``tests/`` alone; the
CUDA library never imports it and shares no code with it.

The losses are written out token by token from their definitions (the pages
the distillation loss follows describe neither), each with its gradient in
closed form; the tests hold the gradients against central differences.

``bounds`` is a list of (begin, end) token ranges, one for each sequence.
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["preference_loss", "policy_loss"]


def _softplus(v: float) -> float:
    return max(v, 0.0) + math.log1p(math.exp(-abs(v)))


def _sigmoid(v: float) -> float:
    return 1.0 / (1.0 + math.exp(-v)) if v >= 0 else math.exp(v) / (1.0 + math.exp(v))


def preference_loss(logp, ref, mask, bounds, beta=0.1, kind="sigmoid", label_smoothing=0.0, margin=0.0, average=False):
    """(loss, chosen rewards, rejected rewards, dloss/dlogp)."""
    lp = np.asarray(logp, np.float64).ravel()
    m = np.ones_like(lp) if mask is None else np.asarray(mask, np.float64).ravel()
    rf = np.zeros_like(lp) if ref is None else np.asarray(ref, np.float64).ravel()
    r, w = [], []
    for b, e in bounds:
        on = [t for t in range(b, e) if m[t] != 0]
        n = math.fsum(m[t] for t in on)
        scale = (1.0 / n if n != 0 else 0.0) if average else 1.0
        r.append(scale * math.fsum(m[t] * (lp[t] - rf[t]) for t in on))
        w.append(scale)
    P = len(bounds) // 2
    total, grad = [], np.zeros_like(lp)
    for i in range(P):
        delta = r[i] - r[P + i]
        D = beta * delta - margin
        if kind == "sigmoid":
            total.append((1 - label_smoothing) * _softplus(-D) + label_smoothing * _softplus(D))
            slope = beta * (_sigmoid(D) - (1 - label_smoothing))
        elif kind == "hinge":
            total.append(max(0.0, 1.0 - D))
            slope = -beta if D < 1.0 else 0.0
        else:
            e = delta - margin - 1.0 / (2.0 * beta)
            total.append(e * e)
            slope = 2.0 * e
        for s, sign in ((i, 1.0), (P + i, -1.0)):
            b, e = bounds[s]
            for t in range(b, e):
                if m[t] != 0:
                    grad[t] += sign * slope * w[s] * m[t] / P
    loss = math.fsum(total) / P if P else 0.0
    return loss, beta * np.array(r[:P]), beta * np.array(r[P:]), grad


def policy_loss(logp, old, adv, ref, mask, bounds, clip_low=0.2, clip_high=0.2, dual_clip=None, kl_coef=0.0, kl="k3",
                reduce="token"):
    """(loss, KL, clipped share, dloss/dlogp); ``adv`` per token."""
    lp = np.asarray(logp, np.float64).ravel()
    od = np.asarray(old, np.float64).ravel()
    av = np.asarray(adv, np.float64).ravel()
    rf = None if ref is None else np.asarray(ref, np.float64).ravel()
    m = np.ones_like(lp) if mask is None else np.asarray(mask, np.float64).ravel()
    sums = [math.fsum(m[b:e]) for b, e in bounds]
    whole = math.fsum(sums)
    S = len(bounds)
    hi, lo = math.log1p(clip_high), math.log1p(-clip_low)
    out, grad = [[], [], []], np.zeros_like(lp)
    for s, (b, e) in enumerate(bounds):
        for t in range(b, e):
            if m[t] == 0:
                continue
            if reduce == "token":
                w = m[t] / whole if whole != 0 else 0.0
            else:
                w = m[t] / (S * sums[s]) if sums[s] != 0 else 0.0
            A, x = av[t], lp[t] - od[t]
            clipped, d = 0.0, 0.0
            if A == 0:
                obj = 0.0
            elif A > 0 and x > hi:
                obj, clipped = (1 + clip_high) * A, 1.0
            elif A < 0 and x < lo:
                obj, clipped = (1 - clip_low) * A, 1.0
            elif A < 0 and dual_clip is not None and x > math.log(dual_clip):
                obj, clipped = dual_clip * A, 1.0
            else:
                obj = math.exp(x) * A
                d = -obj
            k = dk = 0.0
            if rf is not None:
                y = lp[t] - rf[t]
                if kl == "k1":
                    k, dk = y, 1.0
                elif kl == "k2":
                    k, dk = y * y / 2, y
                else:
                    k, dk = math.expm1(-y) + y, -math.expm1(-y)
            out[0].append(w * (kl_coef * k - obj))
            out[1].append(w * k)
            out[2].append(w * clipped)
            grad[t] += w * (d + kl_coef * dk)
    return math.fsum(out[0]), math.fsum(out[1]), math.fsum(out[2]), grad
