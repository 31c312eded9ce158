"""Upstream gradients at the bottom of float32: they vanish over the temperature, and leave zeros, not NaN."""

import pytest
import torch

from test_token_logprobs_gpu import _inputs, kd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1.0, 4.0, 1e6])
@pytest.mark.parametrize("value", [2.0 ** -149, -2.0 ** -140, 2.0 ** -126])
def test_denormal_upstream(kd, T, value):                                    # noqa: F811
    H, W, y, g, h = (t.cuda() for t in _inputs(300, 64, 500, 5, "none"))
    g[::2], h[::2] = value, -value
    _, lse, ent = kd.token_logprobs_forward(H, W, y, T, entropy=True)
    for e in ({}, dict(entropy=ent, dentropy=h)):
        dH, dW = kd.token_logprobs_backward(H, W, y, lse, g, T, **e)
        assert bool(torch.isfinite(dH).all()) and bool(torch.isfinite(dW).all())
        # the entries of a row are bounded by (|g| + |h|) (1 + |log p| + ent) / T, below 64 |value|; W's by 2
        assert float(dH[::2].abs().max()) <= 64 * 2 * 64 * abs(value)
        zero = g.clone(), h.clone()
        zero[0][::2], zero[1][::2] = 0.0, 0.0
        e = dict(e, dentropy=zero[1]) if e else e
        dH0, dW0 = kd.token_logprobs_backward(H, W, y, lse, zero[0], T, **e)
        # two bf16 steps: dH's sum may be cut in other places for other row counts
        assert bool(((dH - dH0)[1::2].abs() <= 2.0 ** -6 * dH0[1::2].abs() + 1e-6 / T).all())
        assert bool(((dW - dW0).abs() <= 1e-6 * (1.0 / T) * (1 + dW0.abs() * T)).all())
