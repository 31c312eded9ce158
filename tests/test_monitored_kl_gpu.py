"""A KL that is only reported (kl_coef 0, the default) does not touch the policy loss or its gradient, however far the
reference is, in 64-bit arithmetic (few sequences) and in 32-bit arithmetic (700 sequences: more than the GPU holds
blocks)."""

import numpy as np
import pytest
import torch

from test_sequence_losses_gpu import kd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [4, 700])
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("reduce", ["token", "sequence"])
def test_reported_kl_leaves_loss_and_gradient_alone(kd, S, kl, reduce):      # noqa: F811
    rng = np.random.default_rng(S)
    N = 300 * S
    c = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()       # noqa: E731
    old = -rng.exponential(1.0, N)
    lp, adv = c(old + 0.1 * rng.standard_normal(N)), c(rng.standard_normal(N))
    ref = lp.clone()
    ref[7::100] += 95.0                       # e^95 overflows float32, e^800 float64
    ref[13::1000] += 800.0
    ref[17::1000] = float("inf")
    off = torch.arange(0, N + 1, 300, device="cuda", dtype=torch.int32)
    plain = kd.policy_loss_forward_backward(lp, c(old), adv, offsets=off, reduce=reduce)
    loss, _, share, dlogp = kd.policy_loss_forward_backward(lp, c(old), adv, ref, offsets=off, kl=kl, reduce=reduce)
    assert torch.equal(loss, plain[0]) and torch.equal(share, plain[2]) and torch.equal(dlogp, plain[3])
    assert bool(torch.isfinite(loss)) and bool(torch.isfinite(dlogp).all())
