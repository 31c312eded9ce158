"""The policy loss's sums are 64-bit: terms that cancel leave what is left of them exactly, by both routes."""

import pytest
import torch

from test_sequence_losses_gpu import U, kd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [4, 700])
@pytest.mark.parametrize("reduce", ["token", "sequence"])
def test_cancelling_terms(kd, S, reduce):                                    # noqa: F811
    """logp = old: each token's ratio is exactly 1 and its loss -A.  Of every four advantages two cancel; what is left, 2
    of 2^27, is below half a float32 step of the large ones, and the sums of 300 are exact in float64."""
    N = 300 * S
    lp = torch.full((N,), -1.5, device="cuda")
    adv = torch.tensor([2.0 ** 27, 1.0, -2.0 ** 27, 1.0], device="cuda").repeat(N // 4)
    ref = lp - torch.tensor([2.0 ** 12, 0.25, -2.0 ** 12, 0.25], device="cuda").repeat(N // 4)
    ref = torch.where(ref.abs() > 4000, ref.round(), ref)         # y = lp - ref is exact: halves and quarters
    off = torch.arange(0, N + 1, 300, device="cuda", dtype=torch.int32)
    loss, kl, share, dlogp = kd.policy_loss_forward_backward(lp, lp, adv, ref, offsets=off, kl="k1", reduce=reduce)
    assert float(loss) == pytest.approx(-0.5, rel=2 * U) and float(share) == 0
    y = lp.double() - ref.double()
    assert float(kl) == pytest.approx(float(y.mean()), rel=2 * U)
    assert torch.allclose(dlogp.double() * N, -adv.double(), rtol=4 * U, atol=0)
