"""The losses' outputs are tensors of their own: a training loop may change the loss or a reported value in place
before it goes backward."""

import pytest
import torch

from test_sequence_losses_gpu import kd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["preference", "policy"])
def test_outputs_can_be_changed_in_place(kd, which):                         # noqa: F811
    lp = torch.linspace(-3, -1, 400, device="cuda").reshape(4, 100).requires_grad_(True)
    old, adv = lp.detach() - 0.05, torch.linspace(-1, 1, 400, device="cuda").reshape(4, 100)

    def call():
        if which == "preference":
            return kd.preference_loss(lp, old)
        return kd.policy_loss(lp, old, adv, ref_logp=old, kl_coef=0.1)
    (want,) = torch.autograd.grad(call()[0], lp)
    loss, a, b = call()
    first = [t.detach().clone() for t in (loss, a, b)]
    a.mul_(2)                                             # reported values
    assert torch.equal(loss, first[0]) and torch.equal(b, first[2])
    b.add_(1)
    assert torch.equal(a, 2 * first[1])
    loss /= 2                                             # gradient accumulation
    loss += 1.0
    loss.backward()
    assert torch.equal(lp.grad, want / 2)
    assert all(not t._is_view() for t in call())
