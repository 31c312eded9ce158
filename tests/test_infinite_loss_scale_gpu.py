"""An upstream gradient that has overflowed (a loss scale grown too far) reaches the tokens that take part; the masked
ones keep a gradient of 0, as in the calls that are given grad_loss."""

import pytest
import torch

from test_sequence_losses_gpu import kd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [float("inf"), float("nan"), 1e30])
@pytest.mark.parametrize("shift", [0, 1])
def test_masked_tokens_have_no_gradient(kd, scale, shift):                   # noqa: F811
    n = 403
    mask = torch.ones(n + shift, device="cuda")[shift:]
    mask[::3] = 0
    lp = torch.linspace(-3, -1, n + shift, device="cuda")[shift:].clone().requires_grad_(True)
    old, adv = lp.detach() - 0.05, torch.linspace(0.5, 1, n, device="cuda")
    off = torch.tensor([2, 100, 200, 300, n - 1], device="cuda", dtype=torch.int32)
    g = torch.tensor(scale, device="cuda")
    for f in (lambda x: kd.preference_loss(x, old, mask, off)[0], lambda x: kd.policy_loss(x, old, adv, mask=mask, offsets=off)[0]):
        (grad,) = torch.autograd.grad(f(lp), lp, g)
        on = mask != 0
        on[:2] = False
        on[-1] = False
        assert bool((grad[~on] == 0).all())
        assert bool((torch.isfinite(grad[on]) == (abs(scale) < 1e38)).all()) and bool((grad[on] != 0).all())
