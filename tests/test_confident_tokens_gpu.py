"""Labels that the head is nearly sure of: logp and 1 - p keep their relative precision down to 1 - p = 1e-9, going
forward and back.

W = I and hidden states with the exact logits in them: z[n, v] = H[n, v], no products to round.  Relative tolerances,
u = 2^-24: an exponent x in log2 units is rounded to |x| u, with |x| <= 64 here, 64 ln 2 u, twice (the column's and the
label's); ex2 2^-22, the sum of V = 64 terms 64 u, log1p, expm1, the division and the products 16 u; the logits' scale,
1 + 6e-8, moves a logit of up to 32 by 32 u.  Together below 256 u = 1.6e-5: FWD.  A dH element of the label's column
is scale * -1 * W in fp32, rounded to bf16 (2^-8); another column's p is rounded to bf16 before it (2^-8 again).
"""

import pytest
import torch

from test_token_logprobs_gpu import kd  # noqa: F401

pytestmark = pytest.mark.gpu

FWD, B16 = 256 * 2.0 ** -24, 2.0 ** -8
V = 64


def _inputs(N, seed, T):
    """H [N, V] (bf16 values), labels: margins from 6 to 26 over the other logits, in sixteenths."""
    gen = torch.Generator().manual_seed(seed)
    H = (torch.randint(-16, 17, (N, V), generator=gen) / 16).double()
    y = torch.randint(0, V, (N,), generator=gen)
    H[torch.arange(N), y] = T * (6 + torch.arange(N) % 21).double()
    H = H.bfloat16()
    return H.cuda(), torch.eye(V).bfloat16().cuda(), y.cuda()


def _exact(H, y, T):
    z = H.double() / T
    at = torch.zeros_like(z).scatter_(1, y[:, None], 1.0) != 0
    r = (z - z.gather(1, y[:, None])).exp().masked_fill(at, 0.0)         # the others beside the label
    s = r.sum(1)
    p = r / (1 + s[:, None])
    logp = -torch.log1p(s)
    gap = torch.where(at, 0.0, z - z.gather(1, y[:, None]))              # log p - log p of the label
    ent = -logp - (p * gap).sum(1)
    return at, s / (1 + s), p, logp, ent, gap


@pytest.mark.parametrize("N", [5, 8, 12, 60, 300])
@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("entropy", [False, True])
def test_forward(kd, N, T, entropy):                                         # noqa: F811
    H, W, y = _inputs(N, N, T)
    logp, lse, ent = kd.token_logprobs_forward(H, W, y, T, entropy=entropy)
    _, _, _, want, went, _ = _exact(H, y, T)
    assert float((logp.double() / want - 1).abs().max()) <= FWD
    assert float((lse.double() / (H.double() / T).logsumexp(1) - 1).abs().max()) <= 8 * 2.0 ** -24
    if entropy:
        assert float((ent.double() / went - 1).abs().max()) <= 2 * FWD


@pytest.mark.parametrize("N", [5, 60, 300])
@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("raw", [False, True])
def test_gradient(kd, N, T, raw):                                            # noqa: F811
    H, W, y = _inputs(N, N + 1, T)
    g = torch.linspace(-2, 1, N, device="cuda")
    if raw:
        logp, lse, _ = kd.token_logprobs_forward(H, W, y, T)
        dH, dW = kd.token_logprobs_backward(H, W, y, lse, g, T, logp=logp)
    else:
        H.requires_grad_(True)
        W.requires_grad_(True)
        dH, dW = torch.autograd.grad(kd.token_logprobs(H, W, y, T=T), (H, W), g)
    at, om, p, _, _, _ = _exact(H.detach(), y, T)
    dz = torch.where(at, om[:, None], -p) * g.double()[:, None] / T
    assert float((dH.double() - dz).abs().div(dz.abs()).nan_to_num(0.0)[at].max()) <= B16 * (1 + FWD) + 2 * FWD
    tol = (2 * B16 + B16 * B16 + 2 * FWD) * dz.abs() + 2.0 ** -149
    assert bool(((dH.double() - dz).abs() <= tol).all())
    # dW = dZ^T H: dZ and scale H rounded to bf16, and the result (autograd's dW is bf16)
    want, size = dz.T @ H.detach().double(), dz.abs().T @ H.detach().double().abs()
    assert bool(((dW.double() - want).abs() <= (3.1 * B16 + 2 * FWD) * size + 2.0 ** -149).all())


@pytest.mark.parametrize("N", [5, 60, 300])
def test_entropy_gradient(kd, N):                                            # noqa: F811
    """The label's entry, g (1 - p) - h p (logp + ent), is of the size of 1 - p too.  Its terms' relative errors are 2 FWD
    each (expm1's and the entropy's), taken without the cancellation between them; it is rounded to bf16 as dZ, unless
    the row is scaled by it, and as dH."""
    H, W, y = _inputs(N, N + 2, 1.0)
    g, h = torch.linspace(-2, 1, N, device="cuda"), torch.linspace(1, 3, N, device="cuda")
    H.requires_grad_(True)
    logp, ent = kd.token_logprobs(H, W, y, entropy=True)
    (dH,) = torch.autograd.grad((logp, ent), H, (g, h))
    at, om, p, lp, en, gap = _exact(H.detach(), y, 1.0)
    pl = 1 - om
    gd, hd = g.double(), h.double()
    label = gd * om - hd * pl * (lp + en)
    size = gd.abs() * om + hd * pl * (lp.abs() + en)
    got = dH.double()[at]
    assert bool(((got - label).abs() <= 2.01 * B16 * label.abs() + 4 * FWD * size).all())
