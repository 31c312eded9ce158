"""The gradient's joint launch in the forms that `dh_plan` chooses for several bands of rows: wide units (two column
tiles) whole and with their K blocks cut, narrow ones cut, with and without dW, by loads (few bands) and by products.

Against the same formulas in 64 bits on the GPU.  Elementwise bounds sum every rounding's worst case, which a missing
range of a long sum could hide in; so the error is also held in the Frobenius norm, where independent roundings of at
most b = 2^-8 of a term (dZ's; H's scaled, for dW) add in squares: dH 2 b sqrt(dZ^2 W^2 summed), dW
2 b sqrt(2 dZ^2 H^2 summed), twice the largest root mean square, plus b of the result where that is rounded to bf16.  A
K range or a column tile left out is a tenth of the norm and more.
"""

import pytest
import torch

from test_token_logprobs_gpu import kd  # noqa: F401

pytestmark = pytest.mark.gpu

B16 = 2.0 ** -8

# live rows, d, V, whether dW is wanted: (column tiles of wide units, K ranges) of the plan with 74 CTA pairs
CASES = [
    (1036, 2880, 500, True),          # wide, whole
    (2394, 2048, 500, True),          # wide, whole, by products
    (260, 264, 36544, True),          # wide, 16 ranges
    (260, 264, 111578, False),        # wide, 33 ranges
    (2394, 776, 6109, False),         # wide, 3 ranges, by products
    (900, 1000, 6000, True),          # narrow, 2 ranges
    (1285, 2880, 20011, True),        # a head's width
]


def _exact(H, W, y, lse, g, h, ent):
    H, W = H.double(), W.double()
    logq = H @ W.T - lse.double()[:, None]
    dz = logq.exp()
    if h is None:
        dz *= -g.double()[:, None]
    else:
        dz *= -(g.double()[:, None] + h.double()[:, None] * (logq + ent.double()[:, None]))
    del logq
    live = y >= 0
    dz[~live] = 0
    dz[live, y[live]] += g.double()[live]
    return dz, dz @ W, dz.T @ H, ((dz * dz) @ (W * W)).sum().sqrt(), ((dz * dz).T @ (H * H)).sum().sqrt()


@pytest.mark.parametrize("rows,d,V,want_dW", CASES)
@pytest.mark.parametrize("form", ["all", "some", "entropy"])
def test_against_64_bits(kd, rows, d, V, want_dW, form):                     # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(rows + V)
    N = rows if form == "all" else rows + 333
    W = (torch.randn(V, d, device="cuda", generator=gen) * d ** -0.5).bfloat16()
    y = torch.randint(0, V, (N,), device="cuda", generator=gen)
    H = (torch.randn(N, d, device="cuda", generator=gen) + 4 * torch.rand(N, 1, device="cuda", generator=gen) *
         W[y].float()).bfloat16()
    y[torch.randperm(N, device="cuda", generator=gen)[:N - rows]] = -1
    g = torch.randn(N, device="cuda", generator=gen)
    h = torch.randn(N, device="cuda", generator=gen) if form == "entropy" else None
    _, lse, ent = kd.token_logprobs_forward(H, W, y, entropy=True)
    e = dict(entropy=ent, dentropy=h) if form == "entropy" else {}
    dz, rH, rW, nH, nW = _exact(H, W, y, lse, g, h, ent)
    for dW_dtype in ((torch.float32, torch.bfloat16) if want_dW else (None,)):
        dH, dW = kd.token_logprobs_backward(H, W, y, lse, g, dW_dtype=dW_dtype, **e)
        assert float((dH.double() - rH).norm()) <= float(2 * B16 * nH + B16 * rH.norm())
        assert not dH[y < 0].any()
        bound = (2 * B16 + 1e-3) * (dz.abs() @ W.double().abs() + rH.abs())
        assert bool(((dH.double() - rH).abs() <= bound).all())
        if dW is not None:
            own = B16 * rW.norm() if dW_dtype == torch.bfloat16 else 0.0
            assert float((dW.double() - rW).norm()) <= float(2 * B16 * 2 ** 0.5 * nW + own)
            bound = (3 * B16 + 1e-3) * (dz.abs().T @ H.double().abs() + rW.abs())
            assert bool(((dW.double() - rW).abs() <= bound).all())
