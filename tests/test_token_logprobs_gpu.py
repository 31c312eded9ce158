"""Label log-probabilities and their gradients on the GPU against the fp64 oracle.

Tolerances, elementwise, with u = 2^-24 and half a bf16 step b = 2^-8:
* z: an fp32 sum of exact bf16 products, d / 16 accumulations that may truncate
  (2^-23 each) of at most sum_j |H W| / T: delta.
* s, the sum of 2^u: 2^-22 for ex2, 30 u for its argument, and V / 64 + 64
  sequential additions; in lse these are absolute, beside u of |lse|.
* logp: 2 delta, the above, and u of its terms.
* entropy: the same relative error on t / s, and delta times sum p |log p + ent|.
* dZ: b of it, and p's error (2 delta + that of lse + 2^-20) times |g| + |h|
  (|log p| + ent + 1); the products sum it over |W| or |H| with fp32
  accumulation (K / 16 2^-23), and are rounded to bf16 (b) or kept in fp32.
  In dW's product H, times the row's scale, is rounded to bf16 too: another b of
  every term.
"""

import sys

import numpy as np
import pytest
import torch

import oracle
from oracle.logprobs import _logq

pytestmark = pytest.mark.gpu

U, B16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def kd():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from chunked_top_kl_b200 import build
    build.build()
    import chunked_top_kl_b200 as k
    return k


def _inputs(N, d, V, seed, ignored, i64=True, pull=6.0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, d, generator=g) * d ** -0.5).bfloat16()
    y = torch.randint(0, V, (N,), generator=g)
    H = (torch.randn(N, d, generator=g) + pull * torch.rand(N, 1, generator=g) * W[y].float()).bfloat16()
    if ignored == "some":
        y[torch.rand(N, generator=g) < 0.4] = -1
        y[N // 2:N // 2 + 3] = -100
    elif ignored == "all":
        y[:] = -100
    return H, W, y if i64 else y.int(), torch.randn(N, generator=g) / N, torch.randn(N, generator=g) / N


def _f64(t):
    return t.detach().double().cpu().numpy()


def _near(got, want, tol, what):
    got = _f64(got)
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - want) - tol
    assert np.all(over <= 0), (what, float(over.max()), got.ravel()[over.argmax()], want.ravel()[over.argmax()])


def _bounds(H, W, T):
    """delta (of z) and the relative error of s, per token."""
    Hn, Wn = np.abs(_f64(H)), np.abs(_f64(W))
    d, V = Hn.shape[1], Wn.shape[0]
    delta = ((d / 16 + 4) * 2 * U * (Hn @ Wn.T).max(axis=1)) / T if Hn.size else np.zeros(len(Hn))
    return delta, 4 * U + 30 * U + (V / 64 + 64) * U


def _check_forward(out, H, W, y, T):
    logp, lse, ent = oracle.token_logprobs(H, W, y.numpy(), T)
    live = y.numpy() >= 0
    delta, rel = _bounds(H, W, T)
    _near(out[0], logp, np.where(live, 2 * delta + rel + 4 * U * (1 + np.abs(logp) + np.abs(lse)), 0.0), "logp")
    _near(out[1], lse, np.where(live, delta + rel + 4 * U * (1 + np.abs(lse)), 0.0), "lse")
    if out[2] is not None:
        V = W.shape[0]
        tol = (2 * delta + rel + 8 * U) * (2 + 2 * ent + np.log(V))
        _near(out[2], ent, np.where(live, tol, 0.0), "entropy")


def _check_backward(dH, dW, H, W, y, g, h, T):
    rH, rW, dz = oracle.token_logprobs_grad(H, W, y.numpy(), _f64(g), None if h is None else _f64(h), T)
    delta, rel = _bounds(H, W, T)
    _, logq = _logq(H, W, T)
    p = np.exp(logq)
    live = (y.numpy() >= 0)[:, None]
    size = np.abs(_f64(g))[:, None] * np.ones_like(p)
    if h is not None:
        ent = -(p * logq).sum(axis=1, keepdims=True)
        size = size + np.abs(_f64(h))[:, None] * (np.abs(logq) + ent + 1)
    tz = np.where(live, B16 * np.abs(dz) + (2 * delta[:, None] + rel + 2.0 ** -20) * p * size / T, 0.0)
    acc = lambda n: (n / 16 + 4) * 2 * U     # noqa: E731
    if dH is not None:
        Wn = np.abs(_f64(W))
        tol = (1 + B16) * (tz @ Wn + acc(W.shape[0]) * (np.abs(dz) @ Wn)) + B16 * np.abs(rH)
        _near(dH, rH, tol, "dH")
        assert bool((dH[(y < 0).to(dH.device)] == 0).all())
    if dW is not None:
        Hn = np.abs(_f64(H))
        tol = (1 + B16) * (tz.T @ Hn) + (B16 + acc(len(H))) * (np.abs(dz).T @ Hn)
        if dW.dtype == torch.bfloat16:
            tol = (1 + B16) * tol + B16 * np.abs(rW)
        _near(dW, rW, tol, "dW")


SIZES = [(1, 8, 1), (1, 64, 300), (2, 2880, 257), (3, 8, 256), (255, 72, 1000), (256, 64, 64), (257, 136, 513),
         (700, 256, 4100), (130, 200, 33001), (1100, 24, 255)]


@pytest.mark.parametrize("N,d,V", SIZES)
@pytest.mark.parametrize("ignored,i64,T,ent", [("none", True, 1.0, False), ("some", False, 0.7, True),
                                               ("some", True, 1.3, False), ("all", True, 1.0, True)])
def test_both_passes(kd, N, d, V, ignored, i64, T, ent):
    H, W, y, g, h = _inputs(N, d, V, N + V, ignored, i64)
    Hc, Wc, yc, gc, hc = (t.cuda() for t in (H, W, y, g, h))
    out = kd.token_logprobs_forward(Hc, Wc, yc, T, entropy=ent)
    _check_forward(out, H, W, y, T)
    e = dict(entropy=out[2], dentropy=hc) if ent else {}
    dH, dW = kd.token_logprobs_backward(Hc, Wc, yc, out[1], gc, T, **e)
    _check_backward(dH, dW, H, W, y, g, h if ent else None, T)
    # chunks of 100: several of them, the last ones short or empty; a bf16 dW through the fp32 sum
    dH2, dW2 = kd.token_logprobs_backward(Hc, Wc, yc, out[1], gc, T, chunk=100, dW_dtype=torch.bfloat16, **e)
    _check_backward(dH2, dW2, H, W, y, g, h if ent else None, T)
    # one chunk, a bf16 dW straight from the product: the fp32 dW rounded
    dH3, dW3 = kd.token_logprobs_backward(Hc, Wc, yc, out[1], gc, T, dW_dtype=torch.bfloat16, **e)
    assert torch.equal(dH3, dH) and torch.equal(dW3, dW.bfloat16())
    # dH alone (a frozen head)
    dH4, none = kd.token_logprobs_backward(Hc, Wc, yc, out[1], gc, T, dW_dtype=None, **e)
    assert none is None
    _check_backward(dH4, None, H, W, y, g, h if ent else None, T)


@pytest.mark.parametrize("N", [1, 7, 8, 9, 16, 17, 33, 64, 127, 128, 129])
@pytest.mark.parametrize("d,V", [(8, 3), (40, 129), (1000, 5003), (2880, 40000)])
@pytest.mark.parametrize("ignored", ["none", "some"])
def test_a_few_tokens(kd, N, d, V, ignored):
    """Both sides of the borders between the streaming pass and the GEMM, with and without entropies, and a token
    that the labels leave out in any place."""
    H, W, y, _, _ = _inputs(N, d, V, N + d, ignored)
    if ignored == "some":
        y[0] = -1
    for ent in (False, True):
        out = kd.token_logprobs_forward(H.cuda(), W.cuda(), y.cuda(), 0.9, entropy=ent)
        _check_forward(out, H, W, y, 0.9)


def test_confident_tokens(kd):
    """Labels at probabilities from 1e-3 to 1 - 1e-6: log-probabilities near 0 and p - 1 keep their precision."""
    H, W, y, g, _ = _inputs(300, 64, 500, 3, "none", pull=60.0)
    out = kd.token_logprobs_forward(H.cuda(), W.cuda(), y.cuda(), entropy=True)
    _check_forward(out, H, W, y, 1.0)
    assert float(out[0].max()) > -1e-5
    dH, dW = kd.token_logprobs_backward(H.cuda(), W.cuda(), y.cuda(), out[1], g.cuda())
    _check_backward(dH, dW, H, W, y, g, None, 1.0)


def test_skipping_zero_gradients_changes_nothing_else(kd):
    """Tokens with a zero upstream gradient are left out: the others' dH rows are the same bits, and dW is that of
    the others alone."""
    H, W, y, g, h = _inputs(600, 64, 700, 4, "some")
    g[::3] = 0.0
    h[::2] = 0.0
    Hc, Wc, yc, gc, hc = (t.cuda() for t in (H, W, y, g, h))
    _, lse, ent = kd.token_logprobs_forward(Hc, Wc, yc, entropy=True)
    for e, d in (({}, None), (dict(entropy=ent, dentropy=hc), h)):
        dH, dW = kd.token_logprobs_backward(Hc, Wc, yc, lse, gc, **e)
        _check_backward(dH, dW, H, W, y, g, d, 1.0)
    zero = torch.zeros_like(gc)
    dH, dW = kd.token_logprobs_backward(Hc, Wc, yc, lse, zero)
    assert not dH.any() and not dW.any()
    for half in (torch.float32, torch.bfloat16):
        for chunk in (100, 8192):
            dH, dW = kd.token_logprobs_backward(Hc, Wc, yc, lse, zero, chunk=chunk, dW_dtype=half)
            assert not dH.any() and not dW.any()


def test_accumulate_and_given_dW(kd):
    H, W, y, g, _ = _inputs(400, 64, 300, 5, "some")
    Hc, Wc, yc, gc = (t.cuda() for t in (H, W, y, g))
    lse = kd.token_logprobs_forward(Hc, Wc, yc)[1]
    base = torch.randn(300, 64, device="cuda")
    for chunk in (64, 8192):
        fresh = kd.token_logprobs_backward(Hc, Wc, yc, lse, gc, chunk=chunk)[1]
        dW = base.clone()
        got = kd.token_logprobs_backward(Hc, Wc, yc, lse, gc, chunk=chunk, dW=dW, accumulate_dW=True)[1]
        assert got is dW
        # base enters the chunks' float additions first: one rounding a chunk, of at most |base| + |dW|
        assert bool(((got - base - fresh).abs() <= 10 * 2 * U * (base.abs() + 1)).all())
        kept = torch.full_like(base, 5.0)
        assert torch.equal(kd.token_logprobs_backward(Hc, Wc, yc, lse, gc, chunk=chunk, dW=kept)[1], fresh)


def test_bad_labels_are_reported(kd):
    H, W, y, g, _ = _inputs(300, 64, 200, 6, "some")
    y[5], y[6], y[250] = 200, 2 ** 40, 199
    Hc, Wc, yc, gc = (t.cuda() for t in (H, W, y, g))
    ws = torch.empty(kd.kd_token_logp_forward_workspace_size(300, 64, 200), dtype=torch.uint8, device="cuda")
    logp, lse, ent = kd.token_logprobs_forward(Hc, Wc, yc, entropy=True, workspace=ws)
    assert kd.check(ws) == (5, 2)
    for t in (logp, lse, ent):
        assert torch.isnan(t[5:7]).all() and int(torch.isnan(t).sum()) == 2
    y[5] = y[6] = -1
    _check_forward((torch.where(torch.isnan(logp), 0.0, logp), torch.where(torch.isnan(lse), 0.0, lse), None), H, W, y, 1.0)
    dH, dW = kd.token_logprobs_backward(Hc, Wc, yc, lse, gc)
    _check_backward(dH, dW, H, W, y, g, None, 1.0)
    kd.token_logprobs_forward(Hc, Wc, y.cuda(), workspace=ws)
    assert kd.check(ws) == (0, 0)


def test_nan_rows_stay_their_own(kd):
    """A token whose hidden state or upstream gradient is NaN spoils its own results and dW, nothing else; one that is
    ignored spoils nothing."""
    H, W, y, g, _ = _inputs(300, 64, 200, 7, "none")
    clean = kd.token_logprobs_forward(H.cuda(), W.cuda(), y.cuda())
    dH0, dW0 = kd.token_logprobs_backward(H.cuda(), W.cuda(), y.cuda(), clean[1], g.cuda())
    H[17] = float("nan")
    out = kd.token_logprobs_forward(H.cuda(), W.cuda(), y.cuda(), entropy=True)
    assert all(torch.isnan(t[17]) for t in out) and int(torch.isnan(out[0]).sum()) == 1
    keep = torch.arange(300, device="cuda") != 17
    assert torch.equal(out[0][keep], clean[0][keep])
    dH, dW = kd.token_logprobs_backward(H.cuda(), W.cuda(), y.cuda(), out[1], g.cuda())
    assert torch.equal(dH[keep], dH0[keep]) and torch.isnan(dH[17]).any() and torch.isnan(dW).any()
    y[17] = -1
    out = kd.token_logprobs_forward(H.cuda(), W.cuda(), y.cuda())
    dH, dW = kd.token_logprobs_backward(H.cuda(), W.cuda(), y.cuda(), out[1], g.cuda())
    assert torch.isfinite(dH).all() and torch.isfinite(dW).all() and not dH[17].any()
    g[3] = float("nan")
    dH, _ = kd.token_logprobs_backward(H.cuda(), W.cuda(), y.cuda(), out[1], g.cuda())
    assert torch.isnan(dH[3]).all()


def test_no_tokens(kd):
    H, W = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16), torch.ones(9, 64, device="cuda", dtype=torch.bfloat16)
    y, z = torch.zeros(0, device="cuda", dtype=torch.int64), torch.zeros(0, device="cuda")
    logp, lse, ent = kd.token_logprobs_forward(H, W, y, entropy=True)
    assert logp.numel() == lse.numel() == ent.numel() == 0
    for half in (torch.float32, torch.bfloat16):
        dH, dW = kd.token_logprobs_backward(H, W, y, z, z, dW_dtype=half)
        assert dH.shape == (0, 64) and not dW.any() and dW.dtype == half


def test_autograd(kd):
    H, W, y, g, h = _inputs(300, 64, 700, 8, "some")
    Hc, Wc = H.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    yc, gc, hc = y.cuda(), g.cuda(), h.cuda()
    raw = kd.token_logprobs_forward(Hc.detach(), Wc.detach(), yc, 0.8, entropy=True)
    want = kd.token_logprobs_backward(Hc.detach(), Wc.detach(), yc, raw[1], gc, 0.8, entropy=raw[2], dentropy=hc,
                                      dW_dtype=torch.bfloat16)
    logp, ent = kd.token_logprobs(Hc, Wc, yc, T=0.8, entropy=True)
    got = torch.autograd.grad((logp * gc + ent * hc).sum(), (Hc, Wc), retain_graph=True)
    assert torch.equal(logp, raw[0]) and torch.equal(ent, raw[2])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[1].dtype == torch.bfloat16
    # an expanded (stride 0) upstream gradient, and only one of the two outputs used
    one = torch.ones(300, device="cuda")
    zero = torch.zeros_like(one)
    want = kd.token_logprobs_backward(Hc.detach(), Wc.detach(), yc, raw[1], one, 0.8, dW_dtype=torch.bfloat16)
    got = torch.autograd.grad(logp.sum(), (Hc, Wc), retain_graph=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = kd.token_logprobs_backward(Hc.detach(), Wc.detach(), yc, raw[1], zero, 0.8, entropy=raw[2], dentropy=one,
                                      dW_dtype=torch.bfloat16)
    got = torch.autograd.grad(ent.sum(), (Hc, Wc))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a frozen head
    logp = kd.token_logprobs(Hc, Wc.detach(), yc, T=0.8)
    (dH,) = torch.autograd.grad(logp, Hc, gc)
    _check_backward(dH, None, H, W, y, g, None, 0.8)
    with torch.no_grad():
        assert not kd.token_logprobs(Hc, Wc, yc).requires_grad


def test_gradient_agrees_with_differences(kd):
    """Central differences of the GPU's own log-probabilities along a direction of W, on a grid where every bf16 step is
    exact.  The remainder is bounded by h^2 times the third derivative (|H v|^3 <= 1 per unit of g) and the fp32
    rounding of logp over 2 h."""
    gen = torch.Generator().manual_seed(9)
    N, d, V, h = 40, 64, 300, 2.0 ** -7
    H = (torch.randint(-4, 5, (N, d), generator=gen) / 16).bfloat16()
    W = (torch.randint(-16, 17, (V, d), generator=gen) / 64).bfloat16()
    v = torch.randint(-1, 2, (V, d), generator=gen).float()
    y, g = torch.randint(0, V, (N,), generator=gen), torch.randn(N, generator=gen)
    f = lambda w: _f64(kd.token_logprobs_forward(H.cuda(), w.bfloat16().cuda(), y.cuda())[0])     # noqa: E731
    up, down = W.float() + h * v, W.float() - h * v
    assert torch.equal(up.bfloat16().float(), up) and torch.equal(down.bfloat16().float(), down)
    slope = float((_f64(g) * (f(up) - f(down))).sum()) / (2 * h)
    lse = kd.token_logprobs_forward(H.cuda(), W.cuda(), y.cuda())[1]
    dW = kd.token_logprobs_backward(H.cuda(), W.cuda(), y.cuda(), lse, g.cuda())[1]
    move = (_f64(H) @ v.numpy().T)
    third = float((np.abs(_f64(g)) * (np.abs(move).max(axis=1) ** 3)).sum())
    _, _, dz = oracle.token_logprobs_grad(H, W, y.numpy(), g.numpy())
    rounding = B16 * float((np.abs(dz) * np.abs(move)).sum()) + float(np.abs(_f64(g)).sum()) * 64 * U / (2 * h)
    assert abs(slope - float((_f64(dW) * v.numpy()).sum())) <= 2 * h * h * third + rounding


def test_same_bits_on_every_run_and_two_streams(kd):
    sets = [_inputs(900, 128, 3000, 10, "some"), _inputs(70, 64, 9000, 11, "some")]
    sets = [tuple(t.cuda() for t in s) for s in sets]

    def call(s):
        logp, lse, ent = kd.token_logprobs_forward(*s[:3], entropy=True)
        return (logp, lse, ent) + kd.token_logprobs_backward(*s[:3], lse, s[3], entropy=ent, dentropy=s[4], chunk=256)
    first = [call(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        outs = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                outs.append(call(s))
        torch.cuda.synchronize()
        for got, want in zip(outs, first):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed_with_other_labels(kd):
    """A captured step follows the labels and gradients that its buffers hold at replay: other tokens take part."""
    H, W, y, g, _ = (t.cuda() for t in _inputs(700, 64, 1500, 12, "some"))

    def step():
        logp, lse, _ = kd.token_logprobs_forward(H, W, y)
        return (logp,) + kd.token_logprobs_backward(H, W, y, lse, g, chunk=256)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        y.copy_(_inputs(700, 64, 1500, 20 + k, ("none", "some", "all", "some")[k])[2])
        g.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_offsets_past_32_bits(kd):
    """11,000 x 201,088 dZ elements (past 2^31) in one chunk: sampled rows of dH and dW against 64 bits on the GPU."""
    N, d, V = 11000, 64, 201088
    gen = torch.Generator(device="cuda").manual_seed(13)
    W = (torch.randn(V, d, device="cuda", generator=gen) * d ** -0.5).bfloat16()
    y = torch.randint(0, V, (N,), device="cuda", generator=gen)
    y[1000:1100] = -1
    H = (torch.randn(N, d, device="cuda", generator=gen) + 3 * W[y.clamp(min=0)].float()).bfloat16()
    g = torch.randn(N, device="cuda", generator=gen)
    logp, lse, _ = kd.token_logprobs_forward(H, W, y)
    dH, dW = kd.token_logprobs_backward(H, W, y, lse, g, chunk=N)
    rows = torch.tensor([0, 999, 1100, 5000, 10900, N - 1], device="cuda")
    cols = torch.cat([torch.tensor([0, 1, 70000, V - 1], device="cuda"), y[[N - 1, N - 2, 3]]])
    Hd, Wd, live = H.double(), W.double(), (y >= 0)
    lse64 = torch.cat([torch.logsumexp(Hd[i:i + 500] @ Wd.T, 1) for i in range(0, N, 500)])
    z = Hd[rows] @ Wd.T
    tol = 1e-4                                                  # of z and lse: far above the bounds of the small cases
    assert bool(((z.gather(1, y[rows, None])[:, 0] - lse64[rows] - logp[rows]).abs() < tol).all())
    assert bool(((lse64 - lse)[live].abs() < tol).all()) and not lse[~live].any()
    dz = -g[rows, None] * torch.exp(z - lse64[rows, None])
    dz.scatter_add_(1, y[rows, None], g[rows, None].double())
    want = dz @ Wd
    assert bool(((dH[rows] - want).abs() <= 2 * B16 * (dz.abs() @ Wd.abs() + want.abs())).all())
    p = torch.exp(Hd @ Wd[cols].T - lse64[:, None])             # [N, columns]
    dzc = (g[:, None] * ((y[:, None] == cols[None, :]).double() - p)) * live[:, None]
    want = dzc.T @ Hd
    assert bool(((dW[cols] - want).abs() <= 2 * B16 * (dzc.abs().T @ Hd.abs())).all())
    assert not dH[1000:1100].any()


def test_a_preference_and_a_policy_step(kd):
    """The operators together, as a training step runs them: log-probabilities, loss, head gradients, against the
    oracles composed.  The losses' gradients reach the head in float32; its tolerance is the head's, with the loss
    gradient's own error (a float32 logp's, 1e-5 of the largest) added through g."""
    N, d, V = 320, 128, 900
    H, W, y, _, _ = _inputs(N, d, V, 14, "some")
    rng = np.random.default_rng(14)
    offsets = np.array([0, 100, 150, 250, 320])
    bounds = list(zip(offsets[:-1].tolist(), offsets[1:].tolist()))
    mask = (y.numpy() >= 0).astype(np.float32)
    logp, _, ent = oracle.token_logprobs(H, W, y.numpy())
    ref = (logp + 0.2 * rng.standard_normal(N)).astype(np.float32)
    x = 0.3 * rng.standard_normal(N)
    for border in (np.log(1.2), np.log(0.8)):
        x[np.abs(x - border) < 1e-3] += 4e-3                    # no token whose clipping a float32 logp decides
    old = (logp - x).astype(np.float32)
    adv = rng.standard_normal(4).astype(np.float32)
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()      # noqa: E731
    off = c(offsets.astype(np.int32))
    Hc, Wc = H.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    steps = []
    lp = kd.token_logprobs(Hc, Wc, y.cuda())
    loss = kd.preference_loss(lp, c(ref), mask=c(mask), offsets=off, beta=0.5)[0]
    L, _, _, G = oracle.preference_loss(logp, ref, mask, bounds, beta=0.5)
    steps.append((loss, L, G, None))
    lp, en = kd.token_logprobs(Hc, Wc, y.cuda(), entropy=True)
    loss = kd.policy_loss(lp, c(old), c(adv), ref_logp=c(ref), mask=c(mask), offsets=off, kl_coef=0.1)[0]
    loss = loss - 0.01 * (en * c(mask)).sum() / c(mask).sum()
    L, _, _, G = oracle.policy_loss(logp, old, np.repeat(adv, np.diff(offsets)), ref, mask, bounds, kl_coef=0.1)
    m = mask.astype(np.float64)
    steps.append((loss, L - 0.01 * (ent * m).sum() / m.sum(), G, -0.01 * m / m.sum()))
    for loss, L, G, E in steps:
        assert abs(float(loss.detach()) - L) < 1e-4
        dH, dW = torch.autograd.grad(loss, (Hc, Wc))
        rH, rW, dz = oracle.token_logprobs_grad(H, W, y.numpy(), G, E)
        tz = 2 * B16 * np.abs(dz) + 1e-4 * np.abs(G).max()  * np.exp(_logq(H, W, 1.0)[1])
        _near(dH, rH, tz @ np.abs(_f64(W)) + B16 * np.abs(rH), "dH")
        _near(dW, rW, tz.T @ np.abs(_f64(H)) + B16 * np.abs(rW), "dW")


def test_binding_refuses(kd):
    H, W = torch.zeros(6, 16, device="cuda", dtype=torch.bfloat16), torch.zeros(9, 16, device="cuda", dtype=torch.bfloat16)
    y, v = torch.zeros(6, device="cuda", dtype=torch.int64), torch.zeros(6, device="cuda")
    bad = [
        (TypeError, lambda: kd.token_logprobs(H.float(), W, y)),
        (TypeError, lambda: kd.token_logprobs(H, W.half(), y)),
        (TypeError, lambda: kd.token_logprobs(H, W, y.float())),
        (TypeError, lambda: kd.token_logprobs(H, W, y.to(torch.int16))),
        (ValueError, lambda: kd.token_logprobs(H, W, y[:5])),
        (ValueError, lambda: kd.token_logprobs(H, W, y.cpu())),
        (ValueError, lambda: kd.token_logprobs(H, W.cpu(), y)),
        (ValueError, lambda: kd.token_logprobs(H, W[:, :8].contiguous(), y)),
        (ValueError, lambda: kd.token_logprobs(H[:, :8], W[:, :8], y)),
        (ValueError, lambda: kd.token_logprobs(H[None], W, y)),
        (ValueError, lambda: kd.token_logprobs(H[:, :12].contiguous(), W[:, :12].contiguous(), y)),     # d % 8
        (kd.KDError, lambda: kd.token_logprobs(H, W, y, T=0.0)),
        (kd.KDError, lambda: kd.token_logprobs(H, W, y, T=1e-7)),
        (ValueError, lambda: kd.token_logprobs_backward(H, W, y, v, v, entropy=v)),
        (ValueError, lambda: kd.token_logprobs_backward(H, W, y, v, v[:3])),
        (TypeError, lambda: kd.token_logprobs_backward(H, W, y, v, v, dW_dtype=torch.float16)),
        (ValueError, lambda: kd.token_logprobs_backward(H, W, y, v, v, accumulate_dW=True)),
        (ValueError, lambda: kd.token_logprobs_backward(H, W, y, v, v, dW=torch.zeros_like(W), accumulate_dW=True)),
        (ValueError, lambda: kd.token_logprobs_backward(H, W, y, v, v, dW=torch.zeros(8, 16, device="cuda"))),
        (ValueError, lambda: kd.token_logprobs_backward(H, W, y, v, v, chunk=0)),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
    with pytest.raises(kd.KDError):
        kd.token_logprobs_forward(H, W, y, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_calls_are_made_on_the_inputs_device_and_stream(kd, monkeypatch):
    """Each library call is made with the inputs' device current and on its current stream (the losses' calls too)."""
    seen = []

    def spy(module, name):
        real = getattr(module, name)

        def call(dev):
            seen.append((name, dev))
            return real(dev)
        monkeypatch.setattr(module, name, call)
    for m in ("logprobs", "sequence_losses"):
        spy(sys.modules["chunked_top_kl_b200." + m], "_on")
        spy(sys.modules["chunked_top_kl_b200." + m], "_stream")
    H, W, y, g, _ = (t.cuda() for t in _inputs(40, 16, 50, 3, "some"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lse = kd.token_logprobs_forward(H, W, y)[1]
        kd.token_logprobs_backward(H, W, y, lse, g)
        x = torch.zeros(2, 20, device="cuda", requires_grad=True)
        kd.preference_loss(x)[0].backward()
        kd.policy_loss(x, x.detach(), x.detach())[0].backward()
    s.synchronize()
    dev = H.device
    assert seen == [("_on", dev), ("_stream", dev)] * 6
