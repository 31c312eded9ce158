"""Preference and policy losses on the GPU against the fp64 oracle.

Tolerances, in steps u = 2^-24 (half a step of float32):
* preference: every sum is fp64 over exact fp32 differences, so loss and
  rewards are off by their final rounding, u each; dlogp is a float
  coefficient (u) times a weight (u): 3 u.  1e-11 of the summed magnitudes
  stands for the fp64 sums.
* policy: a token's ratio is expf (2 ulp = 4 u) of a rounded x (u |x|), times
  A, weights and sums of four floats (6 more u); the KL term's y is one
  rounding (u |y|, in the exponent too) through a series or expf and two
  additions.  So each token's terms are off by at most
  (16 + 2 |x| + 2 |y|) u of |A| r + |A| + kl_coef (1 + e^-y + |y| + y^2), taken
  without cancellation.
"""

import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def kd():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from chunked_top_kl_b200 import build
    build.build()
    import chunked_top_kl_b200 as k
    return k


# lengths of the sequences, tokens before the first and behind the last
LAYOUTS = {
    "one_token_each": ([1, 1], 0, 0),
    "empty_and_one": ([0, 1, 5, 0], 3, 2),
    "all_empty": ([0, 0], 0, 4),
    "short_odd": ([3, 130, 64, 7, 1, 33], 1, 1),
    "many_short": ([(7 * i) % 23 for i in range(600)], 2, 5),
    "block_edges": ([1023, 1024, 1025, 4097], 1, 3),
    "long_pair": ([70001, 65537], 5, 1),
    "one_long_among_short": ([50000, 300, 200, 250, 1, 0, 257, 400], 0, 0),
    "long_among_many_short": ([(11 * i) % 160 + (2047 + i // 40 if i % 40 == 7 else 0) for i in range(601)]
                              + [9001], 3, 1),
    "long_among_many_short_two_launches": ([90 + i % 50 + (3001 if i % 1500 == 1 else 0) for i in range(9500)], 1, 2),
}


def _inputs(layout, seed, wild=True):
    lens, before, behind = LAYOUTS[layout]
    N = before + sum(lens) + behind
    rng = np.random.default_rng(seed)
    offsets = before + np.concatenate([[0], np.cumsum(lens)])
    old = (-rng.exponential(1.0, N)).astype(np.float32)
    lp = (old + 0.25 * rng.standard_normal(N)).astype(np.float32)
    ref = (old + 0.5 * rng.standard_normal(N)).astype(np.float32)
    adv = rng.standard_normal(N).astype(np.float32)
    adv[rng.random(N) < 0.05] = 0.0
    mask = rng.choice([0.0, 1.0, 1.0, 0.25], N).astype(np.float32)
    if len(lens) > 2:                                  # one sequence with nothing left
        mask[offsets[1]:offsets[2]] = 0.0
    if wild:                                           # what masked places hold is not looked at
        off = np.flatnonzero(mask == 0)
        for k, v in enumerate((np.nan, np.inf, -np.inf, np.finfo(np.float32).min)):
            lp[off[k::7]] = v
            old[off[k + 1::7]] = v
            ref[off[k + 2::7]] = v
            adv[off[k + 3::7]] = v
    bounds = list(zip(offsets[:-1].tolist(), offsets[1:].tolist()))
    return dict(lp=lp, old=old, ref=ref, adv=adv, mask=mask, offsets=offsets, bounds=bounds, N=N)


def _gpu(a, shift=0):
    """On the GPU; `shift` elements behind a 16-byte boundary."""
    if a is None:
        return None
    t = torch.empty(a.shape[0] + shift, device="cuda", dtype=torch.from_numpy(a[:0]).dtype)[shift:]
    t.copy_(torch.from_numpy(a))
    return t


def _clean(x, mask):
    return np.where(mask != 0, x.astype(np.float64), 0.0)


def _near(got, want, tol):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert np.all(np.isfinite(got))
    bad = np.abs(got - want) - tol
    assert np.all(bad <= 0), (float(np.max(bad)), np.asarray(got).ravel()[np.argmax(bad)],
                              np.asarray(want).ravel()[np.argmax(bad)])


def _check_pref(out, x, ref, mask, **kw):
    loss, chosen, rejected, dlogp = out
    m = np.ones(x["N"]) if mask is None else mask
    lp, rf = _clean(x["lp"], m), None if ref is None else _clean(ref, m)
    L, C, R, G = oracle.preference_loss(lp, rf, m, x["bounds"], **kw)
    size = sum(np.abs(m[b:e] * (lp[b:e] - (0 if rf is None else rf[b:e]))).sum() for b, e in x["bounds"])
    slack = 1e-11 * (1 + size)
    _near(loss, L, U * abs(L) + slack * (1 + abs(L)))
    _near(chosen, C, U * np.abs(C) + slack)
    _near(rejected, R, U * np.abs(R) + slack)
    _near(dlogp.reshape(-1), G, 3 * U * np.abs(G) + slack * np.abs(m) / max(1, len(C)) * 10)
    assert np.all(dlogp.reshape(-1).cpu().numpy()[G == 0] == 0)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average,reference,i64,shift", [(False, True, False, 0), (True, True, True, 1),
                                                        (True, False, False, 2)])
def test_preference(kd, layout, kind, average, reference, i64, shift):
    x = _inputs(layout, 11 + shift)
    ref = x["ref"] if reference else None
    kw = dict(beta=0.3, kind=kind, label_smoothing=0.1, margin=0.15, average=average)
    off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int64 if i64 else torch.int32)
    out = kd.preference_loss_forward_backward(_gpu(x["lp"], shift), _gpu(ref, shift), _gpu(x["mask"], shift), off, **kw)
    _check_pref(out, x, ref, x["mask"], **kw)


@pytest.mark.parametrize("S,L", [(2, 1), (2, 9), (6, 130), (4, 1027), (2, 100003), (300, 5), (4, 0)])
@pytest.mark.parametrize("with_mask", [True, False])
def test_preference_padded(kd, S, L, with_mask):
    rng = np.random.default_rng(S * 1000 + L)
    lp = (-rng.exponential(1.0, S * L)).astype(np.float32)
    ref = (lp + 0.1 * rng.standard_normal(S * L)).astype(np.float32)
    lens = rng.integers(0, L + 1, S)
    mask = (np.arange(L)[None, :] < lens[:, None]).astype(np.float32).ravel() if with_mask else None
    x = dict(lp=lp, N=S * L, bounds=[(s * L, (s + 1) * L) for s in range(S)])
    two_d = lambda a: None if a is None else torch.from_numpy(a).cuda().reshape(S, L)    # noqa: E731
    out = kd.preference_loss_forward_backward(two_d(lp), two_d(ref), two_d(mask), beta=0.1)
    assert out[3].shape == (S, L)
    _check_pref(out, x, ref, mask, beta=0.1)


def test_no_pairs_no_tokens(kd):
    z = torch.zeros(0, device="cuda")
    loss, c, r, g = kd.preference_loss_forward_backward(z, z, None, torch.zeros(1, device="cuda", dtype=torch.int32))
    assert float(loss) == 0 and c.numel() == r.numel() == g.numel() == 0
    loss, kl, share, g = kd.policy_loss_forward_backward(z, z, z, z, None, torch.zeros(1, device="cuda", dtype=torch.int32))
    assert float(loss) == float(kl) == float(share) == 0 and g.numel() == 0
    t = torch.ones(7, device="cuda")                    # tokens, but no sequence
    g = kd.policy_loss_forward_backward(t, t, t, t, None, torch.zeros(1, device="cuda", dtype=torch.int32))[3]
    assert bool((g == 0).all())


def _check_policy(out, x, adv, ref, mask, **kw):
    loss, kl, share, dlogp = out
    m = np.ones(x["N"]) if mask is None else mask.astype(np.float64)
    lp, od, av = _clean(x["lp"], m), _clean(x["old"], m), _clean(adv, m)
    rf = None if ref is None else _clean(ref, m)
    L, K, C, G = oracle.policy_loss(lp, od, av, rf, m, x["bounds"], **kw)
    y = np.zeros_like(lp) if rf is None else lp - rf
    xx = lp - od
    w = np.zeros_like(lp)
    whole = sum(m[b:e].sum() for b, e in x["bounds"])
    for b, e in x["bounds"]:
        n = m[b:e].sum()
        if kw.get("reduce", "token") == "token":
            w[b:e] = m[b:e] / whole if whole else 0
        else:
            w[b:e] = m[b:e] / n / len(x["bounds"]) if n else 0
    r = np.exp(np.minimum(xx, 80.0))
    size_k = (1 + np.exp(-y) + np.abs(y) + y * y) if rf is not None else np.zeros_like(lp)
    size = np.abs(av) * (r + 1) + kw.get("kl_coef", 0.0) * size_k
    step = (16 + 2 * np.abs(xx) + 2 * np.abs(y)) * U * np.abs(w)
    tol = np.where(m != 0, step * size, 0.0)
    _near(loss, L, tol.sum() + U * abs(L) + 1e-12)
    _near(kl, K, np.where(m != 0, step * size_k, 0.0).sum() + U * abs(K) + 1e-12)
    _near(share, C, 8 * U * abs(C) + 1e-12)
    _near(dlogp.reshape(-1), G, tol)
    assert np.all(dlogp.reshape(-1).cpu().numpy()[(m == 0) | (w == 0)] == 0)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kl,reduce,dual,shift", [("k1", "token", None, 0), ("k2", "sequence", 1.3, 1),
                                                  ("k3", "token", 3.0, 3), ("k3", "sequence", None, 0)])
def test_policy(kd, layout, kl, reduce, dual, shift):
    x = _inputs(layout, 23 + shift)
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=dual, kl_coef=0.05, kl=kl, reduce=reduce)
    off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int64 if shift else torch.int32)
    out = kd.policy_loss_forward_backward(_gpu(x["lp"], shift), _gpu(x["old"], shift),
                                          _gpu(x["adv"], shift).reshape(-1), _gpu(x["ref"], shift),
                                          _gpu(x["mask"], shift), off, **kw)
    _check_policy(out, x, x["adv"], x["ref"], x["mask"], **kw)


@pytest.mark.parametrize("S,L", [(1, 1), (3, 7), (5, 129), (2, 5001), (1, 200003), (2000, 3)])
@pytest.mark.parametrize("reduce", ["token", "sequence"])
@pytest.mark.parametrize("column", [False, True])
def test_policy_padded_advantage_per_sequence(kd, S, L, reduce, column):
    rng = np.random.default_rng(S + L)
    old = (-rng.exponential(1.0, S * L)).astype(np.float32)
    lp = (old + 0.2 * rng.standard_normal(S * L)).astype(np.float32)
    a = rng.standard_normal(S).astype(np.float32)
    mask = (np.arange(L)[None, :] < rng.integers(0, L + 1, S)[:, None]).astype(np.float32).ravel()
    x = dict(lp=lp, old=old, N=S * L, bounds=[(s * L, (s + 1) * L) for s in range(S)])
    two_d = lambda v: torch.from_numpy(v).cuda().reshape(S, L)    # noqa: E731
    adv = torch.from_numpy(a).cuda()
    out = kd.policy_loss_forward_backward(two_d(lp), two_d(old), adv[:, None] if column else adv, None, two_d(mask),
                                          reduce=reduce)
    _check_policy(out, x, np.repeat(a, L), None, mask, reduce=reduce)
    assert float(out[1]) == 0


def test_policy_without_mask_and_offsets(kd):
    """A packed array without offsets is one sequence."""
    x = _inputs("block_edges", 31, wild=False)
    x["bounds"] = [(0, x["N"])]
    out = kd.policy_loss_forward_backward(_gpu(x["lp"]), _gpu(x["old"]), _gpu(x["adv"]), _gpu(x["ref"]), kl_coef=0.1)
    _check_policy(out, x, x["adv"], x["ref"], None, kl_coef=0.1)


def test_policy_at_the_clip_borders(kd):
    """Log ratios within a step of each border, from old log-probabilities of many sizes: the clip decision is
    that of the exact difference, and a token at the border itself is not clipped."""
    rng = np.random.default_rng(5)
    lp, old = [], []
    for border in (math.log1p(0.25), math.log1p(-0.2), math.log(2.0)):
        for o in -rng.exponential(3.0, 200):
            o = np.float32(o)
            p = np.float32(np.float64(o) + border)
            for k in range(-3, 4):
                q = p
                for _ in range(abs(k)):
                    q = np.nextafter(q, np.float32(np.inf if k > 0 else -np.inf))
                lp.append(q)
                old.append(o)
    lp, old = np.array(lp, np.float32), np.array(old, np.float32)
    adv = rng.choice([-1.0, 1.0], lp.size).astype(np.float32)
    x = dict(lp=lp, old=old, N=lp.size, bounds=[(0, lp.size)])
    kw = dict(clip_low=0.2, clip_high=0.25, dual_clip=2.0)
    out = kd.policy_loss_forward_backward(_gpu(lp), _gpu(old), _gpu(adv), **kw)
    _check_policy(out, x, adv, None, None, **kw)
    G = oracle.policy_loss(lp, old, adv, None, None, x["bounds"], **kw)[3]
    assert np.array_equal(out[3].cpu().numpy() == 0, G == 0)


def test_policy_far_ratios(kd):
    """Ratios that overflow float32: clipped ones keep their border's value, A = 0 takes no part, and small KL
    distances keep their relative precision (k3 is of second order)."""
    lp = np.array([0.0, 0.0, -1.0, -200.0, -1.0, -1.0], np.float32)
    old = np.array([-200.0, -200.0, -1.0, 0.0, -1.0, -1.0], np.float32)
    adv = np.array([1.0, 0.0, 0.0, -1.0, 0.0, 0.0], np.float32)
    out = kd.policy_loss_forward_backward(_gpu(lp), _gpu(old), _gpu(adv))
    want = oracle.policy_loss(lp, old, adv, None, None, [(0, 6)])
    assert float(out[0]) == pytest.approx(want[0], rel=4 * U) and float(out[2]) == pytest.approx(2 / 6, rel=4 * U)
    assert bool((out[3] == 0).all())
    lp = np.linspace(-2, -1, 1001).astype(np.float32)
    for gap in (1e-3, 0.499, 0.501, 4.0):
        for sign in (1, -1):
            ref = (lp + np.float32(sign * gap)).astype(np.float32)
            zero = np.zeros_like(lp)
            kl = float(kd.policy_loss_forward_backward(_gpu(lp), _gpu(lp), _gpu(zero), _gpu(ref), kl_coef=1.0)[1])
            assert kl == pytest.approx(oracle.policy_loss(lp, lp, zero, ref, None, [(0, lp.size)])[1], rel=64 * U)


def test_preference_of_pairs_infinitely_far_apart(kd):
    """A chosen or rejected answer of probability 0: the pair's loss is 0 or infinite, its slope 0 or -beta, never NaN
    (without smoothing the second term has no part); other pairs keep their gradients."""
    lp = torch.tensor([-1.0, -2.0, -3.0, -1.0, -2.0, -3.0], device="cuda")
    off = torch.arange(7, device="cuda", dtype=torch.int32)
    base = kd.preference_loss_forward_backward(lp, None, None, off, beta=0.5)
    lp[4] = float("-inf")                                  # pair 1: D = +inf
    loss, chosen, rejected, g = kd.preference_loss_forward_backward(lp, None, None, off, beta=0.5)
    want = 2 / 3 * math.log(2.0)
    assert float(loss) == pytest.approx(want, rel=4 * U) and float(rejected[1]) == -math.inf
    assert g[1] == 0 and g[4] == 0 and torch.equal(g[[0, 2, 3, 5]], base[3][[0, 2, 3, 5]])
    lp[4], lp[1] = -2.0, float("-inf")                     # pair 1: D = -inf
    loss, chosen, rejected, g = kd.preference_loss_forward_backward(lp, None, None, off, beta=0.5)
    assert float(loss) == math.inf and g[1].item() == pytest.approx(-0.5 / 3, rel=4 * U) and g[4] == -g[1]
    for kind, want, slope in (("hinge", math.inf, -0.5 / 3), ("ipo", math.inf, -math.inf)):
        loss, _, _, g = kd.preference_loss_forward_backward(lp, None, None, off, beta=0.5, kind=kind)
        assert float(loss) == want and g[1].item() == pytest.approx(slope, rel=4 * U)


def test_upstream_gradient_and_autograd(kd):
    x = _inputs("short_odd", 41)
    off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int32)
    lp = _gpu(x["lp"]).requires_grad_(True)
    g = torch.tensor(-2.5, device="cuda")
    args = (_gpu(x["ref"]), _gpu(x["mask"]), off)
    base = kd.preference_loss_forward_backward(lp.detach(), *args)
    loss, chosen, rejected = kd.preference_loss(lp, *args)
    assert loss.requires_grad and not chosen.requires_grad and not rejected.requires_grad
    (grad,) = torch.autograd.grad(loss * g, lp, retain_graph=True)
    assert torch.equal(loss.detach(), base[0]) and torch.equal(chosen, base[1]) and torch.equal(rejected, base[2])
    assert torch.equal(grad, base[3] * g)
    (again,) = torch.autograd.grad(loss, lp)            # a second pass through the same graph
    assert torch.equal(again, base[3])
    scaled = kd.preference_loss_forward_backward(lp.detach(), *args, grad_loss=g)[3]
    assert torch.allclose(scaled, base[3] * g, rtol=4 * U, atol=0)

    args = (_gpu(x["old"]), _gpu(x["adv"]), _gpu(x["ref"]), _gpu(x["mask"]), off)
    base = kd.policy_loss_forward_backward(lp.detach(), *args, kl_coef=0.1)
    loss, kl, share = kd.policy_loss(lp, *args, kl_coef=0.1)
    assert loss.requires_grad and not kl.requires_grad and not share.requires_grad
    (grad,) = torch.autograd.grad(loss, lp, g)
    assert torch.equal(grad, base[3] * g)
    scaled = kd.policy_loss_forward_backward(lp.detach(), *args, kl_coef=0.1, grad_loss=g)[3]
    assert torch.allclose(scaled, base[3] * g, rtol=8 * U, atol=0)
    with torch.no_grad():
        assert torch.equal(kd.policy_loss(lp, *args, kl_coef=0.1)[0], base[0])


def test_gradient_agrees_with_differences(kd):
    """Central differences of the GPU's own loss, in a direction: h = 2^-7 moves D and x by far more than a float32
    step.  The third-order remainder (below h^2 times the gradient's scale) and the loss's rounding over 2 h bound it."""
    rng = np.random.default_rng(9)
    n, h = 64, 2.0 ** -7
    old = np.round(-rng.exponential(1.0, n) * 256) / 256                  # exact steps: h is representable beside them
    lp = old + np.round(0.05 * rng.standard_normal(n) * 256) / 256
    ref = old + np.round(0.3 * rng.standard_normal(n) * 256) / 256
    v = rng.choice([-1.0, 1.0], n)
    off = torch.tensor([0, 16, 32, 48, 64], device="cuda", dtype=torch.int32)
    t = lambda a: torch.tensor(a, device="cuda", dtype=torch.float32)     # noqa: E731
    def pref(a): return kd.preference_loss_forward_backward(t(a), t(ref), None, off, beta=0.5)        # noqa: E704
    def pol(a): return kd.policy_loss_forward_backward(t(a), t(old), t(v), t(ref), None, off, 0.9, 9.0, kl_coef=0.3)  # noqa: E704
    for f in (pref, pol):
        out = f(lp)
        slope = (float(f(lp + h * v)[0]) - float(f(lp - h * v)[0])) / (2 * h)
        want = float((out[3].double().cpu().numpy() * v).sum())
        scale = float(out[3].double().abs().sum()) + 1.0
        assert abs(slope - want) <= scale * h * h * 16 + 4 * U * abs(float(out[0])) / (2 * h)


def test_same_bits_on_every_run_and_two_streams(kd):
    x = _inputs("many_short", 51)
    y = _inputs("long_pair", 52)
    calls = []
    for z in (x, y):
        off = torch.tensor(z["offsets"], device="cuda", dtype=torch.int32)
        a = {k: _gpu(z[k]) for k in ("lp", "old", "adv", "ref", "mask")}
        calls.append(lambda a=a, off=off: kd.policy_loss_forward_backward(a["lp"], a["old"], a["adv"], a["ref"], a["mask"],
                                                                         off, kl_coef=0.1) +
                     kd.preference_loss_forward_backward(a["lp"], a["ref"], a["mask"], off))
    first = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        outs = []
        for c, s in zip(calls, streams):               # both in flight at once
            with torch.cuda.stream(s):
                outs.append(c())
        torch.cuda.synchronize()
        for got, want in zip(outs, first):
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_captured_and_replayed(kd):
    x = _inputs("one_long_among_short", 61, wild=False)
    off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int32)
    a = {k: _gpu(x[k]) for k in ("lp", "old", "adv", "ref", "mask")}

    def step():
        return (kd.policy_loss_forward_backward(a["lp"], a["old"], a["adv"], a["ref"], a["mask"], off, kl_coef=0.1) +
                kd.preference_loss_forward_backward(a["lp"], a["ref"], a["mask"], off))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        a["lp"].add_(0.01 * k)                          # new values at the captured addresses
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


def test_bad_offsets_stay_inside(kd):
    """Offsets that decrease or lie outside [0, N]: the values are undefined, but nothing outside the arrays is
    written (the arrays lie between guards) and the call returns."""
    n = 500
    big = torch.full((3 * n,), 7.0, device="cuda")
    lp, old, ref = (-torch.rand(n, device="cuda") for _ in range(3))
    for values in ([0, 400, 100, 500, 300], [-5, 20, 600, 10 ** 6, 10 ** 9], [500, 400, 300, 200, 100]):
        for dtype in (torch.int32, torch.int64):
            off = torch.tensor(values, device="cuda", dtype=dtype)
            kd.policy_loss_forward_backward(lp, old, ref, ref, None, off, reduce="sequence")
            d = big[n:2 * n]
            st = kd.kd_preference_loss(lp.data_ptr(), ref.data_ptr(), None, off.data_ptr(), int(dtype == torch.int64), 4, n,
                                       0.1, 0, 0.0, 0.0, 0, None, *(t.data_ptr() for t in _scalars()), d.data_ptr(),
                                       *_ws(kd, 4), torch.cuda.current_stream().cuda_stream)
            assert st == 0
            torch.cuda.synchronize()
            assert bool((big[:n] == 7).all()) and bool((big[2 * n:] == 7).all())


_KEPT = []


def _scalars():
    _KEPT[:] = [torch.zeros(1, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda")]
    return _KEPT


def _ws(kd, S):
    w = torch.empty(kd.kd_sequence_loss_workspace_size(S), dtype=torch.uint8, device="cuda")
    _KEPT.append(w)
    return w.data_ptr(), w.numel()


def test_binding_refuses(kd):
    x = torch.zeros(10, device="cuda")
    off = torch.tensor([0, 3, 5, 7, 10], device="cuda", dtype=torch.int32)
    ok = torch.zeros(4, device="cuda")
    bad = [
        (TypeError, lambda: kd.preference_loss(x.half(), None, None, off)),
        (TypeError, lambda: kd.preference_loss(x, x.double(), None, off)),
        (TypeError, lambda: kd.preference_loss(x, x, x.bool(), off)),
        (TypeError, lambda: kd.preference_loss(x, x, x, off.float())),
        (ValueError, lambda: kd.preference_loss(x, x[:9], None, off)),
        (ValueError, lambda: kd.preference_loss(x, x, None, None)),
        (ValueError, lambda: kd.preference_loss(x, x, None, off[:4])),
        (ValueError, lambda: kd.preference_loss(x, x, None, off.cpu())),
        (ValueError, lambda: kd.preference_loss(x, x.cpu(), None, off)),
        (ValueError, lambda: kd.preference_loss(torch.zeros(20, device="cuda")[::2], None, None, off)),
        (ValueError, lambda: kd.preference_loss(x, x, None, off, kind="dpo")),
        (kd.KDError, lambda: kd.preference_loss(x, x, None, off, beta=0.0)),
        (kd.KDError, lambda: kd.preference_loss(x, x, None, off, label_smoothing=2.0)),
        (ValueError, lambda: kd.policy_loss(x, x, ok[:3], None, None, off)),
        (ValueError, lambda: kd.policy_loss(x, x, ok.double(), None, None, off)),
        (ValueError, lambda: kd.policy_loss(x, x, x, None, None, off, kl_coef=0.1)),
        (ValueError, lambda: kd.policy_loss(x, x, x, x, None, off, kl="k4")),
        (ValueError, lambda: kd.policy_loss(x, x, x, x, None, off, reduce="mean")),
        (ValueError, lambda: kd.policy_loss(x, x, x, x, None, off, dual_clip=0.5)),
        (kd.KDError, lambda: kd.policy_loss(x, x, x, x, None, off, clip_low=1.5)),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()


def test_advantages_of_as_many_sequences_as_tokens(kd):
    """[N] is per token even where N = S; [S, 1] is per sequence."""
    lp = torch.zeros(4, device="cuda")
    off = torch.tensor([0, 3, 3, 4, 4], device="cuda", dtype=torch.int32)
    a = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")
    assert kd.policy_loss_forward_backward(lp, lp, a, offsets=off)[3].tolist() == (-a / 4).tolist()
    assert kd.policy_loss_forward_backward(lp, lp, a[:, None], offsets=off)[3].tolist() == [-0.25, -0.25, -0.25, -0.75]
