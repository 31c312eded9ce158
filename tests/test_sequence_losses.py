"""Losses over token log-probabilities: the oracle against closed forms and
central differences, and what the calls refuse (no GPU needed: the refusals
come before any CUDA call)."""

import math

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def kd():
    from chunked_top_kl_b200 import build
    build.build()
    import chunked_top_kl_b200 as k
    return k


BOUNDS = [(1, 6), (6, 6), (6, 7), (7, 12)]          # one empty sequence, one of one token, tokens outside at both ends
N = 13


def _tokens(seed, n=N):
    rng = np.random.default_rng(seed)
    old = -rng.exponential(1.0, n)
    return rng, old + 0.3 * rng.standard_normal(n), old, old + 0.2 * rng.standard_normal(n)


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in range(x.size):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
def test_oracle_preference_gradient_is_that_of_differences(kind, average):
    rng, lp, _, ref = _tokens(3)
    mask = rng.choice([0.0, 1.0, 0.5], N)
    kw = dict(beta=0.7, kind=kind, label_smoothing=0.1, margin=0.2, average=average)
    loss, chosen, rejected, grad = oracle.preference_loss(lp, ref, mask, BOUNDS, **kw)
    num = _differences(lambda v: oracle.preference_loss(v, ref, mask, BOUNDS, **kw)[0], lp)
    assert np.max(np.abs(num - grad)) < 1e-8
    assert np.all(grad[[0, 12]] == 0) and chosen.shape == rejected.shape == (2,)


def test_oracle_preference_of_equal_policies():
    """logp = ref: no log ratio, so the sigmoid loss is log 2 and the hinge loss 1."""
    _, lp, _, _ = _tokens(4)
    assert oracle.preference_loss(lp, lp, None, BOUNDS)[0] == pytest.approx(math.log(2), abs=1e-15)
    assert oracle.preference_loss(lp, lp, None, BOUNDS, kind="hinge")[0] == 1.0
    assert oracle.preference_loss(lp, lp, None, BOUNDS, kind="ipo", beta=0.5)[0] == 1.0


@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("reduce", ["token", "sequence"])
@pytest.mark.parametrize("dual", [None, 1.4])
def test_oracle_policy_gradient_is_that_of_differences(kl, reduce, dual):
    rng, lp, old, ref = _tokens(5)
    mask, adv = rng.choice([0.0, 1.0, 0.5], N), rng.standard_normal(N)
    kw = dict(clip_low=0.2, clip_high=0.3, dual_clip=dual, kl_coef=0.3, kl=kl, reduce=reduce)
    _, _, share, grad = oracle.policy_loss(lp, old, adv, ref, mask, BOUNDS, **kw)
    num = _differences(lambda v: oracle.policy_loss(v, old, adv, ref, mask, BOUNDS, **kw)[0], lp)
    assert np.max(np.abs(num - grad)) < 1e-8 and 0 <= share <= 1


def test_oracle_policy_on_policy():
    """logp = old = ref: the ratio is one, nothing is clipped, no KL: -mean(A), gradient -A / n."""
    rng, lp, _, _ = _tokens(6)
    adv = rng.standard_normal(N)
    loss, kl, share, grad = oracle.policy_loss(lp, lp, adv, lp, None, [(0, N)], kl_coef=0.5)
    assert loss == pytest.approx(-adv.mean(), abs=1e-15) and kl == 0 and share == 0
    assert np.allclose(grad, -adv / N, atol=1e-16)


def test_oracle_policy_is_min_of_clipped_and_unclipped():
    rng, lp, old, _ = _tokens(7, 200)
    adv = rng.standard_normal(200)
    r = np.exp(lp - old)
    want = -np.mean(np.minimum(r * adv, np.clip(r, 0.8, 1.3) * adv))
    assert oracle.policy_loss(lp, old, adv, None, None, [(0, 200)], clip_high=0.3)[0] == pytest.approx(want, abs=1e-14)


# ---------------------------------------------------------------- refusals

P = 1 << 20          # a fake, well aligned device address: these calls return before any CUDA call


def _pref(kd, **kw):
    a = dict(logp=P, ref=P, mask=P, offsets=P, i64=0, S=4, N=100, beta=0.1, kind=0, smoothing=0.0, margin=0.0,
             average=0, grad=None, loss=P, chosen=P, rejected=P, dlogp=P, ws=P, nb=1 << 20)
    a.update(kw)
    return kd.kd_preference_loss(*a.values(), None)


def _policy(kd, **kw):
    a = dict(logp=P, old=P, ref=P, adv=P, per_seq=0, mask=P, offsets=P, i64=0, S=4, N=100, lo=0.2, hi=0.2, dual=0.0,
             coef=0.1, kl=2, reduce=0, grad=None, loss=P, dlogp=P, ws=P, nb=1 << 20)
    a.update(kw)
    return kd.kd_policy_loss(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(S=-2), dict(S=3), dict(N=-1), dict(logp=None), dict(logp=P + 2), dict(loss=None), dict(chosen=None),
    dict(dlogp=P + 1), dict(ws=None), dict(ws=P + 64), dict(offsets=P + 4, i64=1), dict(i64=2), dict(beta=0.0),
    dict(beta=float("nan")), dict(beta=float("inf")), dict(kind=3), dict(kind=-1), dict(smoothing=-0.1),
    dict(smoothing=1.1), dict(smoothing=float("nan")), dict(margin=float("inf")), dict(average=2),
    dict(offsets=None, S=6), dict(offsets=None, S=0)])
def test_preference_refuses(kd, bad):
    from chunked_top_kl_b200 import _abi
    assert _pref(kd, **bad) == _abi.KD_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(S=-1), dict(N=-1), dict(old=None), dict(adv=None), dict(old=P + 2), dict(loss=None), dict(ws=P + 4),
    dict(lo=-0.1), dict(lo=1.0), dict(hi=-0.1), dict(hi=float("inf")), dict(dual=1.0), dict(dual=0.5),
    dict(dual=float("inf")), dict(coef=float("nan")), dict(kl=3), dict(reduce=2), dict(per_seq=2),
    dict(offsets=None, S=7)])
def test_policy_refuses(kd, bad):
    from chunked_top_kl_b200 import _abi
    assert _policy(kd, **bad) == _abi.KD_ERR_INVALID_ARG


def test_workspace_and_sizes(kd):
    from chunked_top_kl_b200 import _abi
    ws = kd.kd_sequence_loss_workspace_size
    assert ws(0) > 0 and ws(-1) == 0 and ws(1 << 31) == 0
    assert ws(1) == ws(500) < ws(100000)
    assert ws(200000) - ws(100000) == 16 * 100000
    assert _pref(kd, nb=ws(4) - 1) == _abi.KD_ERR_WORKSPACE
    assert _policy(kd, nb=ws(4) - 1) == _abi.KD_ERR_WORKSPACE
    assert _pref(kd, S=1 << 31) == _abi.KD_ERR_UNSUPPORTED
    assert _policy(kd, N=1 << 40) == _abi.KD_ERR_UNSUPPORTED
    assert kd.kd_scale_gradient(P, None, P, 4, None) == _abi.KD_ERR_INVALID_ARG
    assert kd.kd_scale_gradient(P, P, None, 4, None) == _abi.KD_ERR_INVALID_ARG
    assert kd.kd_scale_gradient(P, P, P + 2, 4, None) == _abi.KD_ERR_INVALID_ARG
    assert kd.kd_scale_gradient(P, P, P, -1, None) == _abi.KD_ERR_INVALID_ARG
    assert kd.kd_scale_gradient(None, P, None, 0, None) == _abi.KD_OK


def test_binding_checks_layout_and_choices():
    """Host logic on CPU tensors."""
    from chunked_top_kl_b200 import sequence_losses as sl
    x, o = torch.zeros(10), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sl._check_token_arrays("f", x, ())
    assert sl._check_layout("f", x, o) == (4, 10, 0)
    assert sl._check_layout("f", x, o.long()) == (4, 10, 1)
    assert sl._check_layout("f", torch.zeros(3, 5), None) == (3, 15, 0)
    for bad in (lambda: sl._check_layout("f", x, None), lambda: sl._check_layout("f", torch.zeros(2, 5), o),
                lambda: sl._check_layout("f", x, o[:0]), lambda: sl._check_layout("f", x, o.reshape(1, 5)),
                lambda: sl._check_layout("f", x, torch.zeros(9, dtype=torch.int32)[::2]),
                lambda: sl._check_layout("f", x, o.to("meta"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        sl._check_layout("f", x, o.float())
    for table, value in ((sl.PREFERENCE_KINDS, "dpo"), (sl.KL_KINDS, None), (sl.REDUCTIONS, ["token"])):
        with pytest.raises(ValueError, match="one of"):
            sl._choice(table, value, "x", "f")
