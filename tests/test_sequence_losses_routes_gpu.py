"""The losses over token log-probabilities by every route that the sizes choose.

A call is one launch (64-bit arithmetic in the policy loss) up to 2^20 tokens
when each item (a sequence, or a range of one) finds a team among the blocks
that an SM count of 148 holds, 592 of 256 threads; otherwise two launches, the
policy loss in 32-bit arithmetic per token.  A warp takes a sequence up to a
mean length of 192, else a block.  The layouts here are chosen for the second
form: many sequences of mean length above 192, or more than 2^20 tokens.
Tolerances are those of test_sequence_losses_gpu, against the fp64 oracle.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import test_sequence_losses_gpu as base
from test_sequence_losses_gpu import U, _check_policy, _check_pref, _gpu, _near, kd  # noqa: F401

pytestmark = pytest.mark.gpu

# Two launches with a block for each sequence, or several.
TWO_LAUNCHES = {
    "a_block_each": ([100 + (37 * i) % 400 for i in range(700)], 2, 3),
    "uneven": ([(13 * i) % 300 + (9000 if i % 211 == 5 else 0) + 130 for i in range(800)], 1, 0),
    "several_blocks_each": ([600001, 1, 0, 450007], 3, 1),
}
SEQS, LENGTH = 700, 300          # 700 blocks are more than the GPU holds at once


def _inputs(monkeypatch, layout, seed):
    monkeypatch.setitem(base.LAYOUTS, layout, TWO_LAUNCHES[layout])
    return base._inputs(layout, seed)


def _tiled(a, n=SEQS * LENGTH):
    """The pattern over and over, n elements of it."""
    return np.resize(np.asarray(a, np.float32), n)


def _offsets(S=SEQS, L=LENGTH):
    return torch.arange(0, (S + 1) * L, L, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("layout", TWO_LAUNCHES)
@pytest.mark.parametrize("kind,average,reference,shift", [("sigmoid", False, True, 0), ("ipo", True, False, 1),
                                                         ("hinge", True, True, 2)])
def test_preference_in_two_launches(kd, monkeypatch, layout, kind, average, reference, shift):      # noqa: F811
    x = _inputs(monkeypatch, layout, 71 + shift)
    ref = x["ref"] if reference else None
    kw = dict(beta=0.3, kind=kind, label_smoothing=0.1, margin=0.15, average=average)
    off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int64 if shift else torch.int32)
    out = kd.preference_loss_forward_backward(_gpu(x["lp"], shift), _gpu(ref, shift), _gpu(x["mask"], shift), off, **kw)
    _check_pref(out, x, ref, x["mask"], **kw)


@pytest.mark.parametrize("layout", TWO_LAUNCHES)
@pytest.mark.parametrize("kl,reduce,dual,shift", [("k1", "token", None, 0), ("k2", "sequence", 1.3, 1),
                                                  ("k3", "token", 3.0, 3), ("k3", "sequence", None, 0)])
def test_policy_in_two_launches(kd, monkeypatch, layout, kl, reduce, dual, shift):                  # noqa: F811
    x = _inputs(monkeypatch, layout, 83 + shift)
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=dual, kl_coef=0.05, kl=kl, reduce=reduce)
    off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int64 if shift else torch.int32)
    out = kd.policy_loss_forward_backward(_gpu(x["lp"], shift), _gpu(x["old"], shift), _gpu(x["adv"], shift),
                                          _gpu(x["ref"], shift), _gpu(x["mask"], shift), off, **kw)
    _check_policy(out, x, x["adv"], x["ref"], x["mask"], **kw)


@pytest.mark.parametrize("S,L", [(800, 261), (3, 400003)])
@pytest.mark.parametrize("with_mask", [True, False])
def test_padded_in_two_launches(kd, S, L, with_mask):                                               # noqa: F811
    rng = np.random.default_rng(S + L)
    old = (-rng.exponential(1.0, S * L)).astype(np.float32)
    lp = (old + 0.2 * rng.standard_normal(S * L)).astype(np.float32)
    ref = (lp + 0.1 * rng.standard_normal(S * L)).astype(np.float32)
    a = rng.standard_normal(S).astype(np.float32)
    lens = rng.integers(0, L + 1, S)
    lens[0] = 0                                            # a row that the mask leaves empty
    mask = (np.arange(L)[None, :] < lens[:, None]).astype(np.float32).ravel() if with_mask else None
    x = dict(lp=lp, old=old, N=S * L, bounds=[(s * L, (s + 1) * L) for s in range(S)])
    two_d = lambda v: None if v is None else torch.from_numpy(v).cuda().reshape(S, L)    # noqa: E731
    for reduce in ("token", "sequence"):
        kw = dict(kl_coef=0.1, reduce=reduce)
        out = kd.policy_loss_forward_backward(two_d(lp), two_d(old), torch.from_numpy(a).cuda(), two_d(ref), two_d(mask), **kw)
        _check_policy(out, x, np.repeat(a, L), ref, mask, **kw)
    if S % 2 == 0:
        out = kd.preference_loss_forward_backward(two_d(lp), two_d(ref), two_d(mask), beta=0.1)
        _check_pref(out, x, ref, mask, beta=0.1)


# ---------------------------------------------------------------- 32-bit token arithmetic at its edges

def _check_tiled(out, period, adv, ref, copies, **kw):
    """out: the call on `copies` repetitions of `period` (lp, old): the oracle's result on one of them, its gradient
    divided among them."""
    lp, old = period
    n = lp.size
    L, K, C, G = oracle.policy_loss(lp, old, adv, ref, None, [(0, n)], **kw)
    x = lp.astype(np.float64) - old
    y = np.zeros(n) if ref is None else lp.astype(np.float64) - ref
    kl_size = (1 + np.exp(-y) + np.abs(y) + y * y) if ref is not None else np.zeros(n)
    size = np.abs(adv) * (np.exp(np.minimum(x, 80.0)) + 1) + kw.get("kl_coef", 0.0) * kl_size
    tol = (16 + 2 * np.abs(x) + 2 * np.abs(y)) * U * size / n
    _near(out[0], L, tol.sum() + U * abs(L) + 1e-12)
    _near(out[1], K, ((16 + 2 * np.abs(y)) * U * kl_size / n).sum() + U * abs(K) + 1e-12)
    _near(out[2], C, 8 * U * abs(C) + 1e-12)
    _near(out[3].reshape(copies, n), np.tile(G / copies, (copies, 1)), np.tile(tol / copies, (copies, 1)))
    assert np.array_equal(out[3].reshape(copies, n).cpu().numpy() == 0, np.tile(G == 0, (copies, 1)))


def test_clip_borders_in_32_bits(kd):                                                               # noqa: F811
    """Log ratios within three steps of each border, old log-probabilities of many sizes, advantages of both signs: the
    decision is that of the exact difference."""
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
    lp, old = np.array(lp, np.float32), np.array(old, np.float32)            # 4200: 14 sequences of 300
    adv = rng.choice([-1.0, 1.0], lp.size).astype(np.float32)
    kw = dict(clip_low=0.2, clip_high=0.25, dual_clip=2.0)
    out = kd.policy_loss_forward_backward(_gpu(_tiled(lp)), _gpu(_tiled(old)), _gpu(_tiled(adv)), offsets=_offsets(), **kw)
    _check_tiled(out, (lp, old), adv, None, SEQS * LENGTH // lp.size, **kw)
    # more than 2^20 tokens of one sequence
    copies = 251
    big = [_gpu(np.tile(a, copies)) for a in (lp, old, adv)]
    out = kd.policy_loss_forward_backward(*big, **kw)
    _check_tiled(out, (lp, old), adv, None, copies, **kw)


def test_far_ratios_in_32_bits(kd):                                                                 # noqa: F811
    """Ratios that overflow float32: clipped ones keep their border's value, and A = 0 takes no part."""
    lp = np.array([0.0, 0.0, -1.0, -200.0, -1.0, -1.0], np.float32)
    old = np.array([-200.0, -200.0, -1.0, 0.0, -1.0, -1.0], np.float32)
    adv = np.array([1.0, 0.0, 0.0, -1.0, 0.0, 0.0], np.float32)
    out = kd.policy_loss_forward_backward(*(_gpu(_tiled(a)) for a in (lp, old, adv)), offsets=_offsets())
    want = oracle.policy_loss(lp, old, adv, None, None, [(0, 6)])
    assert float(out[0]) == pytest.approx(want[0], rel=8 * U) and float(out[2]) == pytest.approx(2 / 6, rel=8 * U)
    assert bool((out[3] == 0).all())
    # a dual clip keeps an overflowing ratio of a negative advantage
    adv[0] = -1.0
    out = kd.policy_loss_forward_backward(*(_gpu(_tiled(a)) for a in (lp, old, adv)), offsets=_offsets(), dual_clip=3.0)
    want = oracle.policy_loss(lp, old, adv, None, None, [(0, 6)], dual_clip=3.0)
    assert float(out[0]) == pytest.approx(want[0], rel=8 * U) and bool((out[3] == 0).all())


@pytest.mark.parametrize("gap", [1e-3, 0.499, 0.501, 4.0])
@pytest.mark.parametrize("sign", [1, -1])
def test_small_kl_in_32_bits(kd, gap, sign):                                                        # noqa: F811
    """k3 is of second order in the distance, and is taken by a series below 1/2."""
    lp = np.linspace(-2, -1, 1000).astype(np.float32)
    ref = (lp + np.float32(sign * gap)).astype(np.float32)
    zero = np.zeros_like(lp)
    out = kd.policy_loss_forward_backward(_gpu(_tiled(lp)), _gpu(_tiled(lp)), _gpu(_tiled(zero)), _gpu(_tiled(ref)),
                                          offsets=_offsets(), kl_coef=1.0)
    _, K, _, G = oracle.policy_loss(lp, lp, zero, ref, None, [(0, 1000)], kl_coef=1.0)
    assert float(out[1]) == pytest.approx(K, rel=64 * U)
    got = out[3].double().cpu().numpy().reshape(-1, 1000) * (SEQS * LENGTH // 1000)
    assert np.max(np.abs(got / G - 1)) <= 64 * U


# ---------------------------------------------------------------- deterministic, streams, graphs, bad offsets

def _both(kd, a, off):                                                                              # noqa: F811
    return (kd.policy_loss_forward_backward(a["lp"], a["old"], a["adv"], a["ref"], a["mask"], off, kl_coef=0.1) +
            kd.policy_loss_forward_backward(a["lp"], a["old"], a["adv"], a["ref"], a["mask"], off, reduce="sequence") +
            kd.preference_loss_forward_backward(a["lp"], a["ref"], a["mask"], off))


def test_two_launches_on_two_streams(kd, monkeypatch):                                              # noqa: F811
    calls = []
    for layout in ("a_block_each", "several_blocks_each"):
        x = _inputs(monkeypatch, layout, 91)
        off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int32)
        a = {k: _gpu(x[k]) for k in ("lp", "old", "adv", "ref", "mask")}
        calls.append(lambda a=a, off=off: _both(kd, a, off))
    first = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        outs = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                outs.append(c())
        torch.cuda.synchronize()
        for got, want in zip(outs, first):
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_two_launches_captured_and_replayed(kd, monkeypatch):                                       # noqa: F811
    x = _inputs(monkeypatch, "a_block_each", 93)
    x["lp"] = np.where(x["mask"] != 0, x["lp"], 0).astype(np.float32)
    off = torch.tensor(x["offsets"], device="cuda", dtype=torch.int32)
    a = {k: _gpu(x[k]) for k in ("lp", "old", "adv", "ref", "mask")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _both(kd, a, off)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _both(kd, a, off)
    for k in range(3):
        a["lp"].add_(0.01 * k)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(p, q) for p, q in zip(got, _both(kd, a, off)))


def test_bad_offsets_stay_inside_in_two_launches(kd):                                               # noqa: F811
    """700 offsets that decrease or lie outside [0, N]: nothing outside the gradient (it lies between guards) is
    written, and the call returns."""
    n = SEQS * LENGTH
    big = torch.full((3 * n,), 7.0, device="cuda")
    lp, old, ref = (-torch.rand(n, device="cuda") for _ in range(3))
    rng = np.random.default_rng(3)
    for values in (rng.integers(-n, 2 * n, SEQS + 1), np.arange(n, n - SEQS - 1, -1) - 5000):
        for dtype in (torch.int32, torch.int64):
            off = torch.tensor(values, device="cuda", dtype=dtype)
            d = big[n:2 * n]
            keep = [torch.zeros(3, device="cuda"), torch.zeros(SEQS, device="cuda"), torch.zeros(SEQS, device="cuda"),
                    torch.empty(kd.kd_sequence_loss_workspace_size(SEQS), dtype=torch.uint8, device="cuda")]
            stream = torch.cuda.current_stream().cuda_stream
            i64 = int(dtype == torch.int64)
            assert kd.kd_preference_loss(lp.data_ptr(), ref.data_ptr(), None, off.data_ptr(), i64, SEQS, n, 0.1, 0, 0.0,
                                         0.0, 0, None, keep[0].data_ptr(), keep[1].data_ptr(), keep[2].data_ptr(),
                                         d.data_ptr(), keep[3].data_ptr(), keep[3].numel(), stream) == 0
            for per_sequence in (0, 1):
                assert kd.kd_policy_loss(lp.data_ptr(), old.data_ptr(), ref.data_ptr(), ref.data_ptr(), 0, None,
                                         off.data_ptr(), i64, SEQS, n, 0.2, 0.2, 0.0, 0.1, 2, per_sequence, None,
                                         keep[0].data_ptr(), d.data_ptr(), keep[3].data_ptr(), keep[3].numel(), stream) == 0
            torch.cuda.synchronize()
            assert bool((big[:n] == 7).all()) and bool((big[2 * n:] == 7).all())
