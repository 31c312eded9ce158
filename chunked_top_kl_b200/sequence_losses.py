"""Losses over token log-probabilities grouped into sequences: the preference
loss over paired answers and the clipped policy loss with a KL term.

The token arrays are float32, either packed, ``[N]`` with ``offsets`` ``[S + 1]``
(int32 or int64: sequence s is ``[offsets[s], offsets[s + 1])``), or padded,
``[S, L]`` without offsets.  ``mask`` is a float32 weight per token (0: the
token takes no part, whatever the other arrays hold there); None is all ones.
Only ``logp`` has a gradient; everything else is a constant.  As elsewhere in
this package no arithmetic happens here: the calls check, allocate and launch.
"""

from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .api import _grad_scalar, _on, _ptr, _raise, _stream

PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}
KL_KINDS = {"k1": 0, "k2": 1, "k3": 2}
REDUCTIONS = {"token": 0, "sequence": 1}


class _Layout(NamedTuple):
    S: int
    N: int
    offsets_i64: int


def _choice(table, value, what: str, where: str) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{where}: {what} must be one of {', '.join(table)}, got {value!r}") from None


def _check_token_arrays(where: str, logp, others) -> None:
    if not logp.is_cuda:
        raise ValueError(f"{where}: logp must be a CUDA tensor")
    dev, shape = logp.device, logp.shape
    for name, t in (("logp", logp),) + others:
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"{where}: {name} is on {t.device}, logp on {dev}")
        if t.dtype != torch.float32:
            raise TypeError(f"{where}: {name} must be float32, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{where}: {name} must have logp's shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")


def _check_layout(where: str, logp, offsets) -> _Layout:
    if offsets is None:
        if logp.dim() != 2:
            raise ValueError(f"{where}: logp must be [S, L], or [N] with offsets; got {tuple(logp.shape)}")
        return _Layout(logp.shape[0], logp.numel(), 0)
    if logp.dim() != 1:
        raise ValueError(f"{where}: with offsets, logp must be [N]; got {tuple(logp.shape)}")
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError(f"{where}: offsets must be [S + 1]")
    if offsets.device != logp.device:
        raise ValueError(f"{where}: offsets is on {offsets.device}, logp on {logp.device}")
    if offsets.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{where}: offsets must be int32 or int64, got {offsets.dtype}")
    if not offsets.is_contiguous():
        raise ValueError(f"{where}: offsets must be contiguous")
    return _Layout(offsets.numel() - 1, logp.numel(), int(offsets.dtype == torch.int64))


def _workspace(S: int, dev) -> torch.Tensor:
    return torch.empty(_abi.kd_sequence_loss_workspace_size(S), dtype=torch.uint8, device=dev)


def _preference(logp, ref_logp, mask, offsets, beta, kind, label_smoothing, margin, average, grad_loss, want_grad):
    where = "preference_loss"
    _check_token_arrays(where, logp, (("ref_logp", ref_logp), ("mask", mask)))
    lay = _check_layout(where, logp, offsets)
    if lay.S % 2:
        raise ValueError(f"{where}: {lay.S} sequences do not make pairs (the chosen ones come first, then the rejected)")
    k = _choice(PREFERENCE_KINDS, kind, "kind", where)
    dev = logp.device
    grad_loss = _grad_scalar(grad_loss, dev)
    loss = logp.new_empty(())
    chosen = logp.new_empty(lay.S // 2)
    rejected = logp.new_empty(lay.S // 2)
    dlogp = torch.empty_like(logp) if want_grad else None
    ws = _workspace(lay.S, dev)
    with _on(dev):
        st = _abi.kd_preference_loss(_ptr(logp), _ptr(ref_logp), _ptr(mask), _ptr(offsets), lay.offsets_i64, lay.S,
                                     lay.N, float(beta), k, float(label_smoothing), float(margin),
                                     int(bool(average)), _ptr(grad_loss), _ptr(loss), _ptr(chosen), _ptr(rejected), _ptr(dlogp), _ptr(ws), ws.numel(),
                                     _stream(dev))
    _raise(st, "kd_preference_loss")
    return loss, chosen, rejected, dlogp


def preference_loss_forward_backward(logp, ref_logp=None, mask=None, offsets=None, beta: float = 0.1,
                                     kind: str = "sigmoid", label_smoothing: float = 0.0, margin: float = 0.0,
                                     average: bool = False, grad_loss: Optional[torch.Tensor] = None
                                     ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Preference loss over paired sequences and its gradient in one call:
    returns (loss [], chosen_rewards [P], rejected_rewards [P], dlogp like logp).

    The 2P sequences are P chosen answers, then the P rejected ones in the
    same order.  r_s = sum_t mask_t (logp_t - ref_t), divided by sum_t mask_t
    with ``average``; delta = r_chosen - r_rejected, D = beta delta - margin:
    ``sigmoid`` -(1 - label_smoothing) log sigma(D) - label_smoothing
    log sigma(-D); ``hinge`` max(0, 1 - D); ``ipo`` (delta - margin -
    1 / (2 beta))^2.  The loss is the mean over the pairs, the rewards are
    beta r.  ``ref_logp=None`` compares the log-probabilities themselves."""
    return _preference(logp, ref_logp, mask, offsets, beta, kind, label_smoothing, margin, average, grad_loss, True)


def _policy(logp, old_logp, advantages, ref_logp, mask, offsets, clip_low, clip_high, dual_clip, kl_coef, kl, reduce,
            grad_loss, want_grad):
    where = "policy_loss"
    if logp.dim() == 1 and offsets is None:
        lay = _Layout(1, logp.numel(), 0)               # one sequence
    else:
        lay = _check_layout(where, logp, offsets)
    per_seq = advantages.shape != logp.shape
    _check_token_arrays(where, logp, (("old_logp", old_logp), ("ref_logp", ref_logp), ("mask", mask)) +
                        (() if per_seq else (("advantages", advantages),)))
    dev = logp.device
    if per_seq:
        if advantages.shape not in ((lay.S,), (lay.S, 1)):
            raise ValueError(f"{where}: advantages must have logp's shape {tuple(logp.shape)} or hold one value for "
                             f"each of the {lay.S} sequences, got {tuple(advantages.shape)}")
        if advantages.dtype != torch.float32 or advantages.device != dev or not advantages.is_contiguous():
            raise ValueError(f"{where}: advantages must be contiguous float32 on {dev}")
    k = _choice(KL_KINDS, kl, "kl", where)
    r = _choice(REDUCTIONS, reduce, "reduce", where)
    if ref_logp is None and kl_coef != 0.0:
        raise ValueError(f"{where}: kl_coef needs ref_logp")
    if dual_clip is not None and not dual_clip > 1.0:
        raise ValueError(f"{where}: dual_clip must be above 1, got {dual_clip}")
    grad_loss = _grad_scalar(grad_loss, dev)
    stats = logp.new_empty(3)
    dlogp = torch.empty_like(logp) if want_grad else None
    ws = _workspace(lay.S, dev)
    with _on(dev):
        st = _abi.kd_policy_loss(_ptr(logp), _ptr(old_logp), _ptr(ref_logp), _ptr(advantages), int(per_seq),
                                 _ptr(mask), _ptr(offsets), lay.offsets_i64, lay.S, lay.N, float(clip_low),
                                 float(clip_high), 0.0 if dual_clip is None else float(dual_clip), float(kl_coef),
                                 k, r, _ptr(grad_loss), _ptr(stats), _ptr(dlogp), _ptr(ws), ws.numel(),
                                 _stream(dev))
    _raise(st, "kd_policy_loss")
    return (*stats.unbind(0), dlogp)


def policy_loss_forward_backward(logp, old_logp, advantages, ref_logp=None, mask=None, offsets=None,
                                 clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: Optional[float] = None,
                                 kl_coef: float = 0.0, kl: str = "k3", reduce: str = "token",
                                 grad_loss: Optional[torch.Tensor] = None
                                 ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Clipped policy loss with a KL term and its gradient in one call:
    returns (loss [], kl [], clip_fraction [], dlogp like logp).

    With r = exp(logp - old_logp) and y = logp - ref_logp, each token's loss is
    -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef KL; for A < 0
    ``dual_clip`` (c > 1) bounds the first term by -c A.  KL is y (``k1``),
    y^2 / 2 (``k2``) or exp(-y) - 1 + y (``k3``); without ``ref_logp`` there is
    none, and with ``kl_coef`` 0 it is reported only.  ``advantages`` of logp's shape is per token, [S, 1] or another [S] per
    sequence.  ``reduce``: ``token`` divides the weighted sum by the mask's sum;
    ``sequence`` averages each sequence over its mask, then over all S
    sequences (an empty one counts 0).  kl and clip_fraction are averaged the
    same way.  A packed ``logp`` without offsets is one sequence.  Sums are in 64
    bits; a token's terms are in 64 bits up to about a million tokens in 592
    sequences (4,736 of a mean length up to 192) and in 32 above, where a ratio
    or exp(-y) beyond 3.4e38 is infinite."""
    return _policy(logp, old_logp, advantages, ref_logp, mask, offsets, clip_low, clip_high, dual_clip, kl_coef, kl,
                   reduce, grad_loss, True)


def _scaled(unit: torch.Tensor, grad: torch.Tensor) -> torch.Tensor:
    """The kept unit gradient times the loss's upstream gradient."""
    dev = unit.device
    g = _grad_scalar(grad, dev)
    out = torch.empty_like(unit)
    with _on(dev):
        st = _abi.kd_scale_gradient(_ptr(unit), _ptr(g), _ptr(out), unit.numel(),
                                    _stream(dev))
    _raise(st, "kd_scale_gradient")
    return out


class PreferenceLossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, ref_logp, mask, offsets, beta, kind, label_smoothing, margin, average):
        loss, chosen, rejected, dlogp = _preference(logp, ref_logp, mask, offsets, beta, kind, label_smoothing, margin,
                                                    average, None, ctx.needs_input_grad[0])
        ctx.save_for_backward(dlogp)
        ctx.mark_non_differentiable(chosen, rejected)
        ctx.set_materialize_grads(False)
        return loss, chosen, rejected

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, *_):
        (dlogp,) = ctx.saved_tensors
        return (None if grad is None else _scaled(dlogp, grad),) + (None,) * 8


class PolicyLossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, old_logp, advantages, ref_logp, mask, offsets, clip_low, clip_high, dual_clip, kl_coef, kl,
                reduce):
        *stats, dlogp = _policy(logp, old_logp, advantages, ref_logp, mask, offsets, clip_low, clip_high, dual_clip,
                                kl_coef, kl, reduce, None, ctx.needs_input_grad[0])
        # .data: tensors of their own over the three floats, not views of one, so that a caller may change the loss
        # or a reported value in place before going backward
        loss, kl_mean, clipped = (t.data for t in stats)
        ctx.save_for_backward(dlogp)
        ctx.mark_non_differentiable(kl_mean, clipped)
        ctx.set_materialize_grads(False)
        return loss, kl_mean, clipped

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, *_):
        (dlogp,) = ctx.saved_tensors
        return (None if grad is None else _scaled(dlogp, grad),) + (None,) * 11


def preference_loss(logp, ref_logp=None, mask=None, offsets=None, beta: float = 0.1, kind: str = "sigmoid",
                    label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Differentiable preference loss (see preference_loss_forward_backward):
    returns (loss, chosen_rewards, rejected_rewards); the loss's gradient
    reaches ``logp``, the rewards are for reporting."""
    return PreferenceLossFunction.apply(logp, ref_logp, mask, offsets, beta, kind, label_smoothing, margin, average)


def policy_loss(logp, old_logp, advantages, ref_logp=None, mask=None, offsets=None, clip_low: float = 0.2,
                clip_high: float = 0.2, dual_clip: Optional[float] = None, kl_coef: float = 0.0, kl: str = "k3",
                reduce: str = "token") -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Differentiable policy loss (see policy_loss_forward_backward): returns
    (loss, kl, clip_fraction); the loss's gradient reaches ``logp``, the other
    two are for reporting."""
    return PolicyLossFunction.apply(logp, old_logp, advantages, ref_logp, mask, offsets, clip_low, clip_high,
                                    dual_clip, kl_coef, kl, reduce)
