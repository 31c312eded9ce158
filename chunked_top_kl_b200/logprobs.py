"""Label log-probabilities of tokens under the LM head, with their gradients:
what losses on labels, preferences and rewards need of the head.

H [N,d] and W [V,d] are bf16, as for the distillation loss, and no logits are
stored.  ``labels`` are int32 or int64; a negative one marks a token without a
label (a prompt token), which costs nothing and contributes nothing.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .api import _check_buffer, _check_workspace, _on, _ptr, _raise, _stream

#: Tokens whose dZ rows (2 V bytes each) are held at once going back.  Larger
#: than the distillation loss's 4096: dW is then written once, without a read
#: and a second write, for batches of up to this many tokens.
LOGP_CHUNK = 8192


def _check(where: str, H, W, labels) -> Tuple[int, int, int]:
    for name, t in (("H", H), ("W", W)):
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{where}: {name} must be bfloat16, got {t.dtype}")
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be a contiguous matrix, got {tuple(t.shape)}")
    if labels.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{where}: labels must be int32 or int64, got {labels.dtype}")
    for name, t in (("W", W), ("labels", labels)):
        if t.device != H.device:
            raise ValueError(f"{where}: {name} is on {t.device}, H on {H.device}")
    N, d = H.shape
    if W.shape[1] != d:
        raise ValueError(f"{where}: H has {d} columns, W {W.shape[1]}")
    if labels.shape != (N,) or not labels.is_contiguous():
        raise ValueError(f"{where}: labels must be contiguous [{N}], got {tuple(labels.shape)}")
    return N, d, W.shape[0]


def token_logprobs_forward(H, W, labels, T: float = 1.0, entropy: bool = False,
                           workspace: Optional[torch.Tensor] = None
                           ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Returns (logp [N], lse [N], entropy [N] or None), fp32: with
    z = H W^T / T, lse = log sum exp z, logp = z[label] - lse and the entropy
    of softmax(z).  All are 0 where the label is negative; a label >= V gives
    NaN and is counted for ``check(workspace)``."""
    return _forward(H, W, labels, T, entropy, workspace, None)


def _forward(H, W, labels, T, entropy, workspace, kept):
    """token_logprobs_forward; logp is also written to ``kept``, if any."""
    where = "token_logprobs"
    N, d, V = _check(where, H, W, labels)
    dev = H.device
    if workspace is None:
        n = _abi.kd_token_logp_forward_workspace_size(N, d, V)
        if n == 0:
            raise ValueError(f"{where}: unsupported sizes")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        _check_workspace(workspace, dev)
    logp = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty_like(logp)
    ent = torch.empty_like(logp) if entropy else None
    with _on(dev):
        st = _abi.kd_token_logp_forward_ex(_ptr(H), _ptr(W), _ptr(labels), int(labels.dtype == torch.int64), N, d, V,
                                           float(T), _ptr(logp), _ptr(lse), _ptr(ent), _ptr(kept), _ptr(workspace),
                                           workspace.numel(), _stream(dev))
    _raise(st, "kd_token_logp_forward_ex")
    return logp, lse, ent


def token_logprobs_backward(H, W, labels, lse, dlogp, T: float = 1.0, chunk: int = LOGP_CHUNK,
                            entropy: Optional[torch.Tensor] = None, dentropy: Optional[torch.Tensor] = None,
                            dW: Optional[torch.Tensor] = None, accumulate_dW: bool = False,
                            dW_dtype: Optional[torch.dtype] = torch.float32,
                            workspace: Optional[torch.Tensor] = None, logp: Optional[torch.Tensor] = None
                            ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Returns (dH [N,d] bf16, dW [V,d]) for the upstream gradients ``dlogp``
    and, with ``entropy`` from the forward pass, ``dentropy``.  ``dW_dtype`` is
    float32, bfloat16 (rounded once, at the end) or None for dH alone; a given
    ``dW`` decides its own type, and a float32 one can be added to
    (``accumulate_dW``).  ``lse`` must come from the forward pass with the same
    inputs, and ``logp`` too: with it the 1 - p of a label that the head is
    nearly sure of keeps its relative precision, without it 1 - p is known to
    about 1e-6 (the rounding of lse).  ``chunk`` tokens' dZ rows are held at
    once."""
    where = "token_logprobs_backward"
    N, d, V = _check(where, H, W, labels)
    dev = H.device
    if (entropy is None) != (dentropy is None):
        raise ValueError(f"{where}: entropy and dentropy come together")
    for name, t in (("lse", lse), ("logp", logp), ("dlogp", dlogp), ("entropy", entropy), ("dentropy", dentropy)):
        if t is not None:
            _check_buffer(t, name, (N,), torch.float32, dev)
    if dW is not None:
        dW_dtype = dW.dtype
    if dW_dtype not in (None, torch.float32, torch.bfloat16):
        raise TypeError(f"{where}: dW must be float32 or bfloat16, got {dW_dtype}")
    if accumulate_dW and (dW is None or dW_dtype != torch.float32):
        raise ValueError(f"{where}: accumulate_dW needs a float32 dW to add to")
    if dW is not None:
        _check_buffer(dW, "dW", (V, d), dW_dtype, dev)
    if workspace is not None:
        _check_workspace(workspace, dev)
    return _backward(H, W, labels, lse, logp, dlogp, T, chunk, entropy, dentropy, dW, accumulate_dW, dW_dtype, workspace)


def _backward(H, W, labels, lse, logp, dlogp, T, chunk, entropy, dentropy, dW, accumulate_dW, dW_dtype, workspace):
    """token_logprobs_backward on checked arguments."""
    N, d = H.shape
    V = W.shape[0]
    dev = H.device
    half = int(dW_dtype == torch.bfloat16)
    if dW is None and dW_dtype is not None:
        dW = torch.empty((V, d), dtype=dW_dtype, device=dev)
    dH = torch.empty_like(H)
    if workspace is None:
        n = _abi.kd_token_logp_backward_workspace_size(N, d, V, int(chunk), half)
        if n == 0:
            raise ValueError("token_logprobs_backward: unsupported sizes")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _abi.kd_token_logp_backward_ex(_ptr(H), _ptr(W), _ptr(labels), int(labels.dtype == torch.int64), N, d, V,
                                            float(T), int(chunk), _ptr(lse), _ptr(entropy), _ptr(logp), _ptr(dlogp),
                                            _ptr(dentropy), _ptr(dH), _ptr(dW), half, int(bool(accumulate_dW)),
                                            _ptr(workspace), workspace.numel(), _stream(dev))
    _raise(st, "kd_token_logp_backward_ex")
    return dH, dW


class TokenLogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, labels, T, chunk, entropy):
        # the gradient's own copy of logp: the one returned may be changed in place
        kept = torch.empty(labels.shape, dtype=torch.float32, device=H.device) if any(ctx.needs_input_grad) else None
        logp, lse, ent = _forward(H, W, labels, T, entropy, None, kept)
        ctx.save_for_backward(H, W, labels, lse, kept, ent)
        ctx.T, ctx.chunk = T, chunk
        ctx.set_materialize_grads(False)
        return (logp, ent) if entropy else logp

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dent=None):
        if dlogp is None and dent is None:
            return (None,) * 6
        H, W, labels, lse, logp, ent = ctx.saved_tensors
        dlogp = torch.zeros_like(lse) if dlogp is None else dlogp.contiguous()
        if dent is None:                # the entropy took no part in the loss
            ent = None
        else:
            dent = dent.contiguous()
        dH, dW = _backward(H, W, labels, lse, logp, dlogp, ctx.T, ctx.chunk, ent, dent, None, False,
                           W.dtype if ctx.needs_input_grad[1] else None, None)
        return dH, dW, None, None, None, None


def token_logprobs(H, W, labels, T: float = 1.0, chunk: int = LOGP_CHUNK, entropy: bool = False):
    """Differentiable label log-probabilities [N] of softmax(H W^T / T), or
    (logp, entropy), both differentiable, with ``entropy``: see
    token_logprobs_forward.  dW comes in W's bf16 (rounded once, at the end),
    and is not computed for a frozen head; call ``token_logprobs_backward`` for
    an fp32 gradient, and the two raw calls to capture a step in a CUDA graph
    (an autograd backward pass runs on the streams of its leaves' other graphs
    too, which a capture does not allow)."""
    return TokenLogprobsFunction.apply(H, W, labels, T, chunk, entropy)
