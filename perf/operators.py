"""The post-training losses at the LM head, as they are measured.

Three operators and the two training steps they make together:

* label log-probabilities of hidden states under the head (and the entropy of
  each token's distribution), with the gradients of both: scoring and training;
* the preference loss over paired sequences of token log-probabilities;
* the clipped policy loss with a KL term over token log-probabilities;
* a preference step and a policy step: log-probabilities, loss, head gradients.

Every case is run in its plain form (elementary torch operations in 32 bits,
64 where 32 lose what matters) or, with ``own``, through the framework's public
calls.  ``exact`` gives the same results from the definitions in 64 bits.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
PROMPT_BLOCK = 64      # in a labelled batch, the last part of every 64 tokens is prompt (no label)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One token scored under a 201,088-entry head: the serving form, W's bytes are all of it.
        _head("score_one_token", N=1, d=2880, V=201088, ignored=0.0, T=1.0, entropy=False, grad=False),
        # A ragged batch scored for a reference or behaviour policy at sampling temperature 0.8, with
        # entropies for monitoring; 35 % of the tokens are prompt.
        _head("score_batch", N=3001, d=2048, V=128256, ignored=0.35, T=0.8, entropy=True, grad=False),
        # Log-probabilities and their gradients for a small student head with an odd vocabulary.
        _head("logp_grad_small", N=257, d=1000, V=32001, ignored=0.25, T=1.0, entropy=False, grad=True),
        # The large head, 8K tokens of which 40 % are prompt, with an entropy bonus' gradient.
        _head("logp_grad_large", N=8192, d=2880, V=201088, ignored=0.4, T=1.0, entropy=True, grad=True),
        # A micro-batch of four short preference pairs: launch latency.
        _pref("pref_few_short", pairs=4, mean=120, padded=False, kind="sigmoid", smoothing=0.0, average=False,
              reference=True, layout=1),
        # An ordinary preference batch, packed, of long and short answers.
        _pref("pref_batch", pairs=64, mean=1500, padded=False, kind="sigmoid", smoothing=0.1, average=False,
              reference=True, layout=2),
        # Long-context pairs in a padded batch, length-averaged.
        _pref("pref_long_padded", pairs=64, mean=20000, padded=True, kind="ipo", smoothing=0.0, average=True,
              reference=True, layout=3),
        # A handful of short rollouts, one advantage per sequence: launch latency.
        _policy("policy_few_short", seqs=8, mean=150, padded=False, per_seq=True, reduce="token", kl="k3", dual=0.0,
                layout=4),
        # An ordinary rollout batch, packed, token advantages, loss averaged over tokens.
        _policy("policy_batch", seqs=512, mean=1000, padded=False, per_seq=False, reduce="token", kl="k3", dual=0.0,
                layout=5),
        # A large padded rollout batch, group advantages, averaged per sequence, dual clip.
        _policy("policy_large_padded", seqs=4096, mean=1800, padded=True, per_seq=True, reduce="sequence", kl="k2",
                dual=3.0, layout=6),
        # A preference step at the long-context sweep's head: log-probabilities, loss, dH and dW.
        _step("preference_step", "pref_step", seqs=16, mean=256, d=2048, V=128256, layout=7),
        # A policy step at the 201,088-entry head.
        _step("policy_step", "policy_step", seqs=9, mean=220, d=2880, V=201088, layout=8),
    ]


def _head(name, **k):
    return {"name": name, "op": "head", **k}


def _pref(name, **k):
    return {"name": name, "op": "pref", **k}


def _policy(name, **k):
    return {"name": name, "op": "policy", **k}


def _step(name, op, **k):
    return {"name": name, "op": op, **k}


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("head", "head", "pref", "policy", "policy", "pref_step", "policy_step"))
    layout = rng.randrange(1 << 20)
    if op == "head":
        return {"op": op, "N": _log_uniform(rng, 1, 6000), "d": 8 * _log_uniform(rng, 8, 360),
                "V": _log_uniform(rng, 1000, 201088), "ignored": rng.choice((0.0, 0.2, 0.55)),
                "T": rng.choice((1.0, 0.7, 1.3)), "entropy": rng.random() < 0.5, "grad": rng.random() < 0.6}
    if op == "pref":
        pairs, mean = _log_uniform(rng, 1, 256), _log_uniform(rng, 4, 8000)
        return {"op": op, "pairs": pairs, "mean": min(mean, 2_000_000 // (2 * pairs)), "padded": rng.random() < 0.4,
                "kind": rng.choice(("sigmoid", "hinge", "ipo")), "smoothing": rng.choice((0.0, 0.05)),
                "average": rng.random() < 0.4, "reference": rng.random() < 0.8, "layout": layout}
    if op == "policy":
        seqs, mean = _log_uniform(rng, 1, 4096), _log_uniform(rng, 3, 4000)
        return {"op": op, "seqs": seqs, "mean": min(mean, 6_000_000 // seqs), "padded": rng.random() < 0.4,
                "per_seq": rng.random() < 0.5, "reduce": rng.choice(("token", "sequence")),
                "kl": rng.choice(("k1", "k2", "k3")), "dual": rng.choice((0.0, 3.0)), "layout": layout}
    return {"op": op, "seqs": 2 * _log_uniform(rng, 1, 8), "mean": _log_uniform(rng, 8, 250),
            "d": 8 * _log_uniform(rng, 16, 256), "V": _log_uniform(rng, 4000, 130000), "layout": layout}


def _lengths(case):
    """The case's sequence lengths, skewed as answers' lengths are: the same for every seed."""
    rng = random.Random(case["layout"])
    n = 2 * case["pairs"] if case["op"] == "pref" else case["seqs"]
    return [max(1, int(case["mean"] * min(3.0, rng.lognormvariate(-0.1, 0.5)))) for _ in range(n)]


def _tokens(case):
    """Token slots of a loss case's arrays: padding included."""
    lens = _lengths(case)
    return max(lens) * len(lens) if case.get("padded") else sum(lens)


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _head_inputs(g, N, d, V):
    """Hidden states whose labels are likely to a spread of degrees, as under a trained head."""
    W = torch.empty(V, d, device=DEV, dtype=torch.bfloat16)
    for lo in range(0, V, 32768):
        W[lo:lo + 32768] = torch.randn(min(32768, V - lo), d, device=DEV, generator=g) * (1.1 / math.sqrt(d))
    labels = torch.randint(0, V, (N,), device=DEV, generator=g)
    pull = 14.0 * torch.rand(N, 1, device=DEV, generator=g) / 1.21
    H = (torch.randn(N, d, device=DEV, generator=g) + pull * W[labels].float()).to(torch.bfloat16)
    return H, W, labels


def _ignored(N, share):
    """Which tokens of a batch of N are prompt (a pattern of the sizes alone)."""
    return [i % PROMPT_BLOCK >= (1 - share) * PROMPT_BLOCK for i in range(N)]


def _loss_inputs(case, g):
    """Token log-probabilities as the new, the behaviour and the reference policy give them."""
    lens = torch.tensor(_lengths(case), device=DEV, dtype=torch.int64)
    S = lens.numel()
    st = {"S": S}
    if case.get("padded"):
        L = max(_lengths(case))
        shape = (S, L)
        pos = torch.arange(L, device=DEV)[None, :]
        prompt = (lens // 8)[:, None]
        st["mask"] = ((pos < lens[:, None]) & (pos >= prompt)).float()
        st["offsets"] = None
    else:
        shape = (int(sum(_lengths(case))),)
        st["offsets"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
        start = st["offsets"][:-1].repeat_interleave(lens)
        prompt = (lens // 8).repeat_interleave(lens)
        st["mask"] = (torch.arange(shape[0], device=DEV) - start >= prompt).float()
    base = -torch.empty(shape, device=DEV).exponential_(1.0, generator=g)
    st["ref"] = base
    st["old"] = base + 0.15 * torch.randn(shape, device=DEV, generator=g)
    st["logp"] = st["old"] + 0.12 * torch.randn(shape, device=DEV, generator=g)
    if case["op"] == "policy":
        a = torch.randn((S,) if case["per_seq"] else shape, device=DEV, generator=g)
        st["adv"] = a
    return st


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("pref", "policy"):
        st.update(_loss_inputs(case, g))
        return st
    if op == "head":
        N = case["N"]
        H, W, labels = _head_inputs(g, N, case["d"], case["V"])
        labels[torch.tensor(_ignored(N, case["ignored"]), device=DEV)] = -1
        st["dlogp"] = torch.randn(N, device=DEV, generator=g) / N
        st["dent"] = torch.randn(N, device=DEV, generator=g) / N
    else:
        lens = torch.tensor(_lengths(case), device=DEV, dtype=torch.int64)
        N = int(sum(_lengths(case)))
        H, W, labels = _head_inputs(g, N, case["d"], case["V"])
        st["offsets"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
        start = st["offsets"][:-1].repeat_interleave(lens)
        pos = torch.arange(N, device=DEV) - start
        labels[pos < (lens // 4).repeat_interleave(lens)] = -1      # the prompts
        st["mask"] = (labels >= 0).float()
        st["ref"] = -torch.empty(N, device=DEV).exponential_(0.2, generator=g)
        st["adv"] = torch.randn(lens.numel(), device=DEV, generator=g)
    if op == "policy_step":
        # the behaviour policy's record: near the new policy's log-probabilities
        old = torch.empty(N, device=DEV)
        Wt = W.float().T
        for lo in range(0, N, 512):
            z = H[lo:lo + 512].float() @ Wt
            old[lo:lo + 512] = z.gather(1, labels[lo:lo + 512, None].clamp(min=0)).squeeze(1) - torch.logsumexp(z, 1)
        x = 0.12 * torch.randn(N, device=DEV, generator=g)
        for border in (math.log(1.2), math.log(0.8)):     # a 32-bit product's rounding decides no token's clipping
            x = torch.where((x - border).abs() < 5e-4, border - 1e-3, x)
        st["old"] = old - x
        st["ref"] = old + 0.2 * torch.randn(N, device=DEV, generator=g)
    st["H"], st["W"], st["labels"] = H, W, labels
    if op != "head" or case["grad"]:
        H.requires_grad_(True)
        W.requires_grad_(True)
    return st


# ---------------------------------------------------------------- one pass

STEP_BETA = 0.1
STEP_KL, STEP_ENTROPY = 0.02, 0.01


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _pref_args(case):
    return dict(beta=0.1, kind=case["kind"], label_smoothing=case["smoothing"], average=case["average"])


def _policy_args(case):
    return dict(clip_low=0.2, clip_high=0.25, dual_clip=case["dual"] or None, kl_coef=0.02, kl=case["kl"],
                reduce=case["reduce"])


def _run_own(st):
    import chunked_top_kl_b200 as kd
    case = st["case"]
    op = case["op"]
    if op == "head":
        out = kd.token_logprobs(st["H"], st["W"], st["labels"], T=case["T"], entropy=case["entropy"])
        out = out if case["entropy"] else (out,)
        if not case["grad"]:
            return {"out": out}
        up = (st["dlogp"], st["dent"])[:len(out)]
        dH, dW = torch.autograd.grad(out, (st["H"], st["W"]), up)
        return {"out": [o.detach() for o in out], "dH": dH, "dW": dW}
    if op == "pref":
        loss, chosen, rejected, dlogp = kd.preference_loss_forward_backward(
            st["logp"], st["ref"] if case["reference"] else None, mask=st["mask"], offsets=st["offsets"],
            **_pref_args(case))
        return {"loss": loss, "chosen": chosen, "rejected": rejected, "dlogp": dlogp}
    if op == "policy":
        loss, kl, clipped, dlogp = kd.policy_loss_forward_backward(
            st["logp"], st["old"], st["adv"], ref_logp=st["ref"], mask=st["mask"], offsets=st["offsets"],
            **_policy_args(case))
        return {"loss": loss, "kl": kl, "clipped": clipped, "dlogp": dlogp}
    if op == "pref_step":
        logp = kd.token_logprobs(st["H"], st["W"], st["labels"])
        loss, chosen, rejected = kd.preference_loss(logp, st["ref"], mask=st["mask"], offsets=st["offsets"],
                                                    beta=STEP_BETA)
        dH, dW = torch.autograd.grad(loss, (st["H"], st["W"]))
        return {"loss": loss.detach(), "chosen": chosen, "rejected": rejected, "dH": dH, "dW": dW}
    logp, ent = kd.token_logprobs(st["H"], st["W"], st["labels"], entropy=True)
    loss, kl, clipped = kd.policy_loss(logp, st["old"], st["adv"], ref_logp=st["ref"], mask=st["mask"],
                                       offsets=st["offsets"], kl_coef=STEP_KL)
    loss = loss - STEP_ENTROPY * (ent * st["mask"]).sum() / st["mask"].sum()
    dH, dW = torch.autograd.grad(loss, (st["H"], st["W"]))
    return {"loss": loss.detach(), "kl": kl, "clipped": clipped, "dH": dH, "dW": dW}


# ---------------------------------------------------------------- plain forms

def _plain_logp(H, W, labels, T):
    """logp, entropy, the probabilities p [N,V] and log p, all in 32 bits (vocabulary sums in 64)."""
    z = H.float() @ W.float().T
    if T != 1.0:
        z /= T
    m = z.amax(1, keepdim=True)
    lse = m.double() + torch.exp(z - m).sum(1, keepdim=True, dtype=torch.float64).log()
    logq = z.sub_(lse.float())
    live = labels >= 0
    logp = torch.where(live, logq.gather(1, labels.clamp(min=0)[:, None]).squeeze(1), 0.0)
    p = torch.exp(logq)
    ent = torch.where(live, -(p * logq).sum(1, dtype=torch.float64), 0.0).float()
    return logp, ent, p, logq


def _plain_head_grad(H, W, labels, T, p, logq, ent, dlogp, dent):
    live = labels >= 0
    g = torch.where(live, dlogp, 0.0)
    if dent is None:
        dz = p.mul_(-g[:, None])
    else:
        h = torch.where(live, dent, 0.0)[:, None]
        dz = logq.add_(ent[:, None]).mul_(h).add_(g[:, None]).neg_().mul_(p)
    dz.scatter_add_(1, labels.clamp(min=0)[:, None], g[:, None])
    if T != 1.0:
        dz /= T
    return (dz @ W.float()).to(H.dtype), (dz.T @ H.float()).to(W.dtype)


def _sequence_of(st, N):
    """Each token slot's sequence."""
    t = torch.arange(N, device=DEV)
    if st["offsets"] is None:
        return t // (N // st["S"])
    return torch.searchsorted(st["offsets"][1:].long(), t, right=True)


def _per_sequence(st, values):
    """Sums over each sequence, in 64 bits."""
    v = values.double()
    if st["offsets"] is None:
        return v.reshape(st["S"], -1).sum(1)
    total = torch.cat([v.new_zeros(1), v.cumsum(0)])[st["offsets"].long()]
    return total[1:] - total[:-1]


def _plain_pref(st, logp, ref, mask, beta, kind, label_smoothing, average):
    m, seq = mask.reshape(-1), _sequence_of(st, mask.numel())
    x = logp.reshape(-1).double() - (0.0 if ref is None else ref.reshape(-1).double())
    r = _per_sequence(st, torch.where(m != 0, m * x, 0.0))
    w = torch.ones_like(r)
    if average:
        n = _per_sequence(st, m)
        w = torch.where(n != 0, 1.0 / n, 0.0)
    r = r * w
    P = r.numel() // 2
    diff = r[:P] - r[P:]
    d = beta * diff
    if kind == "sigmoid":
        soft = lambda v: torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))   # log(1 + e^v)  # noqa: E731
        loss = (1 - label_smoothing) * soft(-d) + label_smoothing * soft(d)
        slope = beta * (1.0 / (1.0 + torch.exp(-d)) - (1 - label_smoothing))
    elif kind == "hinge":
        loss = torch.clamp(1 - d, min=0)
        slope = torch.where(d < 1, -beta, 0.0)
    else:
        e = diff - 1 / (2 * beta)
        loss, slope = e * e, 2 * e
    coef = torch.cat([slope, -slope]) * w / P
    dlogp = torch.where(m != 0, coef[seq] * m, 0.0).float().reshape(logp.shape)
    return loss.mean().float(), (beta * r[:P]).float(), (beta * r[P:]).float(), dlogp


def _plain_policy(st, logp, old, adv, ref, mask, per_seq, clip_low, clip_high, dual_clip, kl_coef, kl, reduce):
    m, seq = mask.reshape(-1), _sequence_of(st, mask.numel())
    lp = logp.reshape(-1).double()
    a = adv[seq] if per_seq else adv.reshape(-1)
    x = lp - old.reshape(-1).double()              # 64 bits: tokens next to a clip border
    hi, lo = math.log1p(clip_high), math.log1p(-clip_low)
    ratio = torch.exp(x.float())
    clipped = ((a > 0) & (x > hi)) | ((a < 0) & (x < lo))
    obj = torch.minimum(ratio * a, torch.clamp(ratio, 1 - clip_low, 1 + clip_high) * a)
    if dual_clip is not None:
        far = (a < 0) & (x > math.log(dual_clip))
        obj = torch.where(far, dual_clip * a, obj)
        clipped = clipped | far
    grad = torch.where(clipped, 0.0, -ratio * a)
    y = lp - ref.reshape(-1).double()              # 64 bits: e^-y - 1 + y cancels
    if kl == "k1":
        k, dk = y, torch.ones_like(y)
    elif kl == "k2":
        k, dk = 0.5 * y * y, y
    else:
        k, dk = torch.expm1(-y) + y, -torch.expm1(-y)
    token = -obj + kl_coef * k
    if reduce == "token":
        total = m.sum(dtype=torch.float64)
        w = torch.where(total != 0, 1.0 / total, 0.0) * m
    else:
        n = _per_sequence(st, m)
        w = (torch.where(n != 0, 1.0 / n, 0.0) / n.numel())[seq] * m
    mean = lambda v: torch.where(m != 0, w * v, 0.0).sum(dtype=torch.float64).float()   # noqa: E731
    dlogp = torch.where(m != 0, w * (grad + kl_coef * dk), 0.0).float().reshape(logp.shape)
    return mean(token), mean(k), mean(clipped.double()), dlogp


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "pref":
        out = _plain_pref(st, st["logp"], st["ref"] if case["reference"] else None, st["mask"], **_pref_args(case))
        return dict(zip(("loss", "chosen", "rejected", "dlogp"), out))
    if op == "policy":
        out = _plain_policy(st, st["logp"], st["old"], st["adv"], st["ref"], st["mask"], case["per_seq"],
                            **_policy_args(case))
        return dict(zip(("loss", "kl", "clipped", "dlogp"), out))
    H, W, labels = st["H"].detach(), st["W"].detach(), st["labels"]
    T = case.get("T", 1.0)
    logp, ent, p, logq = _plain_logp(H, W, labels, T)
    if op == "head":
        out = [logp, ent] if case["entropy"] else [logp]
        if not case["grad"]:
            return {"out": out}
        dH, dW = _plain_head_grad(H, W, labels, T, p, logq, ent, st["dlogp"], st["dent"] if case["entropy"] else None)
        return {"out": out, "dH": dH, "dW": dW}
    if op == "pref_step":
        loss, chosen, rejected, dlogp = _plain_pref(st, logp, st["ref"], st["mask"], STEP_BETA, "sigmoid", 0.0, False)
        dH, dW = _plain_head_grad(H, W, labels, T, p, logq, ent, dlogp, None)
        return {"loss": loss, "chosen": chosen, "rejected": rejected, "dH": dH, "dW": dW}
    loss, kl, clipped, dlogp = _plain_policy(st, logp, st["old"], st["adv"], st["ref"], st["mask"], True, 0.2, 0.2, None,
                                             STEP_KL, "k3", "token")
    n = st["mask"].sum()
    loss = loss - STEP_ENTROPY * (ent * st["mask"]).sum() / n
    dH, dW = _plain_head_grad(H, W, labels, T, p, logq, ent, dlogp, -STEP_ENTROPY * st["mask"] / n)
    return {"loss": loss, "kl": kl, "clipped": clipped, "dH": dH, "dW": dW}


# ---------------------------------------------------------------- work

def work(case):
    """What one pass cannot do without: inputs read once, outputs written once, the products of the labelled rows."""
    op = case["op"]
    if op in ("pref", "policy"):
        n = _tokens(case)
        S = len(_lengths(case))
        if op == "pref":
            arrays = 2 + (1 if case["reference"] else 0)                # logp, mask, ref
            return {"bytes": 4 * n * (arrays + 1) + 8 * S, "flops": 8 * n}
        arrays = 4 + (0 if case["per_seq"] else 1)                       # logp, old, ref, mask, advantages
        return {"bytes": 4 * n * (arrays + 1) + 8 * S, "flops": 40 * n}
    d, V = case["d"], case["V"]
    if op == "head":
        N = case["N"]
        live = N - sum(_ignored(N, case["ignored"]))
        grad, extra = case["grad"], 8 * N + 4 * N * (2 if case["entropy"] else 1)
    else:
        lens = _lengths(case)
        N, live = sum(lens), sum(n - n // 4 for n in lens)
        grad, extra = True, 8 * N + 16 * N
    size = 2 * live * d + 2 * V * d
    if not grad:
        return {"bytes": size + extra, "flops": 2 * live * d * V}
    return {"bytes": size + extra + 4 * N + 2 * N * d + 2 * V * d, "flops": 6 * live * d * V}


# ---------------------------------------------------------------- 64 bits

def _bounds(st, N):
    """Each sequence's [begin, end) on the host."""
    if st.get("offsets") is None:
        L = N // st["S"]
        return [(s * L, (s + 1) * L) for s in range(st["S"])]
    o = st["offsets"].tolist()
    return list(zip(o[:-1], o[1:]))


def _exact_pref(logp, ref, mask, bounds, beta, kind, label_smoothing, average):
    lp, m = logp.double().reshape(-1), mask.double().reshape(-1)
    x = lp if ref is None else lp - ref.double().reshape(-1)
    r, n = [], []
    for b, e in bounds:
        r.append((m[b:e] * x[b:e]).sum())
        n.append(m[b:e].sum())
    r, n = torch.stack(r), torch.stack(n)
    scale = n.reciprocal().masked_fill(n == 0, 0.0) if average else torch.ones_like(n)
    r = (r * scale).requires_grad_(True)
    P = len(bounds) // 2
    gap = r[:P] - r[P:]
    if kind == "sigmoid":
        s = torch.sigmoid(beta * gap)
        each = -(1 - label_smoothing) * torch.log(s) - label_smoothing * torch.log1p(-s)
    elif kind == "hinge":
        each = torch.relu(1 - beta * gap)
    else:
        each = (gap - 0.5 / beta) ** 2
    loss = each.sum() / P
    (dr,) = torch.autograd.grad(loss, r)
    dlogp = torch.zeros_like(lp)
    for s, (b, e) in enumerate(bounds):
        dlogp[b:e] = dr[s] * scale[s] * m[b:e]
    r = r.detach()
    return loss.detach(), beta * r[:P], beta * r[P:], dlogp.reshape(logp.shape)


def _exact_policy(logp, old, adv, ref, mask, bounds, per_seq, clip_low, clip_high, dual_clip, kl_coef, kl, reduce):
    lp = logp.double().reshape(-1).clone().requires_grad_(True)
    m = mask.double().reshape(-1)
    w, a = torch.zeros_like(m), torch.zeros_like(m)
    whole = m.sum()
    sums = [m[b:e].sum() for b, e in bounds]
    for s, (b, e) in enumerate(bounds):
        if reduce == "token":
            w[b:e] = m[b:e] / whole if float(whole) != 0 else 0.0
        elif float(sums[s]) != 0:
            w[b:e] = m[b:e] / sums[s] / len(bounds)
        if per_seq:
            a[b:e] = adv[s].double()
    if not per_seq:
        a = adv.double().reshape(-1)
    ratio = torch.exp(lp - old.double().reshape(-1))
    obj = torch.where(a >= 0, torch.clamp(ratio, max=1 + clip_high) * a, torch.clamp(ratio, min=1 - clip_low) * a)
    out = torch.where(a > 0, ratio > 1 + clip_high, (a < 0) & (ratio < 1 - clip_low))
    if dual_clip is not None:
        obj = torch.where(a < 0, torch.maximum(obj, dual_clip * a), obj)
        out = out | ((a < 0) & (ratio > dual_clip))
    y = lp - ref.double().reshape(-1)
    k = {"k1": y, "k2": y * y / 2, "k3": torch.expm1(-y) + y}[kl]
    loss = (w * (kl_coef * k - obj)).sum()
    (dlogp,) = torch.autograd.grad(loss, lp)
    return (loss.detach(), (w * k).sum().detach(), (w * out.double()).sum().detach(), dlogp.reshape(logp.shape))


def _exact_head(H, W, labels, T, dlogp=None, dent=None, rows=1024):
    """logp, entropy and, for upstream gradients (tensors, or a function of logp that gives them), dH and dW."""
    Wd = W.double()
    N = H.shape[0]
    lse = torch.empty(N, device=DEV, dtype=torch.float64)
    logp, ent = torch.zeros_like(lse), torch.zeros_like(lse)
    live = labels >= 0

    def logits(lo):
        return (H[lo:lo + rows].double() @ Wd.T) / T

    for lo in range(0, N, rows):
        z = logits(lo)
        c = slice(lo, lo + rows)
        lse[c] = torch.logsumexp(z, 1)
        logp[c] = z.gather(1, labels[c].clamp(min=0)[:, None]).squeeze(1) - lse[c]
        ent[c] = lse[c] - (torch.softmax(z, 1) * z).sum(1)
    logp, ent = logp * live, ent * live
    if dlogp is None:
        return logp, ent
    extra = ()
    if callable(dlogp):
        dlogp, dent, *extra = dlogp(logp, ent)
    dH = torch.zeros(N, H.shape[1], device=DEV, dtype=torch.float64)
    dW = torch.zeros(Wd.shape, device=DEV, dtype=torch.float64)
    for lo in range(0, N, rows):
        c = slice(lo, lo + rows)
        logq = logits(lo) - lse[c, None]
        q = torch.exp(logq)
        g = (dlogp[c].double() * live[c])[:, None]
        dz = -g * q
        if dent is not None:
            dz -= (dent[c].double() * live[c])[:, None] * q * (logq + ent[c, None])
        dz.scatter_add_(1, labels[c].clamp(min=0)[:, None], g)
        dz /= T
        dH[c] = dz @ Wd
        dW += dz.T @ H[c].double()
    return (logp, ent, dH, dW, *extra)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("pref", "policy"):
        b = _bounds(st, st["logp"].numel())
        if op == "pref":
            out = _exact_pref(st["logp"], st["ref"] if case["reference"] else None, st["mask"], b, **_pref_args(case))
            return dict(zip(("loss", "chosen", "rejected", "dlogp"), out))
        out = _exact_policy(st["logp"], st["old"], st["adv"], st["ref"], st["mask"], b, case["per_seq"],
                            **_policy_args(case))
        return dict(zip(("loss", "kl", "clipped", "dlogp"), out))
    H, W, labels = st["H"].detach(), st["W"].detach(), st["labels"]
    if op == "head":
        if not case["grad"]:
            out = _exact_head(H, W, labels, case["T"])
            return {"out": list(out[:2 if case["entropy"] else 1])}
        logp, ent, dH, dW = _exact_head(H, W, labels, case["T"], st["dlogp"], st["dent"] if case["entropy"] else None)
        return {"out": [logp, ent] if case["entropy"] else [logp], "dH": dH, "dW": dW}
    b = _bounds(st, labels.numel())
    if op == "pref_step":
        def up(logp, ent):
            loss, chosen, rejected, dlogp = _exact_pref(logp, st["ref"], st["mask"], b, STEP_BETA, "sigmoid", 0.0, False)
            return dlogp, None, loss, chosen, rejected
        _, _, dH, dW, loss, chosen, rejected = _exact_head(H, W, labels, 1.0, up)
        return {"loss": loss, "chosen": chosen, "rejected": rejected, "dH": dH, "dW": dW}

    def up(logp, ent):
        loss, kl, clipped, dlogp = _exact_policy(logp, st["old"], st["adv"], st["ref"], st["mask"], b, True, 0.2, 0.2,
                                                 None, STEP_KL, "k3", "token")
        m = st["mask"].double()
        loss = loss - STEP_ENTROPY * (ent * m).sum() / m.sum()
        return dlogp, -STEP_ENTROPY * m / m.sum(), loss, kl, clipped
    _, _, dH, dW, loss, kl, clipped = _exact_head(H, W, labels, 1.0, up)
    return {"loss": loss, "kl": kl, "clipped": clipped, "dH": dH, "dW": dW}
