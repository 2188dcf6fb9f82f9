"""Losses over a vocabulary from their definitions, in 64 bits on the CPU; gradients by automatic
differentiation. Used by the tests only.

Steps that do not count, and tokens that are not allowed (logits of -inf), are left out by
selection, so what stands there cannot come through."""
import math

import torch

from sequence_reference import ROUNDING, TINY

U = 2.0 ** -24
# A row's sum S of exponentials: each is within 2 ulp (4 U), its argument rounded twice (2 U |v|,
# v <= 17 bits of it where the weights are), and added up in at most 64 additions by a thread and 16
# joins of 3 roundings each: 4 + 34 + 64 + 48 < 160 U at the very worst, all roundings one way.
# log S moves by as much, absolutely; log p and H add the roundings of a few sums.
ROW = 192 * U


def close(name, got, want, scale, dtype=None):
    """|got - want| <= rounding of the type |want| + ROW scale, every element, `scale` the size of
    what the result is a sum of (a tensor that broadcasts, or a number); infinities and NaN alike."""
    dtype = dtype or got.dtype
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape, f"{name}: shape {tuple(got.shape)} != {tuple(want.shape)}"
    if not want.numel():
        return
    scale = torch.as_tensor(scale, dtype=torch.float64)
    bound = ROUNDING[dtype] * want.abs() + TINY[dtype] + ROW * scale
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= bound))
    if bad.any():
        ratio = torch.where(bad, (got - want).abs() / bound, 0.0).nan_to_num(nan=1e30)
        i = int(ratio.flatten().argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst "
                             f"{got.flatten()[i]} for {want.flatten()[i]} (at {i}, "
                             f"{float(ratio.flatten()[i]):.3g} of the bound)")


def inside(tokens, lengths, V):
    """[N, T]: the step lies inside its row, its token inside the vocabulary."""
    ok = (tokens >= 0) & (tokens < V)
    if lengths is not None:
        ok = ok & (torch.arange(tokens.shape[1]) < lengths.clamp(min=0)[:, None])
    return ok


def rows(logits, tau, counted):
    """(log p, p, counted): [N, T, V] of the steps that count and have an allowed token; others
    hold zeros in place of their logits."""
    counted = counted & (logits.detach() > -math.inf).any(-1) | counted & logits.detach().isnan().any(-1)
    x = torch.where(counted[..., None], logits, 0.0) / tau
    allowed = ~(x.detach() == -math.inf)
    m = x.detach().amax(-1, keepdim=True)
    e = torch.where(allowed, torch.exp(torch.where(allowed, x, m) - m), 0.0)
    logs = x - m - torch.log(e.sum(-1, keepdim=True))
    return logs, e / e.sum(-1, keepdim=True), counted


def taken(logs, tokens, counted):
    at = torch.where(counted, tokens.long(), 0)
    return torch.where(counted, logs.gather(-1, at[..., None])[..., 0], 0.0)


def entropy(logs, p, counted):
    some = p > 0
    h = -torch.where(some, p * torch.where(some, logs, 0.0), 0.0).sum(-1)
    h = torch.where(p.isnan().any(-1), math.nan, h)
    return torch.where(counted, h, 0.0)


def token_logprobs(logits, tokens, lengths=None, tau=1.0):
    logs, p, counted = rows(logits, tau, inside(tokens, lengths, logits.shape[-1]))
    return taken(logs, tokens, counted), entropy(logs, p, counted), counted


def policy_loss(logits, tokens, old, adv, ref=None, lengths=None, lo=0.2, hi=0.2, kl_coef=0.0,
                entropy_coef=0.0, tau=1.0):
    """(loss, logp, entropy, kl, counted)"""
    logp, h, counted = token_logprobs(logits, tokens, lengths, tau)
    old = torch.where(counted, old, 0.0)
    adv = torch.where(counted, adv, 0.0)
    ratio = torch.exp(logp - old)
    loss = torch.maximum(-ratio * adv, -ratio.clamp(1 - lo, 1 + hi) * adv)
    kl = None
    if ref is not None:
        d = torch.where(counted, ref, 0.0) - logp
        kl = torch.where(counted, torch.expm1(d) - d, 0.0)
        if kl_coef:
            loss = loss + kl_coef * kl
    if entropy_coef:
        loss = loss - entropy_coef * h
    return torch.where(counted, loss, 0.0), logp, h, kl, counted


def preference_loss(logits, tokens, ref=None, lengths=None, beta=0.1, smoothing=0.0,
                    by_length=False, tau=1.0):
    """(loss, scores, logp, counted)"""
    logp, _, counted = token_logprobs(logits, tokens, lengths, tau)
    ratio = logp if ref is None else logp - torch.where(counted, ref, 0.0)
    scores = beta * torch.where(counted, ratio, 0.0).sum(1)
    if by_length:
        scores = scores / counted.sum(1).clamp(min=1)
    half = logits.shape[0] // 2
    x = scores[:half] - scores[half:]
    soft = lambda v: torch.logaddexp(v, torch.zeros_like(v))
    return (1 - smoothing) * soft(-x) + smoothing * soft(x), scores, logp, counted


def distill_topk(logits, index, teacher, lengths=None, tau=1.0):
    """(loss, counted)"""
    N, T, V = logits.shape
    good = (index >= 0) & (index < V) & (teacher > -math.inf) | (index >= 0) & (index < V) \
        & teacher.isnan()
    if lengths is not None:
        good = good & (torch.arange(T) < lengths.clamp(min=0)[:, None])[..., None]
    logs, _, counted = rows(logits, tau, good.any(-1))
    good = good & counted[..., None]
    t = torch.where(good, teacher / tau, -math.inf)
    t = t - torch.where(counted, t.amax(-1), 0.0)[..., None] if t.shape[-1] else t
    q = torch.exp(t)
    q = torch.where(good, q / q.sum(-1, keepdim=True), 0.0)
    lq = torch.where(good, torch.log(torch.where(q > 0, q, 1.0)), 0.0)
    lp = logs.gather(-1, torch.where(good, index.long(), 0))
    loss = torch.where(q > 0, q * (lq - lp), 0.0).sum(-1)
    return torch.where(counted, loss, 0.0), counted
