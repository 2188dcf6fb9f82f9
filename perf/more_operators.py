"""Losses over a vocabulary as measurable cases: what a policy that the estimators credit is
trained with. Log-probabilities of taken tokens with their entropy, the clipped policy loss with
its KL term, the preference loss of pairs and the distillation from a teacher's top logits, each
with its gradient, in plain form (elementary torch operations in 32 bits) and through the
framework's entry points, with a 64-bit definition to compare both with.

Rows are environments (or prompts), steps are tokens (or actions). A token outside the vocabulary
(prompt, padding) and a step past its row's length do not count: their outputs and gradients
are 0.
"""
import math

import torch

own = False

_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


def _case(name, op, N, T, V, dtype, **kw):
    base = dict(name=name, op=op, N=N, T=T, V=V, dtype=dtype, shifted=False, prompt=False,
                ragged=False, masked=False, entropy=False, temperature=1.0)
    base.update(kw)
    return base


def listed():
    return [
        # Acting: the log-probability of one sampled token for each of a few rows; latency counts.
        _case("logprob_act_16", "logprob", 16, 1, 32768, "bf16", entropy=True),
        # A frozen reference model scores a ragged batch of answers to prompts: an odd vocabulary,
        # half of the steps uncounted, a temperature.
        _case("logprob_ref_ragged", "logprob", 33, 517, 50001, "fp16", shifted=True, prompt=True,
              ragged=True, temperature=0.7),
        # A small model's log-probabilities and entropies with gradients into both, fp32.
        _case("logprob_train_odd", "logprob_train", 7, 300, 1027, "fp32", entropy=True,
              ragged=True),
        # One update of a token policy: losses, KL to a reference, entropy and the gradient.
        _case("policy_16x1024", "policy", 16, 1024, 32768, "bf16", shifted=True, kl=True,
              entropy=True),
        # Ragged answers behind prompts, an odd vocabulary in fp16, without an entropy term.
        _case("policy_ragged", "policy", 24, 700, 50001, "fp16", shifted=True, prompt=True,
              ragged=True, kl=True),
        # Discrete actions of many environments, a quarter of them not allowed (logits of -inf).
        _case("policy_actions", "policy", 4096, 512, 18, "fp32", masked=True, kl=False,
              entropy=True),
        # A small token environment: little work, latency counts.
        _case("policy_small", "policy", 16, 128, 512, "fp32", kl=True, entropy=True),
        # Eight pairs of answers, forward and gradient.
        _case("preference_16x1024", "preference", 16, 1024, 32768, "bf16", shifted=True,
              prompt=True, by_length=False, smoothing=0.0),
        # A small model's pairs, by length, with smoothed labels.
        _case("preference_odd", "preference", 6, 77, 5003, "fp32", shifted=True, ragged=True,
              by_length=True, smoothing=0.1),
        # Distillation from 64 stored logits for each step.
        _case("distill_16x512", "distill", 16, 512, 50000, "bf16", K=64, teacher="bf16"),
        # A small student, few stored logits in fp32, a temperature.
        _case("distill_small", "distill", 8, 65, 2000, "fp16", K=20, teacher="fp32", ragged=True,
              temperature=2.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["logprob", "logprob_train", "policy", "policy", "preference", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    V = _log(rng, 64 if op in ("preference", "distill") else 2, 131072)
    even = 2 if op == "preference" else 1
    # At most the logits of the largest listed case, and at most 2 Mi steps.
    steps = min((1 << 30) // (_BYTES[dtype] * V), 1 << 21)
    T = _log(rng, 1, min(1024, max(1, steps // even)))
    N = even * _log(rng, 1, max(1, min(4096, steps // (even * (T + 1)))))
    c = dict(op=op, N=N, T=T, V=V, dtype=dtype, shifted=rng.random() < 0.5,
             prompt=rng.random() < 0.3, ragged=rng.random() < 0.3,
             masked=op != "distill" and rng.random() < 0.2,
             entropy=op not in ("preference", "distill") and rng.random() < 0.5,
             temperature=rng.choice([1.0, 1.0, 0.7, 1.5]))
    if op == "policy":
        c["kl"] = rng.random() < 0.6
    if op == "preference":
        c["by_length"] = rng.random() < 0.3
        c["smoothing"] = rng.choice([0.0, 0.1])
    if op == "distill":
        c["prompt"] = False
        c["K"] = min(V, _log(rng, 1, 256))
        c["teacher"] = rng.choice([dtype, "fp32"])
    return c


# ------------------------------------------------------------------------------ inputs

CLIP_LOW, CLIP_HIGH, KL_COEF, ENTROPY_COEF, BETA = 0.2, 0.28, 0.05, 0.01, 0.1


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    op, N, T, V = case["op"], case["N"], case["T"], case["V"]
    tau = case["temperature"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device=dev, generator=gen) * std

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen)

    s = {"case": case, "lengths": None}
    # A model gives logits for every token it reads; the last one's and the first token are not
    # used, so both are slices of wider buffers.
    wide = T + 1 if case["shifted"] else T
    logits = torch.randn(N, wide, V, device=dev, generator=gen, dtype=dt).mul_(2.0)[:, :T]
    if case["masked"]:
        block = (uniform(N, T, V) < 0.25)
        block[..., 0] = False
        logits.masked_fill_(block, -math.inf)
        del block
    # Taken tokens: mostly ones that the model finds likely.
    taken = torch.zeros(N, wide, dtype=torch.int64, device=dev)[:, wide - T:]
    choice = (uniform(N, T) * V).long().clamp_(max=V - 1)
    if case["masked"]:
        allowed = torch.isfinite(logits.gather(2, choice[..., None])[..., 0])
        choice = torch.where(allowed, choice, 0)
    taken.copy_(choice)
    boost = torch.where(uniform(N, T) < 0.8, math.log(V) + normal(N, T, std=2.0), 0.0).to(dt)
    logits.scatter_add_(2, taken[..., None], boost[..., None])
    s["logits"] = logits
    if case["ragged"]:
        lengths = (uniform(N) * (T + 1)).int().clamp_(0, T)
        lengths[0] = T
        if N > 2:
            lengths[N // 2] = 0
        s["lengths"] = lengths
    if case["prompt"]:
        first = (uniform(N, 1) * T * 0.5).long()
        taken.masked_fill_(torch.arange(T, device=dev) < first, -1)
    s["tokens"] = taken
    counted = _counted(s, N, T)
    # Losses are means over the counted steps; fp16 gradients are scaled.
    scale = 65536.0 if case["dtype"] == "fp16" else 1.0
    weight = counted.float() * (scale / counted.sum().clamp(min=1))
    if op == "logprob_train":
        s["dlogp"] = normal(N, T) * weight
        s["dentropy"] = normal(N, T, std=0.1) * weight if case["entropy"] else None
    if op in ("policy", "preference"):
        logp = logits.gather(2, taken.clamp(min=0)[..., None])[..., 0].float() / tau \
            - torch.logsumexp(logits.float() / tau, 2)
    if op == "policy":
        # The policy has moved since the tokens were sampled. No ratio lies within 1e-3 of a border
        # of the clipping, where rounding alone would decide on its side.
        moved = normal(N, T, std=0.15)
        for border in (math.log1p(-CLIP_LOW), math.log1p(CLIP_HIGH)):
            near = (moved - border).abs() < 2e-3
            moved = torch.where(near, moved + 4e-3, moved)
        s["old"] = logp - moved
        s["ref"] = logp + normal(N, T, std=0.3) if case["kl"] else None
        s["advantage"] = normal(N, T)
        s["weight"] = weight
    if op == "preference":
        s["ref"] = logp + normal(N, T, std=0.3)
        s["dloss"] = torch.full((N // 2,), scale * 2 / N, device=dev)
    if op == "distill":
        K = case["K"]
        # A teacher that agrees with the student in part; a few of its entries are not in the
        # student's vocabulary.
        order = torch.topk(logits, K, dim=2)
        index = order.indices
        s["index"] = torch.where(uniform(N, T, K) < 0.02, -1, index)
        s["teacher"] = (order.values.float() + normal(N, T, K)).to(_DTYPES[case["teacher"]])
        s["weight"] = torch.full((N, T), scale / (N * T), device=dev)
    return s


# --------------------------------------------------------------------------- plain form


def _counted(s, N, T):
    """Steps that count: inside the row's length, their token inside the vocabulary."""
    counted = (s["tokens"] >= 0) & (s["tokens"] < s["logits"].shape[2])
    if s["lengths"] is not None:
        steps = torch.arange(T, device=counted.device)
        counted = counted & (steps < s["lengths"][:, None])
    return counted


def _distribution(s, tau):
    """(logits minus their largest, their probabilities, the logarithm of the sum) of every
    step."""
    z = s["logits"].float()
    u = (z - z.amax(2, keepdim=True)) / tau
    e = torch.exp(u)
    total = e.sum(2, keepdim=True)
    return u, e / total, torch.log(total)[..., 0]


def _entropy(u, p, log_total):
    """log sum - sum p u, a logit of -inf left out."""
    return log_total - torch.where(p > 0, p * u, 0.0).sum(2)


def _gradient(s, u, p, log_total, counted, g, c, entropy, tau):
    """sum over steps of g logp + c entropy, differentiated by the logits, in their type."""
    d = -p * g[..., None]
    if c is not None:
        d = d - c[..., None] * torch.where(p > 0, p * (u - log_total[..., None]
                                                       + entropy[..., None]), 0.0)
    at = s["tokens"].clamp(0, p.shape[2] - 1)[..., None]
    d = d.scatter_add(2, at, g[..., None]) / tau
    return torch.where(counted[..., None], d, 0.0).to(s["logits"].dtype)


def _plain_logp(s):
    c = s["case"]
    u, p, log_total = _distribution(s, c["temperature"])
    counted = _counted(s, c["N"], c["T"])
    at = s["tokens"].clamp(0, c["V"] - 1)[..., None]
    logp = torch.where(counted, u.gather(2, at)[..., 0] - log_total, 0.0)
    return u, p, log_total, counted, logp


def _plain_logprob(s, train):
    c = s["case"]
    u, p, log_total, counted, logp = _plain_logp(s)
    entropy = torch.where(counted, _entropy(u, p, log_total), 0.0) if c["entropy"] else None
    out = dict(logp=logp, entropy=entropy)
    if train:
        out["dlogits"] = _gradient(s, u, p, log_total, counted, s["dlogp"], s["dentropy"],
                                   entropy, c["temperature"])
    return out


def _plain_policy(s):
    c = s["case"]
    u, p, log_total, counted, logp = _plain_logp(s)
    A, w = s["advantage"], s["weight"]
    ratio = torch.exp(logp - s["old"])
    near = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    first, second = -A * ratio, -A * near
    loss = torch.maximum(first, second)
    slope = torch.where(first >= second, first, 0.0)  # by the log-probability
    kl = entropy = None
    if s["ref"] is not None:
        d = s["ref"].double() - logp.double()
        kl = (torch.expm1(d) - d).float()
        loss = loss + KL_COEF * kl
        slope = slope - KL_COEF * torch.expm1(d).float()
        kl = torch.where(counted, kl, 0.0)
    if c["entropy"]:
        entropy = _entropy(u, p, log_total)
        loss = loss - ENTROPY_COEF * entropy
        entropy = torch.where(counted, entropy, 0.0)
    grad = _gradient(s, u, p, log_total, counted, w * slope,
                     -ENTROPY_COEF * w if c["entropy"] else None, entropy, c["temperature"])
    return dict(loss=torch.where(counted, loss, 0.0), logp=logp, entropy=entropy, kl=kl,
                dlogits=grad)


def _plain_preference(s):
    c = s["case"]
    N, P = c["N"], c["N"] // 2
    u, p, log_total, counted, logp = _plain_logp(s)
    # Long sums of differences: 64 bits.
    score = torch.where(counted, logp.double() - s["ref"].double(), 0.0).sum(1)
    slope = torch.full((N,), BETA, device=logp.device, dtype=torch.float64)
    if c["by_length"]:
        slope = slope / counted.sum(1).clamp(min=1)
    score = score * slope
    margin = score[:P] - score[P:]
    # -log sigmoid(x) = max(-x, 0) + log(1 + exp(-|x|))
    tail = torch.log1p(torch.exp(-margin.abs()))
    eps = c["smoothing"]
    loss = (1 - eps) * (torch.clamp(-margin, min=0) + tail) + eps * (torch.clamp(margin, min=0)
                                                                     + tail)
    by_margin = (eps - 1 / (1 + torch.exp(margin))) * s["dloss"]
    g = (torch.cat([by_margin, -by_margin]) * slope).float()[:, None].expand(N, c["T"])
    grad = _gradient(s, u, p, log_total, counted, g.contiguous(), None, None, c["temperature"])
    return dict(loss=loss.float(), scores=score.float(), logp=logp, dlogits=grad)


def _plain_distill(s):
    c = s["case"]
    tau = c["temperature"]
    u, p, log_total = _distribution(s, tau)
    index = s["index"]
    inside = (index >= 0) & (index < c["V"])
    at = torch.where(inside, index, 0)
    t = torch.where(inside, s["teacher"].float() / tau, -math.inf)
    top = t.amax(2, keepdim=True)
    some = top > -math.inf
    steps = torch.arange(c["T"], device=t.device)
    if s["lengths"] is not None:
        some = some & (steps < s["lengths"][:, None])[..., None]
    v = t - torch.where(some, top, 0.0)
    e = torch.exp(v)
    total = e.sum(2, keepdim=True)
    q = torch.where(some, e / total, 0.0)
    logp = u.gather(2, at) - log_total[..., None]
    logq = v - torch.log(total)
    loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(2)
    w = torch.where(some, s["weight"][..., None], 0.0) / tau
    d = (w * p).scatter_add(2, at, -w * q)
    return dict(loss=loss, dlogits=torch.where(some, d, 0.0).to(s["logits"].dtype))


# ------------------------------------------------------------------------ the framework


def _own(s):
    import segmented_associative_scan_gb300 as rlca

    c = s["case"]
    op = c["op"]
    rows = dict(lengths=s["lengths"], temperature=c["temperature"])
    if op == "distill":
        loss, dlogits = rlca.distill_topk(s["logits"], s["index"], s["teacher"],
                                          weight=s["weight"], **rows, want_grad=True)
        return dict(loss=loss, dlogits=dlogits)
    if op == "policy":
        loss, logp, entropy, kl, dlogits = rlca.policy_loss(
            s["logits"], s["tokens"], s["old"], s["advantage"], ref_logp=s["ref"],
            weight=s["weight"], **rows, clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
            kl_coef=KL_COEF if c["kl"] else 0.0, entropy_coef=ENTROPY_COEF if c["entropy"] else 0.0,
            want_entropy=c["entropy"], want_grad=True)
        return dict(loss=loss, logp=logp, entropy=entropy, kl=kl, dlogits=dlogits)
    if op == "preference":
        loss, scores, logp, saved = rlca.preference_loss(
            s["logits"], s["tokens"], ref_logp=s["ref"], **rows, beta=BETA,
            smoothing=c["smoothing"], by_length=c["by_length"], want_saved=True)
        dlogits = rlca.preference_loss_backward(s["dloss"], s["logits"], s["tokens"], saved, **rows)
        return dict(loss=loss, scores=scores, logp=logp, dlogits=dlogits)
    train = op == "logprob_train"
    logp, entropy, saved = rlca.token_logprobs(s["logits"], s["tokens"], **rows,
                                               want_entropy=c["entropy"], want_saved=train)
    out = dict(logp=logp, entropy=entropy)
    if train:
        out["dlogits"] = rlca.token_logprobs_backward(
            s["dlogp"], s["logits"], s["tokens"], saved, **rows, entropy=entropy,
            dentropy=s["dentropy"])
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "logprob":
        return _plain_logprob(state, train=False)
    if op == "logprob_train":
        return _plain_logprob(state, train=True)
    return {"policy": _plain_policy, "preference": _plain_preference,
            "distill": _plain_distill}[op](state)


# --------------------------------------------------------------------------------- work


def work(case):
    w, op = _BYTES[case["dtype"]], case["op"]
    M, V = case["N"] * case["T"], case["V"]
    # Logits of steps that do not count need not be read: lengths are uniform in 0..T, prompts in
    # 0..T/2. Gradients are written for all steps.
    share = (0.5 if case["ragged"] else 1.0) * (0.75 if case["prompt"] else 1.0)
    grad = op != "logprob"
    steps = {"logprob": 8 + 4, "logprob_train": 8 + 8, "policy": 8 + 12 + 8, "preference": 8 + 8,
             "distill": 8}[op]
    steps += 4 * (bool(case["entropy"]) * (3 if op == "logprob_train" else 1)
                  + 2 * bool(case.get("kl")))
    if op == "distill":
        steps += case["K"] * (8 + _BYTES[case["teacher"]])
    # One exponential, the largest and the sum; an entropy's product; a gradient's.
    flops = 4 + 2 * bool(case["entropy"]) + (2 + 2 * bool(case["entropy"])) * grad
    return {"bytes": w * M * V * (share + grad) + M * steps, "flops": share * M * V * flops}


# ------------------------------------------------------------------- 64-bit definitions


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits; gradients by automatic
    differentiation of those definitions."""
    s = prepare(case, seed)
    op, N, T, V = case["op"], case["N"], case["T"], case["V"]
    dev = s["logits"].device
    with torch.enable_grad():
        z = s["logits"].double().requires_grad_()
        logs = torch.log_softmax(z / case["temperature"], dim=-1)
        length = torch.full((N,), T, device=dev) if s["lengths"] is None else s["lengths"].long()
        alive = torch.arange(T, device=dev)[None, :] < length[:, None]
        if op == "distill":
            index, teacher = s["index"], s["teacher"].double() / case["temperature"]
            valid = (index >= 0) & (index < V) & alive[..., None]
            q = torch.softmax(teacher.masked_fill(~valid, -1e300), -1) * valid
            got = torch.gather(logs, -1, index.clamp(0, V - 1))
            loss = (torch.xlogy(q, q) - q * got).sum(-1)
            (grad,) = torch.autograd.grad((loss * s["weight"].double()).sum(), z)
            return dict(loss=loss.detach(), dlogits=grad)
        live = alive & (s["tokens"] >= 0) & (s["tokens"] < V)
        zero = torch.zeros((), dtype=torch.float64, device=dev)
        taken = torch.gather(logs, -1, s["tokens"].clamp(0, V - 1)[..., None]).squeeze(-1)
        logp = torch.where(live, taken, zero)
        entropy = None
        if case["entropy"]:
            finite = torch.where(torch.isfinite(logs), logs, zero)
            entropy = torch.where(live, -(torch.exp(logs) * finite).sum(-1), zero)
        out = dict(logp=logp, entropy=entropy)
        total = None
        if op == "logprob_train":
            total = (logp * s["dlogp"].double()).sum()
            if entropy is not None:
                total = total + (entropy * s["dentropy"].double()).sum()
        if op == "policy":
            A = s["advantage"].double()
            ratio = torch.exp(logp - s["old"].double())
            loss = -torch.minimum(ratio * A, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * A)
            out["kl"] = None
            if s["ref"] is not None:
                d = s["ref"].double() - logp
                out["kl"] = torch.where(live, torch.expm1(d) - d, zero)
                loss = loss + KL_COEF * out["kl"]
            if entropy is not None:
                loss = loss - ENTROPY_COEF * entropy
            out["loss"] = torch.where(live, loss, zero)
            total = (out["loss"] * s["weight"].double()).sum()
        if op == "preference":
            sums = torch.where(live, logp - s["ref"].double(), zero).sum(1) * BETA
            if case["by_length"]:
                sums = sums / live.sum(1).clamp(min=1)
            better, worse = sums.chunk(2)
            eps = case["smoothing"]
            loss = (1 - eps) * torch.nn.functional.softplus(worse - better, threshold=700) \
                + eps * torch.nn.functional.softplus(better - worse, threshold=700)
            out.update(loss=loss, scores=sums)
            del out["entropy"]
            total = (loss * s["dloss"].double()).sum()
        if total is not None:
            (out["dlogits"],) = torch.autograd.grad(total, z)
    return {k: None if v is None else v.detach() for k, v in out.items()}
