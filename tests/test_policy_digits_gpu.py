"""How far the losses over a vocabulary and their gradients are off, element by element and over many
rows: every element of a gradient against its own size, however small (a long row's are 1 / V of the
largest), and the errors of rows' sums on average."""
import math

import pytest
import torch

import policy_reference as ref
import segmented_associative_scan_gb300 as rlca
from policy_reference import ROW, U
from sequence_reference import ROUNDING, TINY
from test_policy_gpu import BF16, DISTILL, F32, FP16, INF, SIZES, Rows, _id, cuda, policy_inputs
from test_policy_gpu import run_policy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


def softmax(r):
    """(p, |log p|) of every logit, [N, T, V] in 64 bits; of barred tokens and rows (0, 0)."""
    logs = torch.log_softmax(r.z.double() / r.tau, -1)
    some = logs > -INF
    return torch.where(some, logs.exp(), 0.0), torch.where(some, -logs, 0.0)


def one_hot(r, counted):
    hot = torch.zeros(r.shape, dtype=torch.float64)
    return hot.scatter_(2, torch.where(counted, r.tokens.long(), 0)[..., None],
                        counted[..., None].double())


def close_elements(name, got, want, size, share, logs, tau, sharp=0.9):
    """dz_j = (p_j (g + c (H + log p_j)) + [j = a] g) / tau, up to signs. p_j = e^u / S is off by ROW (S)
    + 4 U (the exponential, 2 ulp) + 2 U |u_j| (its argument), |u_j| <= |log p_j| + 4; what it is
    multiplied by, and g at the taken token, by ROW times `size` (a number for every element: |g| and
    |c| (H + |log p_j|), with what their own errors are multiplied by). `share` is p_j, plus 1 at the taken
    token or a teacher's q_j. So 2 (ROW + 12 U + 2 U |log p_j|) share_j size_j / tau, and the type's rounding.

    `sharp`: the least part of the elements other than 0 whose bound is below half of their size, so
    that a lost one shows."""
    got, want, dtype = got.detach().double().cpu(), want.detach(), got.dtype
    bound = (ROUNDING[dtype] * want.abs() + TINY[dtype]
             + 2 * (ROW + 12 * U + 2 * U * logs) * share * size / tau)
    seen = want != 0
    assert (bound < want.abs() / 2)[seen].double().mean() >= sharp, f"{name}: the bound shows nothing"
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        ratio = torch.where(bad, (got - want).abs() / bound, 0.0).nan_to_num(nan=1e30)
        i = int(ratio.flatten().argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst "
                             f"{float(got.flatten()[i])} for {float(want.flatten()[i])} (at {i}, "
                             f"{float(ratio.flatten()[i]):.3g} of the bound)")


LONG = [c for c in SIZES if c["V"] >= 100]


def unit(r):
    """Weights of this size keep a long row's gradient above what fp16 rounds to 0."""
    return 64.0 if r.dtype is FP16 else 1.0


@pytest.mark.parametrize("kl,entropy_coef", [(True, 0.02), (False, 0.0)])
@pytest.mark.parametrize("cfg", LONG, ids=_id)
def test_every_element_of_the_policy_loss_gradient(cuda_device, cfg, kl, entropy_coef):
    r = Rows(**cfg, seed=41)
    V = r.shape[2]
    v, counted = policy_inputs(r)
    v["weight"] = unit(r) * (0.5 + v["weight"])
    dz = run_policy(r, v, kl, entropy_coef)[4]
    z = r.leaf()
    d = {k: t.double() for k, t in v.items()}
    loss, logp, _, _, _ = ref.policy_loss(
        z, r.tokens, d["old"], d["adv"], d["ref"] if kl else None, r.lengths, lo=0.2, hi=0.3,
        kl_coef=0.05 if kl else 0.0, entropy_coef=entropy_coef, tau=r.tau)
    (loss * d["weight"]).sum().backward()
    logp = logp.detach()
    p, logs = softmax(r)
    ratio = torch.exp(logp - d["old"])
    pull = torch.exp(d["ref"] - logp) if kl else torch.zeros(())
    # The slope by log p and its derivatives: |A| r and the KL term's e^d are multiplied by log p's error.
    size = (d["adv"].abs() * ratio + 0.05 * (1 + pull)) * (1 + logp.abs())
    size = size[..., None] + entropy_coef * (math.log(V) + logs)
    close_elements("dlogits", dz, z.grad, size * d["weight"][..., None], p + one_hot(r, counted), logs,
                   r.tau)


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("cfg", LONG, ids=_id)
def test_every_element_of_the_log_probabilities_gradient(cuda_device, cfg, entropy):
    r = Rows(**cfg, seed=42)
    N, T, V = r.shape
    z = r.leaf()
    logp, h, counted = ref.token_logprobs(z, r.tokens, r.lengths, r.tau)
    _, gh, saved = rlca.token_logprobs(r.cz, r.ctok, **r.kw, want_entropy=entropy, want_saved=True)
    dl = unit(r) * (0.5 + torch.rand(N, T, generator=r.g))
    dh = 0.3 * dl if entropy else None
    ((logp * dl).sum() + ((h * dh).sum() if entropy else 0)).backward()
    dz = rlca.token_logprobs_backward(dl.cuda(), r.cz, r.ctok, saved, **r.kw, entropy=gh,
                                      dentropy=cuda(dh))
    p, logs = softmax(r)
    size = dl.double()[..., None]
    if entropy:
        size = size + dh.double()[..., None] * (math.log(V) + logs)
    close_elements("dlogits", dz, z.grad, size, p + one_hot(r, counted), logs, r.tau)


@pytest.mark.parametrize("cfg", [c for c in LONG if c["N"] % 2 == 0 and c["N"] < 400], ids=_id)
def test_every_element_of_the_preference_loss_gradient(cuda_device, cfg):
    r = Rows(**cfg, seed=43)
    N, T, V = r.shape
    base, _, _ = ref.token_logprobs(r.z.double(), r.tokens, r.lengths, r.tau)
    reference = (base + 0.3 * r.rn(N, T)).float()
    z = r.leaf()
    beta = 0.2
    loss, _, logp, counted = ref.preference_loss(z, r.tokens, reference.double(), r.lengths, beta, 0.1,
                                                 False, r.tau)
    dloss = unit(r) * (0.5 + torch.rand(N // 2, generator=r.g))
    (loss * dloss).sum().backward()
    _, _, _, saved = rlca.preference_loss(r.cz, r.ctok, ref_logp=reference.cuda(), **r.kw, beta=beta,
                                          smoothing=0.1, want_saved=True)
    dz = rlca.preference_loss_backward(dloss.cuda(), r.cz, r.ctok, saved, **r.kw)
    # A slope (below 1) moves by at most a quarter of the scores' error.
    err = beta * (counted * (1 + logp.detach().abs())).sum(1)
    size = beta * (dloss.double() * (1 + err[:N // 2] + err[N // 2:])).repeat(2)
    p, logs = softmax(r)
    close_elements("dlogits", dz, z.grad, size[:, None, None], p + one_hot(r, counted), logs, r.tau)


@pytest.mark.parametrize("cfg", [c for c in DISTILL if c["V"] >= 64], ids=_id)
def test_every_element_of_the_distillation_gradient(cuda_device, cfg):
    cfg = dict(cfg)
    K = cfg.pop("K")
    r = Rows(**cfg, seed=44)
    N, T, V = r.shape
    index = torch.rand(N, T, V, generator=r.g).argsort(-1)[..., :K]
    if cfg.get("masked"):
        index = torch.where(r.z.gather(2, index).isinf(), -1, index)
    teacher = 2 * r.rn(N, T, K)
    weight = unit(r) * (0.5 + torch.rand(N, T, generator=r.g))
    z = r.leaf()
    loss, counted = ref.distill_topk(z, index, teacher.double(), r.lengths, r.tau)
    (loss * weight).sum().backward()
    _, dz = rlca.distill_topk(r.cz, index.cuda(), teacher.cuda(), weight=weight.cuda(), **r.kw,
                              want_grad=True)
    good = (index >= 0) & counted[..., None]
    q = torch.softmax(torch.where(good, teacher.double() / r.tau, -INF), -1).nan_to_num(nan=0.0)
    p, logs = softmax(r)
    share = p.scatter_add(2, torch.where(good, index, 0), torch.where(good, q, 0.0))
    close_elements("dlogits", dz, z.grad, weight.double()[..., None], share, logs, r.tau)


# ------------------------------------------------------------------------- errors on average


# Rows of a lane's own, by tiles, in registers, parked, and parked in part.
MANY = [(600, 18), (600, 24), (600, 101), (600, 512), (190, 2051), (640, 1101), (320, 5003), (64, 70001)]


@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("N,V", MANY)
def test_sums_of_rows_on_average(cuda_device, N, V, dtype, entropy, tau):
    """log S from the saved sums over many rows. The exponentials are corrected for what they are low by
    on average, 5e-8 below an exponent of -1 and down to 2e-8 above, and their scale has twice its digits:
    3e-8 is left for the mean. Each row is off by the rounding of S (2^-24) and a share of its
    exponentials' 2 ulp, 1.5e-7 rms.

    A parked row's logits may lie above what its sums are relative to. There 2^v is high by 3.3e-8
    (measured, v from 0 to 8), and corrected as if it were low: 8.3e-8 if all of S lay there. And a warp's
    sums are brought to the largest reference by e^-d, d up to 5 in these rows: three roundings of d, U d
    or 3e-7 rms together, 3.4e-7 with the above. As few as 64 rows leave their deviation besides, four
    times that / sqrt(N)."""
    r = Rows(dtype, N, 1, V, tau=tau, seed=45)
    _, _, saved = rlca.token_logprobs(r.cz, r.ctok, temperature=tau, want_entropy=entropy,
                                      want_saved=True)
    m, s = saved.double().cpu().unbind(-1)
    # The calls take the temperature as a float: 0.7 is 1.7e-8 of itself lower, and log S by 1e-7.
    tau = float(torch.tensor(tau, dtype=F32))
    z = r.z.double()
    err = m / tau + torch.log(s) - torch.logsumexp(z / tau, -1)
    above = bool((z.amax(-1) > m).any())
    rms = 3.4e-7 if above else 1.5e-7
    mean = 8.3e-8 + 4 * rms / math.sqrt(N) if above else 3e-8
    assert abs(err.mean()) <= mean and err.square().mean().sqrt() <= rms


@pytest.mark.parametrize("N,V", MANY)
def test_ratios_of_one(cuda_device, N, V):
    """old_logp as token_logprobs gave it: the ratio is off by the rounding of that value, U |log p|, by as
    much again where the two calls' S round to either side, and by the 2 ulp of an exponential."""
    r = Rows(F32, N, 1, V, seed=46)
    logp, _, _ = rlca.token_logprobs(r.cz, r.ctok)
    adv = 0.5 + torch.rand(N, 1, generator=r.g).cuda()
    loss, _, _, kl, _ = rlca.policy_loss(r.cz, r.ctok, logp, adv, ref_logp=logp, want_grad=True)
    d = U * (2 * logp.abs() + 16)
    assert ((loss + adv).abs() <= d * adv).all()
    assert ((kl >= 0) & (kl <= d * d)).all()


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("T,V", [(700, 40), (700, 501), (300, 1101)])
def test_scores_of_long_answers(cuda_device, T, V, dtype):
    """A score is a sum of many log ratios: what S is off by on average (3e-8) adds up, the roundings of
    log p (U |log p|) as their square root does, here with four deviations' room, over sixteen rows."""
    r = Rows(dtype, 16, T, V, seed=47)
    base, _, _ = ref.token_logprobs(r.z.double(), r.tokens)
    reference = (base + 0.01 * r.rn(16, T)).float()
    beta = 0.5
    _, want, logp, _ = ref.preference_loss(r.z.double(), r.tokens, reference.double(), beta=beta)
    _, scores, _, _ = rlca.preference_loss(r.cz, r.ctok, ref_logp=reference.cuda(), beta=beta)
    err = (scores.double().cpu() - want).abs()
    bound = beta * (3e-8 * T + 4 * math.sqrt(T) * U * (1 + logp.abs().amax(1))) + U * want.abs()
    assert (err <= bound).all()
