"""Losses over a vocabulary on the GPU against their 64-bit definitions: token log-probabilities,
the clipped policy loss, the preference loss and the distillation, with their gradients."""
import math

import pytest
import torch

import policy_reference as ref
import segmented_associative_scan_gb300 as rlca
from policy_reference import U, close

pytestmark = pytest.mark.gpu

F32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


def cuda(v):
    return v.cuda() if torch.is_tensor(v) else v


class Rows:
    """Logits and tokens on the CPU in their type; `c` the same on the GPU, in the layout asked
    for: `shifted` slices one step off wider buffers, `wide` pads the vocabulary by some columns,
    `major` lays steps outside of rows."""

    def __init__(self, dtype, N, T, V, tau=1.0, ragged=False, prompt=False, masked=False,
                 layout="plain", int32=False, seed=0):
        g = torch.Generator().manual_seed(seed + 131 * V + T)
        self.g, self.shape, self.dtype, self.tau = g, (N, T, V), dtype, tau
        z = self.rn(N, T, V) * 2
        tokens = torch.randint(0, V, (N, T), generator=g)
        # Most taken tokens are likely ones.
        z.scatter_add_(2, tokens[..., None],
                       (math.log(V) * (torch.rand(N, T, generator=g) < 0.8))[..., None].float())
        if masked:
            block = torch.rand(N, T, V, generator=g) < 0.3
            block.scatter_(2, tokens[..., None], False)
            z[block] = -INF
        if prompt:
            tokens[torch.rand(N, T, generator=g) < 0.3] = -100
        self.lengths = None
        if ragged:
            self.lengths = torch.randint(0, T + 1, (N,), generator=g, dtype=torch.int32)
            self.lengths[0] = T
            if N > 1:
                self.lengths[1] = 0
        self.z = z.to(dtype)
        self.tokens = tokens.int() if int32 else tokens
        self.place(layout)

    def rn(self, *s):
        return torch.randn(*s, generator=self.g)

    def place(self, layout):
        N, T, V = self.shape
        z, tok = self.z.cuda(), self.tokens.cuda()
        if layout == "shifted":
            buf = torch.full((N, T + 1, V), NAN, dtype=self.dtype, device="cuda")
            buf[:, :T] = z
            z = buf[:, :T]
            wide = torch.full((N, T + 1), -5, dtype=tok.dtype, device="cuda")
            wide[:, 1:] = tok
            tok = wide[:, 1:]
        elif layout == "wide":
            buf = torch.full((N, T, V + 5), NAN, dtype=self.dtype, device="cuda")
            buf[..., 3:3 + V] = z
            z = buf[..., 3:3 + V]
        elif layout == "major":
            buf = torch.empty(T, N, V, dtype=self.dtype, device="cuda")
            buf.copy_(z.transpose(0, 1))
            z = buf.transpose(0, 1)
        self.cz, self.ctok = z, tok
        self.kw = dict(lengths=cuda(self.lengths), temperature=self.tau)

    def leaf(self):
        return self.z.double().requires_grad_()


def grad_scale(g, tau):
    """The size of a row's gradient before anything cancels."""
    return (g.abs() / tau)[..., None]


def _id(c):
    return "-".join(str(v).replace("torch.", "") for v in c.values())


# Every way a row is read: a few lanes, a warp, CTAs of a cluster, streamed; sizes at and around
# the borders, odd ones, one token, one step.
SIZES = [
    dict(dtype=F32, N=3, T=5, V=1),
    dict(dtype=BF16, N=5, T=7, V=2, masked=True),
    dict(dtype=F32, N=9, T=33, V=3, prompt=True),
    dict(dtype=F32, N=40, T=17, V=18, masked=True, ragged=True),
    dict(dtype=FP16, N=4, T=9, V=31, tau=0.7, layout="shifted"),
    dict(dtype=BF16, N=4, T=9, V=32),
    dict(dtype=F32, N=4, T=9, V=33, layout="wide"),
    dict(dtype=BF16, N=3, T=6, V=64, int32=True, ragged=True),
    dict(dtype=F32, N=2, T=5, V=127, tau=2.0),
    dict(dtype=F32, N=2, T=5, V=128, layout="major"),
    dict(dtype=FP16, N=2, T=5, V=129, masked=True),
    dict(dtype=BF16, N=3, T=7, V=250, layout="wide"),
    dict(dtype=F32, N=3, T=7, V=512, prompt=True, ragged=True),
    dict(dtype=BF16, N=2, T=5, V=1000, layout="shifted"),
    dict(dtype=F32, N=2, T=5, V=1023, layout="shifted"),
    dict(dtype=F32, N=2, T=5, V=1024),
    dict(dtype=F32, N=2, T=3, V=1025, layout="shifted", masked=True),
    dict(dtype=FP16, N=2, T=5, V=2047, layout="shifted"),
    dict(dtype=BF16, N=2, T=5, V=2048),
    dict(dtype=BF16, N=1, T=3, V=2049, layout="wide", tau=0.5),
    dict(dtype=F32, N=2, T=4, V=5003, ragged=True, layout="shifted"),
    dict(dtype=BF16, N=3, T=5, V=8192, prompt=True, layout="major"),
    dict(dtype=FP16, N=2, T=5, V=16383, layout="shifted", masked=True),
    dict(dtype=F32, N=1, T=2, V=16384),
    dict(dtype=BF16, N=2, T=3, V=33001, layout="shifted"),
    dict(dtype=F32, N=1, T=3, V=65537, masked=True),
    dict(dtype=BF16, N=1, T=3, V=131071, layout="shifted"),
    dict(dtype=F32, N=1, T=2, V=131072),
    dict(dtype=BF16, N=1, T=2, V=262144),
    dict(dtype=BF16, N=1, T=2, V=300007, layout="wide"),
    dict(dtype=F32, N=1, T=2, V=270001, layout="shifted"),
    dict(dtype=BF16, N=700, T=1, V=4096),
    dict(dtype=BF16, N=333, T=3, V=4099, ragged=True, layout="shifted"),
    dict(dtype=F32, N=1, T=1, V=50000),
    # Rows longer than a CTA parks, and enough of them for CTAs of their own.
    dict(dtype=FP16, N=9, T=4, V=70001, ragged=True, layout="shifted"),
    dict(dtype=F32, N=23, T=1, V=40001, layout="wide", masked=True),
    dict(dtype=BF16, N=22, T=1, V=65544),
    dict(dtype=BF16, N=5, T=9, V=1021, ragged=True, layout="shifted"),
    dict(dtype=F32, N=4, T=9, V=700, prompt=True, layout="wide"),
    dict(dtype=FP16, N=7, T=6, V=1608),
]

# Rows enough for CTAs that park them in shared memory (sixty, and six hundred short ones), whole and
# in part, several to a CTA.
PARKED = [
    dict(dtype=BF16, N=68, T=10, V=1032, layout="wide"),
    dict(dtype=FP16, N=40, T=17, V=1101, ragged=True, layout="shifted"),
    dict(dtype=F32, N=34, T=7, V=2049, prompt=True, masked=True),
    dict(dtype=BF16, N=3, T=54, V=8192, tau=0.7, layout="major"),
    dict(dtype=FP16, N=4, T=18, V=16387, masked=True, layout="shifted"),
    dict(dtype=BF16, N=2, T=32, V=33000, ragged=True, prompt=True),
    dict(dtype=F32, N=13, T=5, V=40001, layout="wide"),
    dict(dtype=BF16, N=32, T=2, V=70001, ragged=True, layout="shifted"),
    dict(dtype=BF16, N=63, T=1, V=65544),
    dict(dtype=F32, N=400, T=2, V=1500, layout="shifted", prompt=True),
]
SIZES += PARKED


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("cfg", SIZES, ids=_id)
def test_token_logprobs(cuda_device, cfg, entropy):
    r = Rows(**cfg)
    N, T, V = r.shape
    z = r.leaf()
    logp, h, counted = ref.token_logprobs(z, r.tokens, r.lengths, r.tau)
    got, gh, saved = rlca.token_logprobs(r.cz, r.ctok, **r.kw, want_entropy=entropy,
                                         want_saved=True)
    logv = 1 + math.log(V)
    close("logp", got, logp, 1 + logp.abs())
    if entropy:
        close("entropy", gh, h, logv)
    dl, dh = r.rn(N, T), 0.3 * r.rn(N, T) if entropy else None
    loss = (logp * dl).sum()
    if entropy:
        loss = loss + (h * dh).sum()
    loss.backward()
    dz = rlca.token_logprobs_backward(dl.cuda(), r.cz, r.ctok, saved, **r.kw, entropy=gh,
                                      dentropy=cuda(dh))
    size = dl.abs() + (dh.abs() * logv if entropy else 0)
    close("dlogits", dz, z.grad, grad_scale(size, r.tau))
    assert dz.is_contiguous() and not dz[~counted.cuda()].any()


POLICY = dict(clip_low=0.2, clip_high=0.3)


def policy_inputs(r, moved=0.25):
    """old, advantages, ref and weights of a policy that has moved; no ratio within 2e-3 of a border,
    where rounding decides on its side (a ratio is good to ROW, 1e-5, here)."""
    N, T, _ = r.shape
    logp, _, counted = ref.token_logprobs(r.z.double(), r.tokens, r.lengths, r.tau)
    d = moved * r.rn(N, T).double()
    for border in (math.log(1 - POLICY["clip_low"]), math.log(1 + POLICY["clip_high"])):
        d = torch.where((d - border).abs() < 2e-3, d + 5e-3, d)
    old = (logp - d).float()
    return dict(old=old, adv=r.rn(N, T), ref=(logp + 0.4 * r.rn(N, T)).float(),
                weight=torch.rand(N, T, generator=r.g)), counted


def run_policy(r, v, kl, entropy_coef, **kw):
    c = {k: t.cuda() for k, t in v.items()}
    return rlca.policy_loss(r.cz, r.ctok, c["old"], c["adv"], ref_logp=c["ref"] if kl else None,
                            weight=c["weight"], **r.kw, **POLICY, kl_coef=0.05 if kl else 0.0,
                            entropy_coef=entropy_coef, want_entropy=bool(entropy_coef),
                            want_grad=True, **kw)


def check_policy(r, v, kl, entropy_coef, got):
    N, T, V = r.shape
    z = r.leaf()
    d = {k: t.double() for k, t in v.items()}
    loss, logp, h, rkl, _ = ref.policy_loss(
        z, r.tokens, d["old"], d["adv"], d["ref"] if kl else None, r.lengths, lo=0.2, hi=0.3,
        kl_coef=0.05 if kl else 0.0, entropy_coef=entropy_coef, tau=r.tau)
    (loss * d["weight"]).sum().backward()
    gl, glogp, gh, gkl, dz = got
    logv = 1 + math.log(V)
    ratio = torch.exp(logp.detach() - d["old"]).clamp(max=10)
    pull = torch.exp(d["ref"] - logp.detach()).clamp(max=100) if kl else torch.zeros(())
    # What log p's error is multiplied by, and the roundings of the sum itself.
    size = d["adv"].abs() * ratio + 0.05 * (1 + pull) + entropy_coef * logv
    # log p itself is rounded: 2 U |log p| in a difference.
    size = size * (1 + logp.detach().abs())
    close("logp", glogp, logp, 1 + logp.abs())
    close("loss", gl, loss, size)
    if kl:
        close("kl", gkl, rkl, (1 + pull) * (1 + logp.detach().abs()))
    if entropy_coef:
        close("entropy", gh, h, logv)
    close("dlogits", dz, z.grad, grad_scale(size * d["weight"], r.tau))


@pytest.mark.parametrize("kl,entropy_coef", [(True, 0.02), (False, 0.0), (True, 0.0),
                                             (False, 0.02)])
@pytest.mark.parametrize("cfg", SIZES, ids=_id)
def test_policy_loss(cuda_device, cfg, kl, entropy_coef):
    r = Rows(**cfg, seed=1)
    v, counted = policy_inputs(r)
    got = run_policy(r, v, kl, entropy_coef)
    check_policy(r, v, kl, entropy_coef, got)
    assert (got[3] is None) == (not kl)
    assert not got[4][~counted.cuda()].any() and not got[0][~counted.cuda()].any()


PREFERENCE = [c for c in SIZES if c["N"] % 2 == 0 and c["N"] < 400] + [
    dict(dtype=BF16, N=2, T=700, V=40, prompt=True),
    dict(dtype=F32, N=6, T=77, V=501, prompt=True, ragged=True, layout="shifted"),
]


@pytest.mark.parametrize("smoothing,by_length,with_ref", [(0.0, False, True), (0.1, True, True),
                                                          (1.0, False, False)])
@pytest.mark.parametrize("cfg", PREFERENCE, ids=_id)
def test_preference_loss(cuda_device, cfg, smoothing, by_length, with_ref):
    r = Rows(**cfg, seed=2)
    N, T, V = r.shape
    base, _, _ = ref.token_logprobs(r.z.double(), r.tokens, r.lengths, r.tau)
    reference = (base + 0.3 * r.rn(N, T)).float() if with_ref else None
    z = r.leaf()
    beta = 0.2
    loss, scores, logp, counted = ref.preference_loss(
        z, r.tokens, None if reference is None else reference.double(), r.lengths, beta, smoothing,
        by_length, r.tau)
    dloss = r.rn(N // 2)
    (loss * dloss).sum().backward()
    gl, gs, glogp, saved = rlca.preference_loss(
        r.cz, r.ctok, ref_logp=cuda(reference), **r.kw, beta=beta, smoothing=smoothing,
        by_length=by_length, want_saved=True)
    count = counted.sum(1).double()
    by_logp = beta / count.clamp(min=1) if by_length else torch.full((N,), beta).double()
    # Every log p of a row off by its bound, the same way.
    err = by_logp * (counted * (1 + logp.detach().abs())).sum(1)
    pair = err[:N // 2] + err[N // 2:]
    close("logp", glogp, logp, 1 + logp.abs())
    close("scores", gs, scores, err)
    close("loss", gl, loss, pair)
    dz = rlca.preference_loss_backward(dloss.cuda(), r.cz, r.ctok, saved, **r.kw)
    # The slope moves by at most a quarter of the score's error.
    size = (dloss.abs() * (1 + pair)).repeat(2) * by_logp
    close("dlogits", dz, z.grad, grad_scale(size[:, None].expand(N, T), r.tau))


DISTILL = [
    dict(dtype=F32, N=2, T=3, V=1, K=1),
    dict(dtype=F32, N=5, T=7, V=18, K=18, masked=True),
    dict(dtype=BF16, N=3, T=9, V=64, K=5, ragged=True),
    dict(dtype=FP16, N=2, T=5, V=257, K=256, layout="shifted"),
    dict(dtype=F32, N=2, T=5, V=1024, K=33, tau=2.0, layout="wide"),
    dict(dtype=BF16, N=2, T=5, V=2051, K=20, layout="shifted", ragged=True),
    dict(dtype=F32, N=2, T=4, V=5003, K=64, tau=0.5),
    dict(dtype=FP16, N=2, T=5, V=16383, K=100, layout="shifted"),
    dict(dtype=BF16, N=1, T=5, V=33000, K=256),
    dict(dtype=BF16, N=1, T=2, V=131071, K=64, layout="shifted"),
    dict(dtype=F32, N=1, T=2, V=270001, K=64),
    dict(dtype=BF16, N=260, T=3, V=4099, K=8, layout="shifted"),
    dict(dtype=F32, N=7, T=9, V=100, K=100, masked=True),
    dict(dtype=FP16, N=6, T=7, V=2051, K=200, ragged=True, layout="shifted"),
    dict(dtype=BF16, N=4, T=11, V=33000, K=64, tau=1.5),
    dict(dtype=F32, N=13, T=5, V=40001, K=33, layout="wide"),
    dict(dtype=BF16, N=32, T=2, V=70001, K=17, ragged=True, layout="shifted"),
]


@pytest.mark.parametrize("fp32_teacher,int32", [(True, False), (False, True)])
@pytest.mark.parametrize("cfg", DISTILL, ids=_id)
def test_distill_topk(cuda_device, cfg, fp32_teacher, int32):
    cfg = dict(cfg)
    K = cfg.pop("K")
    r = Rows(**cfg, seed=3)
    N, T, V = r.shape
    index = torch.rand(N, T, V, generator=r.g).argsort(-1)[..., :K]
    if cfg.get("masked"):  # a teacher that gives weight to a token the student may not take: see below
        index = torch.where(r.z.gather(2, index).isinf(), -1, index)
    if K > 3:
        index[..., 1] = index[..., 0]             # a token given twice
        index[..., 2] = -1                        # left out
        index[torch.rand(N, T, K, generator=r.g) < 0.05] = V
    teacher = (2 * r.rn(N, T, K)).to(F32 if fp32_teacher else r.dtype)
    teacher[torch.rand(N, T, K, generator=r.g) < 0.05] = -INF
    weight = torch.rand(N, T, generator=r.g)
    z = r.leaf()
    loss, counted = ref.distill_topk(z, index, teacher.double(), r.lengths, r.tau)
    (loss * weight).sum().backward()
    gl, dz = rlca.distill_topk(r.cz, (index.int() if int32 else index).cuda(), teacher.cuda(),
                               weight=weight.cuda(), **r.kw, want_grad=True)
    # log p of the least likely entry enters with its own rounding.
    size = 2 + (z.detach().abs().nan_to_num(posinf=0, neginf=0).amax(-1) / r.tau) * 2
    close("loss", gl, loss, size)
    close("dlogits", dz, z.grad, grad_scale(weight.double(), r.tau))
    assert not dz[~counted.cuda()].any()


# ------------------------------------------------------------------------ masks and bad values


WAYS = [18, 100, 700, 1500, 4500, 40000, 300000]


@pytest.mark.parametrize("N", [1, 8, 80])
@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("V", WAYS)
def test_rows_without_a_distribution(cuda_device, dtype, V, N):
    """A row of -inf does not count; one of the type's lowest value is uniform; a NaN or +inf in a
    row makes that row NaN and no other; steps that do not count may hold anything."""
    if V == 300000 and dtype is FP16:
        V = 300008
    if N * V > 4_000_000:
        pytest.skip("long rows are parked from fewer on")
    T = 9
    r = Rows(dtype, N, T, V, seed=5)
    z = r.z
    z[0, 1] = -INF
    z[0, 2] = torch.finfo(dtype).min
    z[0, 3, V // 2] = NAN
    z[0, 4, V - 1] = INF
    z[0, 5] = torch.where(torch.arange(V) == 2, 1.0, -INF).to(dtype)
    z[0, 6] = NAN
    z[0, 7, ::2] = torch.finfo(dtype).min
    r.tokens[0, 2], r.tokens[0, 4], r.tokens[0, 5] = 0, 0, 2
    r.tokens[0, 6] = V
    r.tokens[0, 7] = 1
    r.place("plain")
    v, _ = policy_inputs(r)
    for k in ("old", "ref", "adv", "weight"):
        v[k] = v[k].nan_to_num(nan=0.1, posinf=0.1, neginf=0.1)
        v[k][0, 6] = NAN
        v[k][0, 1] = 1.0
    v["adv"][0, 2] = 1.0
    got = run_policy(r, v, True, 0.02)
    loss, logp, h, kl, dz = (t[0].cpu() for t in got)
    for row in (1, 6):
        assert loss[row] == 0 and logp[row] == 0 and h[row] == 0 and kl[row] == 0
        assert not dz[row].any()
    for row in (3, 4):
        assert loss[row].isnan() and logp[row].isnan() and h[row].isnan() and kl[row].isnan()
        assert dz[row].isnan().all()
    close("uniform logp", logp[2], torch.tensor(-math.log(V)).double(), 1 + math.log(V))
    close("uniform entropy", h[2], torch.tensor(math.log(V)).double(), 1 + math.log(V))
    assert logp[5] == 0 and h[5] == 0 and not dz[5].any()
    keep = [0, 2, 5, 7, 8]
    sub = Rows(dtype, 1, T, V, seed=5)
    sub.z, sub.tokens, sub.shape = z[:1, keep], r.tokens[:1, keep], (1, len(keep), V)
    check_policy(sub, {k: t[:1, keep] for k, t in v.items()}, True, 0.02,
                 [t[:1, keep] for t in got])
    for t in got:
        assert t[1:].isfinite().all()
    # The same rows through the log-probabilities and their gradient.
    glogp, gh, saved = rlca.token_logprobs(r.cz, r.ctok, want_entropy=True, want_saved=True)
    assert glogp[0, 1] == 0 and gh[0, 6] == 0 and glogp[0, 3].isnan() and gh[0, 4].isnan()
    one = torch.ones(N, T, device="cuda")
    one[0, 6] = NAN
    dz = rlca.token_logprobs_backward(one, r.cz, r.ctok, saved, entropy=gh, dentropy=one)[0]
    assert not dz[1].any() and not dz[6].any() and dz[3].isnan().all() and dz[4].isnan().all()
    assert dz[[0, 2, 5, 7, 8]].isfinite().all()


@pytest.mark.parametrize("N", [1, 12, 120])
@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("V", WAYS)
def test_logits_of_any_size(cuda_device, dtype, V, N):
    """Rows near the ends of the type: tokens that are not allowed among ones at its lowest value,
    large logits a step of the type apart, at either end."""
    if V == 300000 and dtype is FP16:
        V = 300008
    if N * V > 4_000_000:
        pytest.skip("long rows are parked from fewer on")
    r = Rows(dtype, N, 6, V, seed=19)
    f = torch.finfo(dtype)
    z = r.z
    z[0, 0, ::2] = f.min
    z[0, 0, 1::2] = -INF
    big = 60000.0 if dtype is FP16 else 1e30
    z[0, 1], z[0, 2] = (big + 0 * z[0, 1].float()).to(dtype), (-big + 0 * z[0, 2].float()).to(dtype)
    z[0, 1, 3:] = (z[0, 1, 3:].float() * (1 - 4 * f.eps)).to(dtype)
    z[0, 2, :3] = (z[0, 2, :3].float() * (1 - 4 * f.eps)).to(dtype)
    z[0, 3] = (1e5 if dtype is not FP16 else 5e4) * (1 if V % 4 else -1)
    z[0, 4, 1:] = f.min
    z[0, 5] = (z[0, 5].float() * 1000).to(dtype)
    r.tokens[0] = torch.tensor([0, 1, 2, 0, 0, int(z[0, 5].float().argmax())])
    r.place("plain")
    v, _ = policy_inputs(r)
    # A row thousands wide: exponents of thousands, rounded to 2^-24 of themselves, decide nothing.
    check_policy(r, v, True, 0.02, run_policy(r, v, True, 0.02))


@pytest.mark.parametrize("N", [2, 21, 210])
@pytest.mark.parametrize("V", WAYS)
def test_a_weight_of_zero_is_a_gradient_of_zero(cuda_device, V, N):
    if N * V > 10_000_000:
        pytest.skip("long rows are parked from fewer on")
    r = Rows(BF16, N, 3, V, seed=6)
    r.z[0, 1, 0] = NAN
    r.place("plain")
    v, _ = policy_inputs(r)
    v = {k: t.nan_to_num(nan=0.0) for k, t in v.items()}
    v["weight"][0, 1] = 0.0
    loss, *_, dz = run_policy(r, v, True, 0.02)
    assert loss[0, 1].isnan() and not dz[0, 1].any() and dz[0, 0].any()
    index = torch.zeros(N, 3, 1, dtype=torch.int64, device="cuda")
    loss, dz = rlca.distill_topk(r.cz, index, torch.zeros(N, 3, 1, device="cuda"),
                                 weight=v["weight"].cuda(), want_grad=True)
    assert loss[0, 1].isnan() and not dz[0, 1].any() and dz[0, 0].any()


def test_a_taken_token_that_is_not_allowed(cuda_device):
    """log p = -inf: the ratio is 0, a KL term is inf, the entropy as without that token."""
    r = Rows(F32, 1, 2, 40, seed=7)
    r.z[0, 0, int(r.tokens[0, 0])] = -INF
    r.place("plain")
    z = torch.zeros(1, 2, device="cuda")
    adv = torch.full((1, 2), 2.0, device="cuda")
    loss, logp, h, kl, dz = rlca.policy_loss(r.cz, r.ctok, z - 1, adv, want_entropy=True,
                                             want_grad=True)
    assert logp[0, 0] == -INF and loss[0, 0] == 0 and kl is None and not dz[0, 0].any()
    assert h[0, 0].isfinite()
    loss, _, _, kl, dz = rlca.policy_loss(r.cz, r.ctok, z - 1, -adv, ref_logp=z - 1, want_grad=True)
    assert kl[0, 0] == INF and abs(loss[0, 0].item() - 1.6) <= 4 * U and not dz[0, 0].any()
    loss, _, _, _, _ = rlca.policy_loss(r.cz, r.ctok, z - 1, adv, ref_logp=z - 1, kl_coef=0.1)
    assert loss[0, 0] == INF and loss[0, 1].isfinite()


def test_distillation_from_odd_teachers(cuda_device):
    """No entries; none that is left; a token that the student may not take (an infinite loss); one
    entry; the same one K times."""
    V, K = 50, 7
    r = Rows(F32, 1, 6, V, seed=8)
    index = torch.randint(0, V, (1, 6, K), generator=r.g)
    teacher = r.rn(1, 6, K)
    index[0, 1] = -1
    teacher[0, 2] = -INF
    index[0, 3, 1:] = V + 3
    index[0, 4] = index[0, 4, 0]
    r.z[0, 5, index[0, 5, 2]] = -INF
    r.place("plain")
    loss, dz = rlca.distill_topk(r.cz, index.cuda(), teacher.cuda(), want_grad=True)
    for row in (1, 2):
        assert loss[0, row] == 0 and not dz[0, row].any()
    assert loss[0, 5] == INF and dz[0, 5].isfinite().all()
    z = r.leaf()
    want, _ = ref.distill_topk(z, index, teacher.double())
    want[0, :5].sum().backward()
    close("loss", loss[:, :5], want[:, :5], 20.0)
    close("dlogits", dz[:, :5], z.grad[:, :5], 1.0)
    loss, dz = rlca.distill_topk(r.cz, index[..., :0].cuda(), teacher[..., :0].cuda(),
                                 want_grad=True)
    assert not loss.any() and not dz.any()


# ------------------------------------------------------------------------------- layouts


def test_no_rows_no_steps(cuda_device):
    for N, T in ((0, 3), (4, 0)):
        z = torch.empty(N, T, 10, device="cuda")
        tok = torch.empty(N, T, dtype=torch.int64, device="cuda")
        s = torch.empty(N, T, device="cuda")
        assert rlca.token_logprobs(z, tok)[0].shape == (N, T)
        assert rlca.policy_loss(z, tok, s, s, want_grad=True)[4].shape == z.shape
        k = torch.empty(N, T, 2, device="cuda")
        assert rlca.distill_topk(z, k.long(), k, want_grad=True)[0].shape == (N, T)
        loss, scores, _, saved = rlca.preference_loss(z, tok, want_saved=True)
        assert loss.shape == (N // 2,) and not scores.any()
        assert torch.allclose(loss, torch.full_like(loss, math.log(2.0)))
        assert rlca.preference_loss_backward(None, z, tok, saved).shape == z.shape


@pytest.mark.parametrize("V,N", [(18, 6), (700, 6), (5000, 6), (40000, 6), (3000, 400)])
def test_one_step_of_rows(cuda_device, V, N):
    """[N, V] is the one step of [N, 1, V], strided rows and tokens too."""
    r = Rows(BF16, N, 3, V, seed=9)
    whole, wh, _ = rlca.token_logprobs(r.cz, r.ctok, want_entropy=True)
    one, oh, _ = rlca.token_logprobs(r.cz[:, 1], r.ctok[:, 1], want_entropy=True)
    close("logp", one, whole[:, 1].double().cpu(), 1 + whole[:, 1].abs().cpu())
    close("entropy", oh, wh[:, 1].double().cpu(), 1 + math.log(V))
    v, _ = policy_inputs(r)
    full = run_policy(r, v, True, 0.02)
    r.cz, r.ctok = r.cz[:, 1], r.ctok[:, 1]
    step = run_policy(r, {k: t[:, 1] for k, t in v.items()}, True, 0.02)
    for a, b in zip(full, step):
        assert b.shape == a[:, 1].shape
        rounding = 2 * ref.ROUNDING[a.dtype]
        assert ((a[:, 1] - b).abs() <= rounding * b.abs() + 1e-4).all()


@pytest.mark.parametrize("V", [18, 500, 4096])
def test_broadcast_rows_and_values(cuda_device, V):
    """One row of logits for every environment (a stride of 0), one weight and one reference for
    all rows."""
    r = Rows(F32, 1, 5, V, seed=10)
    N = 4
    logits = r.cz.expand(N, 5, V)
    tokens = torch.randint(0, V, (N, 5), generator=r.g)
    old, adv, w = -3 + 0.1 * r.rn(N, 5), r.rn(N, 5), torch.rand(1, 5, generator=r.g)
    reference = -3 + 0.1 * r.rn(1, 5)
    args = lambda f: (f(logits), tokens.cuda(), old.cuda(), f(adv.cuda()))
    more = lambda f: dict(ref_logp=f(reference.cuda().expand(N, 5)),
                          weight=f(w.cuda().expand(N, 5)), kl_coef=0.1, entropy_coef=0.1,
                          want_entropy=True, want_grad=True)
    same, copy = (lambda t: t), (lambda t: t.contiguous())
    # A row's packs begin where its memory does, so a copy's sums are taken in another order: each
    # form is within ROW of the definition, the two within twice that. Sizes: |A| r, the KL term and
    # its slope, H; weights of at most 1.
    size = 1 + old.abs() + adv.abs() * 3 + 0.1 * (1 + 20) + 0.1 * (1 + math.log(V))
    for a, b in zip(rlca.policy_loss(*args(same), **more(same)),
                    rlca.policy_loss(*args(copy), **more(copy))):
        s = (size * 8).cuda()  # |log p| <= 8 + log V here, and r <= 3
        bound = 2 * (ref.ROW * (s[..., None] if a.dim() == 3 else s) + U * b.abs())
        assert ((a - b).abs() <= bound).all()


@pytest.mark.parametrize("cfg", [c for c in SIZES if c["V"] in (3, 18, 129, 1000, 2049, 5003, 33001,
                                                                300007)] + PARKED, ids=_id)
def test_gradients_in_place_of_the_logits(cuda_device, cfg):
    r = Rows(**cfg, seed=11)
    v, _ = policy_inputs(r)
    want = run_policy(r, v, True, 0.02)
    spare = r.cz.clone(memory_format=torch.preserve_format) if r.cz.is_contiguous() else None
    got = run_policy(r, v, True, 0.02, dlogits=r.cz)
    assert got[4].data_ptr() == r.cz.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert spare is None or not torch.equal(spare, r.cz)
    r.place(cfg.get("layout", "plain"))
    logp, h, saved = rlca.token_logprobs(r.cz, r.ctok, **r.kw, want_entropy=True, want_saved=True)
    d = torch.rand(r.shape[:2], generator=r.g).cuda()
    kw = dict(r.kw, entropy=h, dentropy=d)
    want = rlca.token_logprobs_backward(d, r.cz, r.ctok, saved, **kw)
    got = rlca.token_logprobs_backward(d, r.cz, r.ctok, saved, **kw, dlogits=r.cz)
    assert torch.equal(got, want)
    r.place(cfg.get("layout", "plain"))
    K = min(r.shape[2], 9)
    index = torch.randint(-1, r.shape[2], (*r.shape[:2], K), generator=r.g).cuda()
    teacher = r.rn(*r.shape[:2], K).cuda()
    want = rlca.distill_topk(r.cz, index, teacher, **r.kw, want_grad=True)
    got = rlca.distill_topk(r.cz, index, teacher, **r.kw, dlogits=r.cz)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("N", [2, 104])
@pytest.mark.parametrize("V", [7, 30, 301, 1001, 3001, 40001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nothing_else_is_written(cuda_device, dtype, V, N):
    """Gradients as slices of a wider buffer, at every offset to the logits: what lies between
    their rows stays, and the bits do not depend on the offset."""
    r = Rows(dtype, N, 3, V, seed=12, prompt=True)
    v, _ = policy_inputs(r)
    want = run_policy(r, v, True, 0.02)[4]
    for off in range(0, 9):
        buf = torch.full((N, 4, V + 11), 7.0, dtype=dtype, device="cuda")
        run_policy(r, v, True, 0.02, dlogits=buf[:, :3, off:off + V])
        assert torch.equal(buf[:, :3, off:off + V], want)
        buf[:, :3, off:off + V] = 7.0
        assert (buf == 7.0).all()
        _, h, saved = rlca.token_logprobs(r.cz, r.ctok, want_entropy=True, want_saved=True)
        one = torch.ones(N, 3, device="cuda")
        rlca.token_logprobs_backward(one, r.cz, r.ctok, saved, entropy=h, dentropy=one,
                                     dlogits=buf[:, 1:, off:off + V])
        buf[:, 1:, off:off + V] = 7.0
        assert (buf == 7.0).all()


@pytest.mark.parametrize("V,T", [(18, 2), (1000, 2), (40000, 2), (4000, 160)])
def test_offsets_past_2_31_elements(cuda_device, V, T):
    """Rows 2^31 elements and more apart (bf16: over 4 GB)."""
    gap = (1 << 31) + 24
    r = Rows(BF16, 2, T, V, seed=13)
    buf = torch.empty(gap + T * V, dtype=BF16, device="cuda")
    far = buf.as_strided((2, T, V), (gap, V, 1))
    far.copy_(r.cz)
    gbuf = torch.empty(gap + T * V, dtype=BF16, device="cuda")
    grad = gbuf.as_strided((2, T, V), (gap, V, 1))
    v, _ = policy_inputs(r)
    r.cz = far
    check_policy(r, v, True, 0.02, run_policy(r, v, True, 0.02, dlogits=grad))


# ------------------------------------------------------------------------------ as it is used


@pytest.mark.parametrize("cfg", [c for c in SIZES if c["V"] in (18, 512, 2049, 33001, 270001)]
                         + PARKED, ids=_id)
def test_calls_repeat_bit_for_bit(cuda_device, cfg):
    r = Rows(**cfg, seed=14)
    v, _ = policy_inputs(r)
    first = run_policy(r, v, True, 0.02)
    for _ in range(3):
        for a, b in zip(run_policy(r, v, True, 0.02), first):
            assert torch.equal(a, b)


def _all_calls(r, v, out):
    """Every operator once, into `out` where that is given."""
    c = {k: t.cuda() for k, t in v.items()}
    N, T, V = r.shape
    z, tok = r.cz, r.ctok
    logp, h, saved = rlca.token_logprobs(z, tok, want_entropy=True, want_saved=True)
    d = rlca.token_logprobs_backward(c["adv"], z, tok, saved, entropy=h, dentropy=c["weight"])
    p = rlca.policy_loss(z, tok, c["old"], c["adv"], ref_logp=c["ref"], weight=c["weight"],
                         kl_coef=0.1, entropy_coef=0.01, want_entropy=True, want_grad=True)
    loss, scores, _, s = rlca.preference_loss(z, tok, ref_logp=c["ref"], want_saved=True)
    dp = rlca.preference_loss_backward(None, z, tok, s)
    dl, dd = rlca.distill_topk(z, out["index"], out["teacher"], weight=c["weight"], want_grad=True)
    return [logp, h, d, *p, loss, scores, dp, dl, dd]


@pytest.mark.parametrize("V,T", [(18, 6), (600, 6), (5000, 6), (40000, 6), (5001, 80), (70000, 16)])
def test_streams_and_graphs(cuda_device, V, T):
    """On a stream of its own, and captured into a graph that is replayed on new data."""
    r, other = Rows(BF16, 4, T, V, seed=15), Rows(BF16, 4, T, V, seed=16)
    v, _ = policy_inputs(r)
    w, _ = policy_inputs(other)
    t = dict(index=torch.randint(0, V, (4, T, 5), generator=r.g).cuda(),
             teacher=r.rn(4, T, 5).cuda())
    want, want_other = _all_calls(r, v, t), _all_calls(other, w, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late = Rows(BF16, 4, T, V, seed=15)
        got = _all_calls(late, v, t)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    static = {k: x.cuda() for k, x in v.items()}
    holder = Rows(BF16, 4, T, V, seed=15)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _all_calls(holder, static, t)
    for src, vals, expect in ((other, w, want_other), (r, v, want)):
        holder.cz.copy_(src.cz)
        holder.ctok.copy_(src.ctok)
        for k in static:
            static[k].copy_(vals[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, expect):
            assert torch.equal(a, b)


@pytest.mark.parametrize("V", [20, 600, 5000])
def test_gradients_against_differences(cuda_device, V):
    """The slope along a random direction by central differences of the call's own losses, fp32, a
    step of h = 0.01: the third derivative over 6 leaves h^2 / 6 of a few units, the losses' rounding
    (1e-6 each, M of them, at random) M^1/2 1e-6 / h."""
    r = Rows(F32, 3, 4, V, seed=17)
    v, _ = policy_inputs(r)
    # Steps by less than a border's distance: ratios stay on their side.
    v["old"] = (ref.token_logprobs(r.z.double(), r.tokens)[0] - 0.1 * r.rn(3, 4).clamp(-1, 1)).float()
    c = {k: t.cuda() for k, t in v.items()}
    direction = r.rn(3, 4, V)
    h = 0.01
    direction = (direction / direction.abs().amax()).cuda()

    def total(z):
        loss = rlca.policy_loss(z, r.ctok, c["old"], c["adv"], ref_logp=c["ref"],
                                kl_coef=0.1, entropy_coef=0.05, clip_low=0.5, clip_high=0.5)[0]
        return (loss.double() * c["weight"]).sum()

    dz = rlca.policy_loss(r.cz, r.ctok, c["old"], c["adv"], ref_logp=c["ref"], weight=c["weight"],
                          kl_coef=0.1, entropy_coef=0.05, clip_low=0.5, clip_high=0.5,
                          want_grad=True)[4]
    want = (total(r.cz + h * direction) - total(r.cz - h * direction)) / (2 * h)
    got = (dz.double() * direction).sum()
    assert abs(got - want) <= 1e-3 * (1 + abs(want))
    index = torch.randint(0, V, (3, 4, 6), generator=r.g).cuda()
    teacher = r.rn(3, 4, 6).cuda()
    distill = lambda z: (rlca.distill_topk(z, index, teacher)[0].double() * c["weight"]).sum()
    _, dz = rlca.distill_topk(r.cz, index, teacher, weight=c["weight"], want_grad=True)
    want = (distill(r.cz + h * direction) - distill(r.cz - h * direction)) / (2 * h)
    assert abs((dz.double() * direction).sum() - want) <= 1e-3 * (1 + abs(want))


def test_the_first_update_has_a_ratio_of_one(cuda_device):
    """old_logp as token_logprobs gave it: ratios are 1 to the rounding of log p."""
    r = Rows(F32, 4, 50, 1000, seed=18)
    logp, _, _ = rlca.token_logprobs(r.cz, r.ctok)
    adv = r.rn(4, 50).cuda()
    loss, again, _, kl, _ = rlca.policy_loss(r.cz, r.ctok, logp, adv, ref_logp=logp)
    assert ((loss + adv).abs() <= (ref.ROW + 2 * U * logp.abs()) * adv.abs()).all()
    assert (kl <= 1e-9).all() and (kl >= 0).all()


@pytest.mark.parametrize("V,rows", [(40, 600), (3000, 300)])
def test_two_calls_at_once(cuda_device, V, rows):
    """Calls on two streams share nothing: no workspace, no state."""
    r, other = Rows(BF16, rows, 2, V, seed=20), Rows(BF16, rows, 2, V, seed=21)
    v, _ = policy_inputs(r)
    w, _ = policy_inputs(other)
    want, want_other = run_policy(r, v, True, 0.02), run_policy(other, w, True, 0.02)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(a):
            got = run_policy(r, v, True, 0.02)
        with torch.cuda.stream(b):
            got_other = run_policy(other, w, True, 0.02)
        torch.cuda.synchronize()
        for x, y in zip((*got, *got_other), (*want, *want_other)):
            assert torch.equal(x, y)


def test_many_uncounted_rows_between(cuda_device):
    """Runs of steps that do not count, longer than what a CTA looks ahead, at a row's beginning, in
    it and at its end: only the counted ones' values, zeros between."""
    r = Rows(BF16, 3, 30000, 1100, seed=22)
    r.tokens[:] = -1
    r.tokens[0, 5], r.tokens[1, 29999], r.tokens[2, 17000:17003] = 3, 1099, 7
    r.place("plain")
    logp, _, saved = rlca.token_logprobs(r.cz, r.ctok, want_saved=True)
    counted = r.tokens >= 0
    assert int((logp != 0).sum()) == 5 and not logp.cpu()[~counted].any()
    z = r.z[counted].double()
    want = torch.log_softmax(z, -1).gather(1, r.tokens[counted][:, None])[:, 0]
    close("logp", logp.cpu()[counted], want, 1 + want.abs())
    adv = torch.ones(3, 30000, device="cuda")
    loss, _, _, _, dz = rlca.policy_loss(r.cz, r.ctok, logp, adv, want_grad=True)
    dz, loss = dz.cpu(), loss.cpu()
    assert not dz[~counted].any() and not loss[~counted].any() and dz[counted].any(1).all()
    assert ((loss[counted] + 1).abs() <= ref.ROW + 2 * U * want.abs()).all()
