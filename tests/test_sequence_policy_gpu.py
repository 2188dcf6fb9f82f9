"""The example policy: the losses together with the trunk and the estimators, as they are used; the
whole model's gradients against plain PyTorch operations in 64 bits."""
import pytest
import torch

import policy_reference as pref
import segmented_associative_scan_gb300 as rlca
import sequence_policy as sp
import sequence_reference as ref

pytestmark = pytest.mark.gpu

VOCAB = 48


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


class Frozen:
    """An optimizer that keeps the gradients and changes nothing."""

    def __init__(self, policy):
        self.policy, self.grads = policy, None

    def zero_grad(self, set_to_none=True):
        for p in self.policy.parameters():
            p.grad = None

    def step(self):
        self.grads = {k: p.grad for k, p in self.policy.named_parameters()}


@pytest.fixture
def policy(cuda_device):
    torch.manual_seed(4)
    torch.backends.cuda.matmul.allow_tf32 = False
    return sp.SequencePolicy(VOCAB, width=16, channels=32, dtype=torch.float32)


def plain(policy, tokens, terminated):
    """The model's 64-bit parameters, logits and values from the operators' definitions."""
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in policy.named_parameters()}
    rows = dict(terminated=terminated.cpu())
    h = ref.embed(tokens.cpu(), p["table"], policy.scale)
    x, z = (h @ p["w_in"]).split(policy.channels, dim=-1)
    u, _ = ref.conv(x, p["conv_w"], p["conv_b"], **rows)
    dt, b, c = (u @ p["w_bc"]).split([policy.rank, policy.states, policy.states], dim=-1)
    y, _ = ref.scan(u, dt @ p["w_dt"], -torch.exp(p["log_a"]), b.unsqueeze(2), c.unsqueeze(2),
                    p["d"], z, p["dt_bias"], **rows)
    return p, y @ p["w_logits"], (y @ p["w_out"]).squeeze(-1)


def check_gradients(got, p):
    """fp32 through some ten operators and sums over rows and steps: 1e-4 of the largest, as the
    critic's."""
    for name, v in p.items():
        if v.grad is None:
            assert got[name] is None, name
            continue
        want = v.grad
        assert (got[name].double().cpu() - want).abs().max() <= 1e-4 * want.abs().max(), name


def gae(reward, values, terminated, gamma, lam):
    out = torch.zeros_like(values)
    for n in range(values.shape[0]):
        a = 0.0
        for t in reversed(range(values.shape[1])):
            end = bool(terminated[n, t])
            after = 0.0 if end or t + 1 == values.shape[1] else values[n, t + 1]
            a = reward[n, t] + gamma * after - values[n, t] + (0.0 if end else gamma * lam * a)
            out[n, t] = a
    return out


def test_a_policy_update(policy):
    batch = sp.synthetic_batch(3, 20, VOCAB, seed=1)
    batch["actions"][0, :4] = -1
    g = torch.Generator().manual_seed(2)
    logp = sp.behaviour(policy, batch)
    old = logp + 0.05 * torch.randn(3, 20, generator=g).cuda()
    reference = logp + 0.3 * torch.randn(3, 20, generator=g).cuda()
    frozen = Frozen(policy)
    loss, value_loss, kl = sp.update(policy, frozen, batch, old, reference)

    p, logits, values = plain(policy, batch["tokens"], batch["terminated"])
    c = {k: v.cpu() for k, v in batch.items()}
    adv = gae(c["reward"].double(), values.detach(), c["terminated"], 0.9, 0.95)
    each, _, _, each_kl, counted = pref.policy_loss(
        logits, c["actions"], old.double().cpu(), adv, reference.double().cpu(), kl_coef=0.05,
        entropy_coef=0.01)
    w = counted.double() / counted.sum()
    policy_loss = (each * w).sum()
    want_value = ((values - (adv + values.detach())) ** 2 * w).sum()
    (policy_loss + 0.5 * want_value).backward()
    assert abs(loss.item() - policy_loss.item()) <= 1e-4 * (1 + abs(policy_loss.item()))
    assert abs(value_loss.item() - want_value.item()) <= 1e-4 * (1 + want_value.item())
    assert abs(kl.item() - (each_kl * w).sum().item()) <= 1e-4
    check_gradients(frozen.grads, p)


def test_a_preference_step(policy):
    pairs = sp.synthetic_pairs(3, 16, VOCAB, seed=3)
    with torch.no_grad():
        logits, _ = policy(pairs["tokens"], pairs["terminated"], None)
    base = rlca.token_logprobs(logits, pairs["targets"])[0]
    base = base + 0.2 * torch.randn(6, 16, generator=torch.Generator().manual_seed(4)).cuda()
    frozen = Frozen(policy)
    loss, scores = sp.prefer(policy, frozen, pairs, base, beta=0.3)
    p, logits, _ = plain(policy, pairs["tokens"], pairs["terminated"])
    want, want_scores, _, _ = pref.preference_loss(logits, pairs["targets"].cpu(),
                                                   base.double().cpu(), beta=0.3)
    want.mean().backward()
    assert abs(loss.item() - want.mean().item()) <= 1e-4
    assert (scores.double().cpu() - want_scores).abs().max() <= 1e-4
    check_gradients(frozen.grads, p)


def test_a_distillation_step(policy):
    batch = sp.synthetic_batch(2, 18, VOCAB, seed=5)
    g = torch.Generator().manual_seed(6)
    index = torch.rand(2, 18, VOCAB, generator=g).argsort(-1)[..., :7]
    teacher = torch.randn(2, 18, 7, generator=g)
    frozen = Frozen(policy)
    loss = sp.distil(policy, frozen, batch, index.cuda(), teacher.cuda())
    p, logits, _ = plain(policy, batch["tokens"], batch["terminated"])
    want, _ = pref.distill_topk(logits, index, teacher.double())
    want.mean().backward()
    assert abs(loss.item() - want.mean().item()) <= 1e-4
    check_gradients(frozen.grads, p)


def test_the_example_runs(cuda_device):
    """bf16, each step once with a real optimizer: parameters move and stay finite."""
    torch.manual_seed(0)
    policy = sp.SequencePolicy(64, width=32, channels=64)
    optimizer = torch.optim.Adam(policy.parameters(), lr=1e-3)
    before = {k: v.detach().clone() for k, v in policy.named_parameters()}
    batch = sp.synthetic_batch(8, 40, 64)
    old = sp.behaviour(policy, batch)
    loss, value_loss, kl = sp.update(policy, optimizer, batch, old, old)
    pairs = sp.synthetic_pairs(4, 32, 64)
    preferred, scores = sp.prefer(policy, optimizer, pairs, None)
    index = torch.randint(0, 64, (8, 40, 5), device="cuda")
    distilled = sp.distil(policy, optimizer, batch, index, torch.randn(8, 40, 5, device="cuda"))
    for v in (loss, value_loss, kl, preferred, scores, distilled):
        assert torch.isfinite(v).all()
    for name, v in policy.named_parameters():
        assert torch.isfinite(v).all() and not torch.equal(v.detach(), before[name]), name
