"""A recurrent token policy and how it is trained with this library's losses: the trunk of the
sequence operators, advantages of the estimators, and

  update    a clipped policy update on rollouts, with a KL term to a frozen reference
  prefer    the preference loss of paired answers
  distil    distillation from a teacher's top logits

    tokens -> embed_tokens -> causal_conv -> selective_scan -> logits, values
    rewards, values -> gae -> advantages
    logits, advantages, behaviour log-probabilities -> policy_loss -> gradients back

The losses give their gradients by the logits themselves (`policy_loss` and `distill_topk` from the
read that gives the loss), so a step hands them to the logits' own backward pass.

Run: python sequence_policy.py
"""
from __future__ import annotations

import torch

import segmented_associative_scan_gb300 as rlca
from sequence_critic import CausalConv, EmbedTokens, SelectiveScan, SequenceCritic


class SequencePolicy(SequenceCritic):
    """Logits [N, T, vocab] of the next token and values [N, T] of token windows [N, T]."""

    def __init__(self, vocab, **kw):
        super().__init__(vocab, **kw)
        fan = self.channels
        w = torch.randn(fan, vocab, device=self.w_out.device) / fan ** 0.5
        self.w_logits = torch.nn.Parameter(w.to(self.w_out.dtype))

    def forward(self, tokens, terminated, truncated):
        h = EmbedTokens.apply(tokens, self.table, self.scale)
        x, z = (h @ self.w_in).split(self.channels, dim=-1)
        u = CausalConv.apply(x, self.conv_w, self.conv_b, terminated, truncated)
        dt, b, c = self._project(u)
        y = SelectiveScan.apply(u, dt, -torch.exp(self.log_a), b, c, self.d, z, self.dt_bias,
                                terminated, truncated)
        return y @ self.w_logits, (y @ self.w_out).squeeze(-1).float()


def counted_mean(tokens, vocab):
    """Weights [N, T] of a mean over the steps whose token counts."""
    inside = ((tokens >= 0) & (tokens < vocab)).float()
    return inside / inside.sum().clamp(min=1)


@torch.no_grad()
def behaviour(policy, batch):
    """Log-probabilities [N, T] of a batch's actions under a policy: that of the acting policy, or
    of a frozen reference."""
    logits, _ = policy(batch["tokens"], batch["terminated"], None)
    return rlca.token_logprobs(logits, batch["actions"])[0]


def update(policy, optimizer, batch, old_logp, ref_logp, gamma=0.9, lam=0.95, kl_coef=0.05,
           entropy_coef=0.01, value_coef=0.5):
    """One clipped policy update; returns (policy loss, value loss, KL) on the device. The window
    ends its episodes (`terminated`)."""
    logits, values = policy(batch["tokens"], batch["terminated"], None)
    advantages, returns = rlca.gae(batch["reward"], values.detach(), batch["terminated"],
                                   gamma=gamma, lam=lam)
    weight = counted_mean(batch["actions"], logits.shape[-1])
    loss, _, _, kl, dlogits = rlca.policy_loss(
        logits.detach(), batch["actions"], old_logp, advantages, ref_logp=ref_logp, weight=weight,
        kl_coef=kl_coef, entropy_coef=entropy_coef, want_grad=True)
    value_loss = ((values - returns) ** 2 * weight).sum()
    optimizer.zero_grad(set_to_none=True)
    torch.autograd.backward([logits, value_coef * value_loss], [dlogits, None])
    optimizer.step()
    return (loss * weight).sum(), value_loss.detach(), (kl * weight).sum()


def prefer(policy, optimizer, pairs, ref_logp, beta=0.1):
    """One step on the preference loss of pairs (`tokens`, `targets` [2 P, T], the preferred
    answers first; targets outside the vocabulary do not count); returns (mean loss, scores)."""
    logits, _ = policy(pairs["tokens"], pairs["terminated"], None)
    held = logits.detach()
    loss, scores, _, saved = rlca.preference_loss(held, pairs["targets"], ref_logp=ref_logp,
                                                  beta=beta, want_saved=True)
    dloss = torch.full_like(loss, 1.0 / loss.numel())
    dlogits = rlca.preference_loss_backward(dloss, held, pairs["targets"], saved)
    optimizer.zero_grad(set_to_none=True)
    logits.backward(dlogits)
    optimizer.step()
    return loss.mean(), scores


def distil(policy, optimizer, batch, index, teacher):
    """One step towards a teacher's top logits (index, teacher [N, T, K]); returns the mean loss."""
    logits, _ = policy(batch["tokens"], batch["terminated"], None)
    weight = torch.full(logits.shape[:2], 1.0 / logits[..., 0].numel(), device=logits.device)
    loss, dlogits = rlca.distill_topk(logits.detach(), index, teacher, weight=weight, want_grad=True)
    optimizer.zero_grad(set_to_none=True)
    logits.backward(dlogits)
    optimizer.step()
    return (loss * weight).sum()


def synthetic_batch(rows, steps, vocab, seed=0, device="cuda"):
    """Token windows and actions; an action that repeats the step's token is rewarded."""
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, vocab, (rows, steps), generator=g)
    guess = torch.randint(0, vocab, (rows, steps), generator=g)
    actions = torch.where(torch.rand(rows, steps, generator=g) < 0.3, tokens, guess)
    terminated = torch.rand(rows, steps, generator=g) < 0.05
    terminated[:, -1] = True
    batch = dict(tokens=tokens, actions=actions, terminated=terminated,
                 reward=(actions == tokens).float())
    return {k: v.to(device) for k, v in batch.items()}


def synthetic_pairs(pairs, steps, vocab, seed=0, device="cuda"):
    """Answers to the same prompts: the preferred ones repeat the prompt's last token, the others do
    not. The prompt (the first quarter) does not count."""
    g = torch.Generator().manual_seed(seed)
    prompt = steps // 4
    tokens = torch.randint(0, vocab, (2 * pairs, steps + 1), generator=g)
    tokens[pairs:, :prompt + 1] = tokens[:pairs, :prompt + 1]
    tokens[:pairs, prompt + 1:] = tokens[:pairs, prompt:prompt + 1]
    targets = tokens[:, 1:].clone()
    targets[:, :prompt] = -1
    batch = dict(tokens=tokens[:, :-1].contiguous(), targets=targets,
                 terminated=torch.zeros(2 * pairs, steps, dtype=torch.bool))
    return {k: v.to(device) for k, v in batch.items()}


def main():
    torch.manual_seed(0)
    vocab = 256
    policy, reference = SequencePolicy(vocab), SequencePolicy(vocab)
    reference.load_state_dict(policy.state_dict())
    optimizer = torch.optim.Adam(policy.parameters(), lr=1e-3)
    for i in range(8):
        batch = synthetic_batch(32, 128, vocab, seed=i)
        old, ref = behaviour(policy, batch), behaviour(reference, batch)
        for _ in range(4):
            loss, value_loss, kl = update(policy, optimizer, batch, old, ref)
        print(f"update {i}: policy loss {loss.item():.4f}, value loss {value_loss.item():.4f}, "
              f"KL to the reference {kl.item():.4f}")
    pairs = synthetic_pairs(16, 64, vocab)
    with torch.no_grad():
        logits, _ = reference(pairs["tokens"], pairs["terminated"], None)
        ref = rlca.token_logprobs(logits, pairs["targets"])[0]
    for i in range(8):
        loss, scores = prefer(policy, optimizer, pairs, ref)
        print(f"preference {i}: loss {loss.item():.4f}")
    for i in range(8):
        batch = synthetic_batch(32, 128, vocab, seed=100 + i)
        with torch.no_grad():
            top = reference(batch["tokens"], batch["terminated"], None)[0].topk(16, dim=-1)
        loss = distil(policy, optimizer, batch, top.indices, top.values)
        print(f"distillation {i}: loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
