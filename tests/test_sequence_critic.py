"""The example's training step on the host: what it bootstraps from, with the model and the
estimator replaced by plain ones (no GPU needed)."""
import pytest
import torch

import sequence_critic as sc

VOCAB, DECAY = 50, 0.8


def value_of(tokens):
    """The stand-in's value after the tokens of an episode so far."""
    v = 0.0
    for token in tokens:
        v = DECAY * v + token + 1
    return v


class PlainCritic(torch.nn.Module):
    """A recurrence over the episode's tokens, times a parameter."""

    def __init__(self):
        super().__init__()
        self.scale = torch.nn.Parameter(torch.ones((), dtype=torch.float64))

    def forward(self, tokens, terminated, truncated):
        ended = terminated if truncated is None else terminated | truncated
        rows = []
        for row, ends in zip(tokens.tolist(), ended.tolist()):
            v, out = 0.0, []
            for token, end in zip(row, ends):
                v = DECAY * v + token + 1
                out.append(v)
                v = 0.0 if end else v
            rows.append(out)
        return self.scale * torch.tensor(rows, dtype=torch.float64)


def test_a_step_bootstraps_from_the_observation_after_it(monkeypatch):
    """A truncated step's successor is the value of what was observed next in its episode, the
    window's that of the token after it; neither is the step's own value, nor that of the next
    episode's first step."""
    rows, steps = 12, 40
    batch = sc.synthetic_batch(rows, steps, VOCAB, seed=3, device="cpu")
    batch["truncated"][0, 7] = True   # ends of both kinds, and one at the window's end
    batch["terminated"][0, 7] = False
    batch["truncated"][1, 9:11] = True
    batch["terminated"][1, 9:11] = False
    batch["terminated"][2, 5] = batch["truncated"][2, 5] = True
    batch["truncated"][3, -1], batch["terminated"][3, -1] = True, False
    batch["terminated"][4, -1] = True
    batch = sc.with_successors(batch)
    got = {}

    def gae(reward, value, terminated, truncated, trunc_value, bootstrap, gamma, lam):
        got.update(value=value, trunc_value=trunc_value, bootstrap=bootstrap)
        return None, torch.zeros_like(value)

    monkeypatch.setattr(sc.rlca, "gae", gae)
    critic = PlainCritic()
    loss = sc.train_step(critic, torch.optim.SGD(critic.parameters(), lr=0.0), batch)
    seen = 0
    want = torch.zeros(rows, steps, dtype=torch.float64)
    for n in range(rows):
        episode = []
        for t in range(steps):
            episode.append(int(batch["tokens"][n, t]))
            want[n, t] = value_of(episode)
            term, trunc = bool(batch["terminated"][n, t]), bool(batch["truncated"][n, t])
            after = value_of(episode + [int(batch["next_tokens"][n, t])])
            if trunc and not term:
                assert got["trunc_value"][n, t].item() == pytest.approx(after, rel=1e-12)
                seen += 1
            elif t == steps - 1 and not term:
                assert got["bootstrap"][n].item() == pytest.approx(after, rel=1e-12)
            if term or trunc:
                episode = []
    assert seen >= 4
    assert torch.allclose(got["value"], want, rtol=1e-12)
    # The loss is over the window's steps, once each (the targets here are 0).
    assert loss.item() == pytest.approx(want.square().mean().item(), rel=1e-12)


def test_next_tokens_are_the_windows_own_where_the_episode_goes_on():
    batch = sc.synthetic_batch(6, 30, VOCAB, seed=4, device="cpu")
    ended = batch["terminated"] | batch["truncated"]
    on = ~ended[:, :-1]
    assert on.any() and ended.any()
    assert torch.equal(batch["next_tokens"][:, :-1][on], batch["tokens"][:, 1:][on])
    assert batch["next_tokens"].min() >= 0 and batch["next_tokens"].max() < VOCAB


@pytest.mark.parametrize("name", ["EmbedTokens", "CausalConv", "SelectiveScan"])
def test_a_second_derivative_is_refused(monkeypatch, name):
    """The gradients' kernels have no gradients: a derivative of one that would need them fails,
    it does not come out without their part. The kernels are replaced by a sine and its
    derivative."""
    x = torch.linspace(-1, 1, 6, dtype=torch.float64).view(1, 6, 1).requires_grad_()
    w = torch.zeros(1, 1)
    sine = lambda v: torch.sin(v.detach())
    slope = lambda dout, v: dout.detach() * torch.cos(v.detach())
    monkeypatch.setattr(sc.rlca, "embed_tokens", lambda tok, table, scale: sine(table))
    monkeypatch.setattr(sc.rlca, "embed_tokens_backward",
                        lambda dout, tok, vocab, scale: slope(dout, x))
    monkeypatch.setattr(sc.rlca, "causal_conv", lambda v, *a: (sine(v), None))
    monkeypatch.setattr(sc.rlca, "causal_conv_backward",
                        lambda dout, v, *a: (slope(dout, v), None, None))
    monkeypatch.setattr(sc.rlca, "selective_scan",
                        lambda v, *a, want_saved: (sine(v), None, torch.zeros(1)))
    monkeypatch.setattr(sc.rlca, "selective_scan_backward",
                        lambda dout, v, *a: (slope(dout, v),) + (None,) * 8)
    if name == "EmbedTokens":
        out = sc.EmbedTokens.apply(torch.zeros(1, dtype=torch.int64), x, 1.0)
    elif name == "CausalConv":
        out = sc.CausalConv.apply(x, w, None, None, None)
    else:
        out = sc.SelectiveScan.apply(x, w, w, w, w, None, None, None, None, None)
    (first,) = torch.autograd.grad((out * x).sum(), x, create_graph=True)
    assert torch.allclose(first, torch.sin(x) + x * torch.cos(x))
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(first.sum(), x, retain_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        first.sum().backward()
