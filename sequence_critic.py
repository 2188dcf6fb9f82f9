"""A recurrent critic over token observations, trained on this library's GAE targets and then
run one token at a time: how the sequence operators and the estimators are used together.

    tokens -> embed_tokens -> input projection -> causal_conv -> selective_scan -> values
    rewards, values -> gae -> returns -> loss -> gradients back through the same operators

The recurrence restarts where an episode ends, in training (flags of the window) as in acting
(`reset`), so a window gives the values that acting gave. Projections are plain matrix
products of PyTorch; everything between them runs in the library's kernels.

Run: python sequence_critic.py
"""
from __future__ import annotations

import math

import torch

import segmented_associative_scan_gb300 as rlca


class Gradients(torch.autograd.Function):
    """The gradients `call` takes, as a function of its tensors: it has no derivative, so a second
    one through an operator fails where it would come out without that part."""

    @staticmethod
    def forward(ctx, call, *tensors):
        return call(*tensors)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the sequence operators are differentiable once")


class EmbedTokens(torch.autograd.Function):
    """scale * table[tokens]; the table's gradient by sorted tokens."""

    @staticmethod
    def forward(ctx, tokens, table, scale):
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale, ctx.dtype = table.shape[0], scale, table.dtype
        return rlca.embed_tokens(tokens, table, scale=scale)

    @staticmethod
    def backward(ctx, dout):
        (tokens,) = ctx.saved_tensors
        grad = Gradients.apply(
            lambda d: rlca.embed_tokens_backward(d, tokens, ctx.vocab, scale=ctx.scale),
            dout.contiguous())
        return None, grad.to(ctx.dtype), None


class CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, terminated, truncated):
        ctx.save_for_backward(x, weight, bias, terminated, truncated)
        return rlca.causal_conv(x, weight, bias, terminated, truncated)[0]

    @staticmethod
    def backward(ctx, dout):
        dx, dw, db = Gradients.apply(rlca.causal_conv_backward, dout.contiguous(),
                                     *ctx.saved_tensors)
        return dx, dw, db, None, None


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, terminated, truncated):
        out, _, saved = rlca.selective_scan(x, dt, A, B, C, D, z, dt_bias, terminated, truncated,
                                            want_saved=True)
        ctx.save_for_backward(x, dt, A, B, C, saved, D, z, dt_bias, terminated, truncated)
        return out

    @staticmethod
    def backward(ctx, dout):
        dx, ddt, dA, dB, dC, dD, dz, ddt_bias, _ = Gradients.apply(
            rlca.selective_scan_backward, dout.contiguous(), *ctx.saved_tensors)
        return dx, ddt, dA, dB, dC, dD, dz, ddt_bias, None, None


class SequenceCritic(torch.nn.Module):
    """Values [N, T] of token windows [N, T]; `step` gives those of one token per row."""

    def __init__(self, vocab, width=64, channels=128, states=16, taps=4, rank=8,
                 dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.scale, self.states, self.rank, self.channels = math.sqrt(width), states, rank, channels

        def weight(*shape, fan):
            w = torch.randn(*shape, device=device) / math.sqrt(fan)
            return torch.nn.Parameter(w.to(dtype))

        self.table = weight(vocab, width, fan=width)
        self.w_in = weight(width, 2 * channels, fan=width)
        self.w_bc = weight(channels, rank + 2 * states, fan=channels)
        self.w_dt = weight(rank, channels, fan=rank)
        self.w_out = weight(channels, 1, fan=channels)
        # Parameters of the operators themselves are fp32.
        f32 = dict(dtype=torch.float32, device=device)
        self.conv_w = torch.nn.Parameter((torch.rand(channels, taps, **f32) * 2 - 1)
                                         / math.sqrt(taps))
        self.conv_b = torch.nn.Parameter(torch.zeros(channels, **f32))
        self.log_a = torch.nn.Parameter(torch.log(torch.arange(1, states + 1, **f32))
                                        .repeat(channels, 1))
        self.d = torch.nn.Parameter(torch.ones(channels, **f32))
        step = torch.exp(torch.rand(channels, **f32) * math.log(100.0) + math.log(0.001))
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))

    def _project(self, u):
        bc = u @ self.w_bc
        dt, b, c = bc.split([self.rank, self.states, self.states], dim=-1)
        return dt @ self.w_dt, b, c

    def forward(self, tokens, terminated, truncated):
        h = EmbedTokens.apply(tokens, self.table, self.scale)
        x, z = (h @ self.w_in).split(self.channels, dim=-1)
        u = CausalConv.apply(x, self.conv_w, self.conv_b, terminated, truncated)
        dt, b, c = self._project(u)
        y = SelectiveScan.apply(u, dt, -torch.exp(self.log_a), b, c, self.d, z, self.dt_bias,
                                terminated, truncated)
        return (y @ self.w_out).squeeze(-1).float()

    def start(self, rows):
        """The states of `rows` environments before their first token."""
        k = self.conv_w.shape[1]
        return (torch.zeros(rows, k - 1, self.channels, dtype=self.table.dtype,
                            device=self.table.device),
                torch.zeros(rows, self.channels, self.states, device=self.table.device))

    @torch.no_grad()
    def step(self, tokens, states, reset=None):
        """Values [N] of one token per row; the states move on in place. `reset`: rows whose
        previous step ended an episode."""
        window, state = states
        h = rlca.embed_tokens(tokens, self.table, scale=self.scale)
        x, z = (h @ self.w_in).split(self.channels, dim=-1)
        u, _ = rlca.causal_conv_step(x, window, self.conv_w, self.conv_b, reset=reset)
        dt, b, c = self._project(u)
        y, _ = rlca.selective_scan_step(u, dt, -torch.exp(self.log_a), b, c, state, D=self.d,
                                        z=z, dt_bias=self.dt_bias, reset=reset)
        return (y @ self.w_out).squeeze(-1).float()


def targets(values, batch, gamma, lam):
    """GAE returns [N, T] of the window's steps, from detached values of the observed tokens
    (`with_successors`): what follows a step that was cut is the value of what was observed
    next."""
    at = batch["at"]
    successors = values.gather(1, at + 1)
    _, returns = rlca.gae(batch["reward"], values.gather(1, at), batch["terminated"],
                          batch["truncated"], successors, successors[:, -1].contiguous(),
                          gamma=gamma, lam=lam)
    return returns


def train_step(critic, optimizer, batch, gamma=0.5, lam=0.95):
    """One update of the critic on a window of rollouts; returns the loss (on the device)."""
    observed = critic(batch["observed"], batch["ends"], None)
    returns = targets(observed.detach(), batch, gamma, lam)
    loss = ((observed.gather(1, batch["at"]) - returns) ** 2).mean()
    optimizer.zero_grad(set_to_none=True)
    loss.backward()
    optimizer.step()
    return loss.detach()


def with_successors(batch):
    """Adds the tokens as they were observed: behind every truncated step, and behind the
    window's last, stands the token that was seen next in its episode (`next_tokens`), which is
    where that episode ends for the critic. `observed` and `ends` [N, L] (padding at the end of
    a row: -1), `at` [N, T]: where the window's steps are in them."""
    tokens, terminated = batch["tokens"], batch["terminated"]
    rows, steps = tokens.shape
    cut = batch["truncated"] & ~terminated
    cut[:, -1] = True
    at = torch.arange(steps, device=tokens.device) + cut.cumsum(1) - cut.long()
    width = steps + int(cut.sum(1).max())
    observed = tokens.new_full((rows, width), -1).scatter(1, at, tokens)
    ends = terminated.new_zeros(rows, width).scatter(1, at, terminated)
    n, t = cut.nonzero(as_tuple=True)
    observed[n, at[n, t] + 1] = batch["next_tokens"][n, t]
    ends[n, at[n, t] + 1] = True
    return dict(batch, observed=observed, ends=ends, at=at)


def synthetic_batch(rows, steps, vocab, seed=0, device="cuda"):
    """Token windows whose reward depends on the running episode's recent tokens, and the token
    seen after each step: the next one of the window, or, where an episode or the window ends,
    one of its own."""
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, vocab, (rows, steps), generator=g)
    reward = (tokens % 7 == 0).float() + 0.5 * (tokens.roll(1, 1) % 5 == 0).float()
    batch = dict(tokens=tokens, reward=reward,
                 terminated=torch.rand(rows, steps, generator=g) < 0.02,
                 truncated=torch.rand(rows, steps, generator=g) < 0.01)
    last = batch["terminated"] | batch["truncated"]
    last[:, -1] = True
    batch["next_tokens"] = torch.where(last, torch.randint(0, vocab, (rows, steps), generator=g),
                                       tokens.roll(-1, 1))
    return {k: v.to(device) for k, v in with_successors(batch).items()}


def main():
    torch.manual_seed(0)
    rows, steps, vocab = 64, 256, 512
    critic = SequenceCritic(vocab)
    optimizer = torch.optim.Adam(critic.parameters(), lr=3e-3)
    for i in range(60):
        loss = train_step(critic, optimizer, synthetic_batch(rows, steps, vocab, seed=i))
        if i % 10 == 0:
            print(f"update {i}: value loss {loss.item():.4f}")
    # The window's values again, one token at a time.
    batch = synthetic_batch(rows, steps, vocab, seed=1000)
    with torch.no_grad():
        window = critic(batch["tokens"], batch["terminated"], batch["truncated"])
    states, reset, values = critic.start(rows), None, []
    ended = batch["terminated"] | batch["truncated"]
    for t in range(steps):
        values.append(critic.step(batch["tokens"][:, t].contiguous(), states, reset))
        reset = ended[:, t].contiguous()
    diff = (torch.stack(values, 1) - window).abs().max().item()
    print(f"acting token by token: largest difference to the window's values {diff:.4f} "
          f"(values up to {window.abs().max().item():.2f})")


if __name__ == "__main__":
    main()
