"""The example model: operators and estimators together, trained and then run token by token."""
import pytest
import torch

import segmented_associative_scan_gb300 as rlca
import sequence_critic as sc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


def test_training_lowers_the_loss(cuda_device):
    """Updates on one batch towards fixed returns (bootstrapped ones move with the values)."""
    torch.manual_seed(0)
    critic = sc.SequenceCritic(64, width=32, channels=64)
    optimizer = torch.optim.Adam(critic.parameters(), lr=3e-3)
    batch = sc.synthetic_batch(16, 96, 64)
    target = rlca.discounted_return(batch["reward"], batch["terminated"], gamma=0.5)
    losses = []
    for _ in range(40):
        values = critic(batch["tokens"], batch["terminated"], batch["truncated"])
        loss = (values - target).square().mean()
        optimizer.zero_grad(set_to_none=True)
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    assert sum(losses[-5:]) < 0.7 * sum(losses[:5])
    for name, p in critic.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all(), name


def test_an_update_with_gae_targets(cuda_device):
    torch.manual_seed(0)
    critic = sc.SequenceCritic(64, width=32, channels=64)
    before = {k: v.detach().clone() for k, v in critic.named_parameters()}
    optimizer = torch.optim.Adam(critic.parameters(), lr=3e-3)
    loss = sc.train_step(critic, optimizer, sc.synthetic_batch(16, 96, 64))
    assert torch.isfinite(loss) and loss > 0
    for name, p in critic.named_parameters():
        assert not torch.equal(p.detach(), before[name]), name


def test_acting_gives_the_windows_values(cuda_device):
    """In fp32 the two forms differ by rounding only: the sums run in other orders, some tens of
    roundings of 2^-24 relative to the largest value."""
    torch.manual_seed(1)
    critic = sc.SequenceCritic(64, width=32, channels=64, dtype=torch.float32)
    batch = sc.synthetic_batch(8, 60, 64, seed=5)
    torch.backends.cuda.matmul.allow_tf32 = False
    with torch.no_grad():
        window = critic(batch["tokens"], batch["terminated"], batch["truncated"])
    states, reset, values = critic.start(8), None, []
    ended = batch["terminated"] | batch["truncated"]
    for t in range(60):
        values.append(critic.step(batch["tokens"][:, t].contiguous(), states, reset))
        reset = ended[:, t].contiguous()
    assert ended.any()
    diff = (torch.stack(values, 1) - window).abs().max()
    assert diff <= 256 * 2.0 ** -24 * window.abs().max()


def test_gradients_against_plain_operators(cuda_device):
    """The example's gradients, fp32, against the same model on plain PyTorch operations in 64
    bits."""
    torch.manual_seed(2)
    critic = sc.SequenceCritic(40, width=16, channels=32, dtype=torch.float32)
    batch = sc.synthetic_batch(3, 30, 40, seed=9)
    torch.backends.cuda.matmul.allow_tf32 = False
    critic(batch["tokens"], batch["terminated"], batch["truncated"]).square().sum().backward()

    import sequence_reference as ref
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in critic.named_parameters()}
    rows = dict(terminated=batch["terminated"].cpu(), truncated=batch["truncated"].cpu())
    h = ref.embed(batch["tokens"].cpu(), p["table"], critic.scale)
    x, z = (h @ p["w_in"]).split(critic.channels, dim=-1)
    u, _ = ref.conv(x, p["conv_w"], p["conv_b"], **rows)
    dt, b, c = (u @ p["w_bc"]).split([critic.rank, critic.states, critic.states], dim=-1)
    y, _ = ref.scan(u, dt @ p["w_dt"], -torch.exp(p["log_a"]), b.unsqueeze(2), c.unsqueeze(2),
                    p["d"], z, p["dt_bias"], **rows)
    (y @ p["w_out"]).square().sum().backward()
    for name, q in critic.named_parameters():
        got, want = q.grad.double().cpu(), p[name].grad
        assert (got - want).abs().max() <= 1e-4 * want.abs().max(), name


def test_targets_against_their_definition(cuda_device):
    """GAE returns step by step in 64 bits, each bootstrapped from the value of the observation
    after it. The estimator's own bound: 1e-4 of 1 plus the largest."""
    batch = sc.synthetic_batch(6, 50, 64, seed=11)
    assert batch["truncated"].any() and batch["terminated"].any()
    torch.manual_seed(3)
    critic = sc.SequenceCritic(64, width=32, channels=64, dtype=torch.float32)
    with torch.no_grad():
        values = critic(batch["observed"], batch["ends"], None)
        window = critic(batch["tokens"], batch["terminated"], batch["truncated"])
    gamma, lam = 0.9, 0.8
    got = sc.targets(values, batch, gamma, lam).double().cpu()
    b = {k: v.cpu() for k, v in batch.items()}
    v = values.double().cpu()
    # The window's own values are the same with and without the successors put in.
    assert (v.gather(1, b["at"]) - window.double().cpu()).abs().max() <= 1e-4 * (1 + v.abs().max())
    want = torch.zeros(6, 50, dtype=torch.float64)
    for n in range(6):
        advantage = 0.0
        for t in reversed(range(50)):
            i = int(b["at"][n, t])
            term = bool(b["terminated"][n, t])
            ended = term or bool(b["truncated"][n, t])
            after = 0.0 if term else v[n, i + 1]
            delta = b["reward"][n, t].double() + gamma * after - v[n, i]
            advantage = delta + (0.0 if ended else gamma * lam * advantage)
            want[n, t] = v[n, i] + advantage
    assert (got - want).abs().max() <= 1e-4 * (1 + want.abs().max())
