"""The losses over a vocabulary over the whole range of logits and temperatures that they take:
logits at the ends of their type, tokens that are not allowed, temperatures of 1e-6 to 1e6, in
every kernel, against the 64-bit definitions."""
import math

import pytest
import torch

import policy_reference as ref
import segmented_associative_scan_gb300 as rlca
from policy_reference import close
from test_policy_gpu import BF16, F32, FP16, INF, Rows, check_policy, grad_scale, policy_inputs
from test_policy_gpu import run_policy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


def check_rows(r, tau_in_weights=False):
    """The policy loss with every term and the log-probabilities, with gradients of both; what is not
    allowed gets exactly 0. `tau_in_weights`: weights in proportion to the temperature, so that
    gradients, which it divides, stay inside the type."""
    N, T, V = r.shape
    v, counted = policy_inputs(r)
    unit = r.tau if tau_in_weights else 1.0
    v["weight"] *= unit
    got = run_policy(r, v, True, 0.02)
    check_policy(r, v, True, 0.02, got)
    barred = (r.z == -INF).cuda()
    assert not got[4][barred].any()
    z = r.leaf()
    logp, h, _ = ref.token_logprobs(z, r.tokens, r.lengths, r.tau)
    glogp, gh, saved = rlca.token_logprobs(r.cz, r.ctok, **r.kw, want_entropy=True,
                                           want_saved=True)
    logv = 1 + math.log(V)
    close("logp", glogp, logp, 1 + logp.abs())
    close("entropy", gh, h, logv)
    dl, dh = unit * r.rn(N, T), unit * r.rn(N, T)
    ((logp * dl).sum() + (h * dh).sum()).backward()
    dz = rlca.token_logprobs_backward(dl.cuda(), r.cz, r.ctok, saved, **r.kw, entropy=gh,
                                      dentropy=dh.cuda())
    close("dlogits", dz, z.grad, grad_scale(dl.abs() + dh.abs() * logv, r.tau))
    assert not dz[barred].any()


# Rows that are parked in shared memory: whole, in part, and at offsets to 16 bytes.
FIRST_PARTS = [
    dict(N=8, T=40, V=4096, layout="plain"),
    dict(N=8, T=40, V=4099, layout="wide"),
    dict(N=8, T=40, V=4100, layout="shifted"),
    dict(N=9, T=8, V=33001, layout="shifted"),
    dict(N=8, T=8, V=70001, layout="wide"),
    dict(N=8, T=8, V=131072, layout="plain"),
]


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("cfg", FIRST_PARTS, ids=lambda c: f"{c['V']}-{c['layout']}")
def test_lowest_values_before_ordinary_ones(cuda_device, cfg, dtype):
    """Rows whose first thousands of logits are the type's lowest value, -inf, or both, and the
    others ordinary; and the other way round."""
    r = Rows(dtype, **cfg, seed=31)
    N, T, V = r.shape
    low = torch.finfo(dtype).min
    z = r.z
    part = 3 * V // 4
    z[:, 0::6, :part] = low
    z[:, 1::6, :part] = low
    z[:, 1::6, :part:3] = -INF
    z[:, 2::6, :part] = -INF
    z[:, 3::6, part // 2:] = low
    z[:, 3::6, part // 2::5] = -INF
    z[:, 4::6, :part] = -INF
    z[:, 4::6, part // 4:part] = low
    # The taken token has an ordinary logit.
    top = z.float().topk(5, -1).indices
    r.tokens = top[..., 4].to(r.tokens.dtype)
    r.place(cfg["layout"])
    check_rows(r)


@pytest.mark.parametrize("V", [4096, 40000, 131072])
def test_steps_above_the_lowest_value(cuda_device, V):
    """fp16 at a temperature where the steps of 32 above -65504 are a fraction of an exponent each."""
    r = Rows(FP16, 8, 40 if V == 4096 else 8, V, tau=24.0, seed=32)
    z = -65504 + 32 * torch.randint(0, 3, r.shape, generator=r.g).float()
    z[..., :3 * V // 4] = -65504
    z.scatter_(2, r.tokens[..., None], -65440.0)
    r.z = z.to(FP16)
    r.place("plain")
    check_rows(r, tau_in_weights=True)


@pytest.mark.parametrize("cfg", FIRST_PARTS, ids=lambda c: f"{c['V']}-{c['layout']}")
def test_steps_above_the_lowest_value_among_barred_tokens(cuda_device, cfg):
    """fp16 at a temperature where the steps of 32 above -65504 are a fraction of an exponent each."""
    r = Rows(FP16, **cfg, tau=24.0, seed=32)
    N, T, V = r.shape
    z = -65504 + 32 * torch.randint(0, 3, (N, T, V), generator=r.g).float()
    z[..., :3 * V // 4] = -65504
    z[:, 1::2, 5::7] = -INF
    z.scatter_(2, r.tokens[..., None], -65440.0)
    r.z = z.to(FP16)
    r.place(cfg["layout"])
    check_rows(r, tau_in_weights=True)


# A row to a lane, to lanes of a group (whole packs and not), rows in registers of a few warps and of
# many, parked rows, and parked in part.
KERNELS = [
    dict(N=7, T=9, V=18, layout="plain"),
    dict(N=7, T=9, V=24, layout="plain"),
    dict(N=7, T=9, V=101, layout="wide"),
    dict(N=7, T=9, V=512, layout="plain"),
    dict(N=5, T=5, V=2051, layout="shifted"),
    dict(N=2, T=2, V=70001, layout="shifted"),
    dict(N=40, T=17, V=1101, layout="wide"),
    dict(N=32, T=10, V=4096, layout="plain"),
    dict(N=8, T=8, V=70001, layout="wide"),
]


def kernel_id(c):
    return f"{c['N'] * c['T']}x{c['V']}"


@pytest.mark.parametrize("tau", [1e-6, 1e-3, 30.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("cfg", KERNELS, ids=kernel_id)
def test_temperatures(cuda_device, cfg, dtype, tau):
    """Every temperature that the calls take, with tokens that are not allowed. At low ones whole logits,
    so that the largest are often alike."""
    r = Rows(dtype, **cfg, tau=tau, masked=True, seed=33)
    if tau < 1:
        r.z = r.z.float().round().to(dtype)
        r.place(cfg["layout"])
    check_rows(r, tau_in_weights=True)


@pytest.mark.parametrize("dtype,base,unit,tau", [
    (FP16, -65000.0, 32.0, 300.0), (FP16, -65000.0, 32.0, 2.0), (FP16, -60000.0, 32.0, 1e4),
    (FP16, 60000.0, 32.0, 300.0), (FP16, 60000.0, 32.0, 1e-6), (FP16, -6000.0, 4.0, 1e-6),
    (BF16, 1e38, 2.0 ** 119, 1e-6), (BF16, -3e38, 2.0 ** 120, 1e-3), (BF16, -3.3e38, 2.0 ** 120, 1e6),
    (BF16, 1e8, 2.0 ** 19, 1e6), (BF16, -1e8, 2.0 ** 19, 1e6), (F32, 1e37, 2.0 ** 101, 1e-6),
    (F32, -1e8, 8.0, 1e2)])
@pytest.mark.parametrize("cfg", KERNELS, ids=kernel_id)
def test_logits_far_from_zero(cuda_device, cfg, dtype, base, unit, tau):
    """Logits a few steps of the type apart, near its ends and far from zero, with tokens that are not
    allowed; the taken token is the likeliest."""
    r = Rows(dtype, **cfg, tau=tau, masked=True, seed=34)
    r.z = (base + unit * r.z.double().round().clamp(max=12)).to(dtype)
    r.tokens = r.z.float().argmax(-1).to(r.tokens.dtype)
    r.place(cfg["layout"])
    check_rows(r, tau_in_weights=True)


@pytest.mark.parametrize("tau", [1e-4, 1e4, 1e6])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("N,T,V", [(6, 5, 301), (6, 5, 4001), (40, 17, 1101), (8, 8, 70001)])
def test_bits_at_any_offset_and_temperature(cuda_device, N, T, V, dtype, tau):
    """A gradient's bits do not depend on where its row lies, at temperatures where the type's own
    range ends before exponents do."""
    r = Rows(dtype, N, T, V, tau=tau, masked=True, seed=35)
    v, _ = policy_inputs(r)
    v["weight"] *= tau
    want = run_policy(r, v, True, 0.02)[4]
    for off in (1, 3, 8):
        buf = torch.zeros(N, T, V + 11, dtype=dtype, device="cuda")
        run_policy(r, v, True, 0.02, dlogits=buf[..., off:off + V])
        assert torch.equal(buf[..., off:off + V], want)


@pytest.mark.parametrize("dtype,tau", [(FP16, 1e4), (BF16, 1.0), (F32, 1e4)])
@pytest.mark.parametrize("cfg", KERNELS, ids=kernel_id)
def test_in_place_where_rows_hold_anything(cuda_device, cfg, dtype, tau):
    """Gradients in the place of logits among which are -inf, the type's lowest value and rows of nothing
    else: the bits of a gradient elsewhere."""
    r = Rows(dtype, **cfg, tau=tau, masked=True, seed=36)
    low = torch.finfo(dtype).min
    r.z[:, 1] = low
    r.z[1::2, 1, ::2] = -INF
    r.z[0, 0] = -INF
    r.z[1, 0, r.shape[2] // 3:] = low
    r.place(cfg["layout"])
    v, _ = policy_inputs(r)
    v = {k: t.nan_to_num(nan=-1.0, posinf=-1.0, neginf=-1.0) for k, t in v.items()}
    v["weight"] *= tau
    logp, h, saved = rlca.token_logprobs(r.cz, r.ctok, **r.kw, want_entropy=True, want_saved=True)
    one = torch.full(r.shape[:2], tau, device="cuda")
    kw = dict(r.kw, entropy=h, dentropy=one)
    want = run_policy(r, v, True, 0.02)
    slope = rlca.token_logprobs_backward(one, r.cz, r.ctok, saved, **kw)
    got = run_policy(r, v, True, 0.02, dlogits=r.cz)
    for a, b in zip(got, want):
        assert torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))
    r.place(cfg["layout"])
    assert torch.equal(rlca.token_logprobs_backward(one, r.cz, r.ctok, saved, **kw, dlogits=r.cz),
                       slope)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("cfg", KERNELS, ids=kernel_id)
def test_taken_tokens_that_are_barred(cuda_device, cfg, dtype):
    """log p is -inf and its gradient the formula's, 1 at the token and -p elsewhere; the entropy is that
    of the other tokens, and rows beside are as they are."""
    r = Rows(dtype, **cfg, masked=True, seed=37)
    N, T, V = r.shape
    taken = r.tokens[:, 0].clone()
    r.z[:, 0].scatter_(1, taken[:, None], -INF)
    r.place(cfg["layout"])
    logp, h, saved = rlca.token_logprobs(r.cz, r.ctok, want_entropy=True, want_saved=True)
    want, wh, _ = ref.token_logprobs(r.z.double(), r.tokens)
    close("logp", logp, want, 1 + want.abs().nan_to_num(posinf=0.0))
    close("entropy", h, wh, 1 + math.log(V))
    assert (logp[:, 0] == -INF).all() and logp[:, 1:].isfinite().all()
    dl = torch.rand(N, T, generator=r.g)
    dz = rlca.token_logprobs_backward(dl.cuda(), r.cz, r.ctok, saved)
    p = torch.softmax(r.z.double(), -1)
    hot = torch.zeros_like(p).scatter_(2, r.tokens[..., None].long(), 1.0)
    close("dlogits", dz, (hot - p) * dl[..., None], dl.double()[..., None])
    # An infinite loss (a KL term) stays in its row.
    v, _ = policy_inputs(r)
    v = {k: t.nan_to_num(nan=-1.0, posinf=-1.0, neginf=-1.0) for k, t in v.items()}
    loss, _, _, kl, dz = run_policy(r, v, True, 0.02)
    assert (loss[:, 0] == INF).all() and (kl[:, 0] == INF).all()
    assert loss[:, 1:].isfinite().all() and dz[:, 1:].isfinite().all()


# ----------------------------------------------------------------------------- long sums


@pytest.mark.parametrize("dtype,N,V", [(BF16, 64, 300007), (F32, 64, 200001), (FP16, 2, 1 << 24),
                                       (F32, 1, (1 << 25) + 3), (BF16, 1, 1 << 27),
                                       (BF16, 1, 1 << 30)])
def test_sums_of_many_like_logits(cuda_device, dtype, N, V):
    """Rows whose first logits are 0 and whose others are all alike, so that every addition to a long
    sum rounds the same way: log p and H from the formula, within the bound of any row."""
    first = 1 << 17
    low = -torch.linspace(0.3, 2.7, N).to(dtype)
    z = low.cuda()[:, None, None].expand(N, 1, V).contiguous()
    z[..., :first] = 0.0
    tokens = torch.full((N, 1), 5, dtype=torch.int64, device="cuda")
    logp, h, _ = rlca.token_logprobs(z, tokens, want_entropy=True)
    c = -low.double()
    s = first + (V - first) * torch.exp(-c)
    want = -torch.log(s)
    entropy = torch.log(s) + (V - first) * torch.exp(-c) * c / s
    close("logp", logp[:, 0], want, 1 + want.abs())
    close("entropy", h[:, 0], entropy, 1 + math.log(V))
