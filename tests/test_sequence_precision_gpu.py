"""Elementwise accuracy of the functions inside the sequence operators, where one shows alone: a
call is set up so that its output is the function's value, and compared relative to it. Bounds are
sums of the roundings on the way (u = 2^-24, a rounding in 32 bits)."""
import pytest
import torch

import segmented_associative_scan_gb300 as rlca
import sequence_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


def relative(got, want):
    return ((got.double() - want) / want).abs().max().item()


def _gates(lo, hi, n=1 << 16):
    return torch.linspace(lo, hi, n, device="cuda").view(1, 1, n)


def test_gates_in_fp32(cuda_device):
    """x sigmoid(x), down to where it is smallest: CUDA's expf (2 u), the sum, the reciprocal and
    the product (1 u each), 5 u, and a sixth for second order."""
    z = _gates(-80.0, 20.0)
    E = z.shape[-1]
    want = z.double() * torch.sigmoid(z.double())
    one, zero = torch.ones(E, 1, device="cuda"), torch.zeros(1, 1, 1, device="cuda")
    out, _ = rlca.causal_conv(z, one)
    assert relative(out, want) <= 6 * U
    step, _ = rlca.causal_conv_step(z[:, 0], torch.empty(1, 0, E, device="cuda"), one)
    assert relative(step, want[:, 0]) <= 6 * U
    # y = D x = 1, gated.
    x, A, D = torch.ones_like(z), -one, one[:, 0].contiguous()
    out, _, _ = rlca.selective_scan(x, x, A, zero, zero, D=D, z=z)
    assert relative(out, want) <= 6 * U
    step, _ = rlca.selective_scan_step(x[:, 0], x[:, 0], A, zero[:, 0], zero[:, 0],
                                       torch.zeros(1, E, 1, device="cuda"), D=D, z=z[:, 0])
    assert relative(step, want[:, 0]) <= 6 * U


def test_gate_derivatives_in_fp32(cuda_device):
    """s (1 + p (1 - s)) with s = sigmoid(p) (4 u, no product): 1 - s, the multiply-add and the
    product add 1 u each, times p / (1 + p) <= 1.5 in front of the bracket for p <= -3: 9 u."""
    p = _gates(-80.0, -3.0)
    E = p.shape[-1]
    s = torch.sigmoid(p.double())
    one = torch.ones(E, 1, device="cuda")
    dx, _, _ = rlca.causal_conv_backward(torch.ones_like(p), p, one)
    assert relative(dx, s * (1 + p.double() * (1 - s))) <= 9 * U
    # ddt = x (q C B) sigmoid(dt), all ones but the last.
    dt, x, b = _gates(-80.0, 20.0), torch.ones_like(p), torch.ones(1, 1, 1, device="cuda")
    _, _, saved = rlca.selective_scan(x, dt, -one, b, b, want_saved=True)
    ddt = rlca.selective_scan_backward(x, x, dt, -one, b, b, saved)[1]
    assert relative(ddt, torch.sigmoid(dt.double())) <= 6 * U


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("lo,hi", [(-80.0, -10.0), (-10.0, 20.0)])
def test_step_sizes(cuda_device, dtype, lo, hi):
    """softplus, read off the fp32 state that one step from 0 leaves with x = B = 1. The fast
    exponential is 4 u off, the reciprocal 2 u; the correction of the exponential, 2 + e, e / (2 + e),
    the polynomial (with its own error) and the last sum 1 u each: 11 u. CUDA's functions are
    nearer."""
    E = 1 << 16
    bias = torch.linspace(lo, hi, E, device="cuda")
    zero = torch.zeros(1, 1, E, dtype=dtype, device="cuda")
    one, b = torch.ones_like(zero), torch.ones(1, 1, 1, dtype=dtype, device="cuda")
    A = -torch.ones(E, 1, device="cuda")
    want = torch.logaddexp(bias.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    _, final, _ = rlca.selective_scan(one, zero, A, b, b, dt_bias=bias, want_state=True)
    assert relative(final[0, :, 0], want) <= 11 * U
    state = torch.zeros(1, E, 1, device="cuda")
    rlca.selective_scan_step(one[:, 0], zero[:, 0], A, b[:, 0], b[:, 0], state, dt_bias=bias)
    assert relative(state[0, :, 0], want) <= 11 * U


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
def test_step_sizes_at_infinity(cuda_device, dtype):
    inf, nan = float("inf"), float("nan")
    dt = torch.tensor([-inf, inf, nan, -1e4, 1e4, 0.0], device="cuda").to(dtype).view(1, 1, 6)
    one, b = torch.ones_like(dt), torch.ones(1, 1, 1, dtype=dtype, device="cuda")
    A = -torch.ones(6, 1, device="cuda")
    _, final, _ = rlca.selective_scan(one, dt, A, b, b, want_state=True)
    got, want = final[0, :, 0].cpu(), torch.logaddexp(dt[0, 0].double().cpu(), torch.zeros(6).double())
    assert got[0] == 0 and got[1] == inf and got[2].isnan() and got[3] == 0
    assert got[4] == want[4] and relative(got[5:], want[5:]) <= 11 * U


def _norm(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("T,S", [(90, 16), (300, 8)])
def test_fp32_results_keep_their_digits(cuda_device, dtype, T, S):
    """What is fp32 in every type: final states and the gradients of parameters and initial states,
    from inputs that the definition in 64 bits gets exactly as the kernels do. A state of some ten
    steps' memory sums ten products whose step size (1.5 u rms), decays (0.6 u rms a step) and
    products (1 u) are rounded at random: 4 u rms. Four times that is allowed, 1e-6 of the norm, for
    states and for sums over them alike."""
    g = torch.Generator().manual_seed(7 + T)
    rn = lambda *s: torch.randn(*s, generator=g)
    N, E = 3, 48
    v = dict(x=rn(N, T, E).to(dtype), dt=(0.5 * rn(N, T, E)).to(dtype),
             A=-torch.rand(E, S, generator=g) * 2 - 0.5, B=rn(N, T, 1, S).to(dtype),
             C=rn(N, T, 1, S).to(dtype), D=rn(E), z=rn(N, T, E).to(dtype),
             dt_bias=-2.0 + 0.3 * rn(E), init_state=rn(N, E, S))
    rows = dict(terminated=torch.rand(N, T, generator=g) < 0.02,
                lengths=torch.tensor([T, T - 37, T // 2], dtype=torch.int32))
    dout, d_final = rn(N, T, E).to(dtype), rn(N, E, S)
    leaves = {k: t.double().requires_grad_() for k, t in v.items()}
    out, final = ref.scan(**leaves, **rows)
    ((out * dout.double()).sum() + (final * d_final.double()).sum()).backward()
    c = {k: t.cuda() for k, t in v.items()}
    r = {k: t.cuda() for k, t in rows.items()}
    _, got, saved = rlca.selective_scan(**c, **r, want_state=True, want_saved=True)
    c.pop("init_state")
    grads = rlca.selective_scan_backward(dout.cuda(), saved=saved, **c, **r,
                                         d_final_state=d_final.cuda(), want_d_init=True)
    assert _norm(got, final.detach()) <= 16 * U
    for k, i in (("A", 2), ("D", 5), ("dt_bias", 7), ("init_state", 8)):
        assert _norm(grads[i], leaves[k].grad) <= 16 * U, k


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
def test_fp32_filter_gradients_keep_their_digits(cuda_device, dtype):
    """dweight and dbias: gates within 6 u (16-bit: 4 u rms for |p| <= 5), products, and sums of 32
    steps, 4 warps and a few spans in a row, whose roundings add up at random to a few u: 16 u."""
    g = torch.Generator().manual_seed(9)
    N, T, E, K = 3, 333, 65, 4
    rn = lambda *s: torch.randn(*s, generator=g)
    x, dout, w, b = rn(N, T, E).to(dtype), rn(N, T, E).to(dtype), rn(E, K) / 2, rn(E)
    x6, w6, b6 = (t.double().requires_grad_() for t in (x, w, b))
    ref.conv(x6, w6, b6)[0].backward(dout.double())
    _, dw, db = rlca.causal_conv_backward(dout.cuda(), x.cuda(), w.cuda(), b.cuda())
    assert _norm(dw, w6.grad) <= 16 * U and _norm(db, b6.grad) <= 16 * U
