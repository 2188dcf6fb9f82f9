"""Sequence-model operators on the GPU against their 64-bit definitions: the selective scan,
the causal convolution and the token embedding, their gradients and their one-token forms."""
import math

import pytest
import torch

import segmented_associative_scan_gb300 as rlca
import sequence_reference as ref
from sequence_reference import check

pytestmark = pytest.mark.gpu

F32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _flags(N, T, g, p=0.15):
    return torch.rand(N, T, generator=g) < p


def _lengths(N, T, g):
    v = torch.randint(0, T + 1, (N,), generator=g, dtype=torch.int32)
    v[0] = T
    if N > 1:
        v[1] = 0
    return v


class ScanCase:
    """Inputs on the CPU in their type; `cuda()` arguments and 64-bit leaves."""

    def __init__(self, dtype, N, T, E, S, G=1, flags=False, ragged=False, init=False, gate=True,
                 bias=True, skip=True, softplus=True, seed=0):
        g = _gen(seed)
        rn = lambda *s: torch.randn(*s, generator=g)
        self.softplus = softplus
        self.v = dict(x=rn(N, T, E).to(dtype), dt=(0.5 * rn(N, T, E)).to(dtype),
                      B=rn(N, T, G, S).to(dtype), C=rn(N, T, G, S).to(dtype),
                      A=-torch.rand(E, S, generator=g) * S - 0.05)
        if not softplus:
            self.v["dt"] = torch.rand(N, T, E, generator=g).mul(0.2).to(dtype)
        self.v["D"] = rn(E) if skip else None
        self.v["z"] = rn(N, T, E).to(dtype) if gate else None
        self.v["dt_bias"] = -2.0 + rn(E) if bias else None
        self.v["init_state"] = rn(N, E, S) if init else None
        self.rows = dict(terminated=_flags(N, T, g) if flags else None,
                         truncated=_flags(N, T, g, 0.05) if flags else None,
                         lengths=_lengths(N, T, g) if ragged else None)
        self.dout = rn(N, T, E).to(dtype)
        self.d_final = rn(N, E, S)

    def args(self):
        c = {k: None if v is None else v.cuda() for k, v in self.v.items()}
        r = {k: None if v is None else v.cuda() for k, v in self.rows.items()}
        return c, r

    def forward(self, **kw):
        c, r = self.args()
        return rlca.selective_scan(**c, **r, dt_softplus=self.softplus, **kw)

    def reference(self, grads=False):
        leaves = {k: None if v is None else v.double().requires_grad_(grads)
                  for k, v in self.v.items()}
        out, final = ref.scan(**leaves, **self.rows, dt_softplus=self.softplus)
        if not grads:
            return out, final
        loss = (out * self.dout.double()).sum() + (final * self.d_final.double()).sum()
        loss.backward()
        zero = lambda t: torch.zeros_like(t) if t.grad is None else t.grad
        return out, final, {k: None if t is None else zero(t) for k, t in leaves.items()}


SCANS = [
    dict(dtype=F32, N=2, T=40, E=24, S=16),
    dict(dtype=BF16, N=2, T=40, E=256, S=16, flags=True),
    dict(dtype=FP16, N=3, T=37, E=129, S=16, flags=True, ragged=True, init=True),
    dict(dtype=F32, N=3, T=50, E=130, S=10, G=2, flags=True, ragged=True, init=True, gate=False),
    dict(dtype=BF16, N=2, T=33, E=64, S=16, G=4, bias=False, skip=False),
    dict(dtype=F32, N=2, T=17, E=12, S=1, flags=True, init=True),
    dict(dtype=F32, N=2, T=35, E=140, S=4),
    dict(dtype=FP16, N=2, T=35, E=136, S=5, flags=True),
    dict(dtype=BF16, N=2, T=20, E=72, S=32, init=True),
    dict(dtype=F32, N=2, T=20, E=9, S=33, G=3, flags=True),
    dict(dtype=F32, N=1, T=35, E=40, S=64, init=True),
    dict(dtype=F32, N=2, T=21, E=16, S=16, softplus=False, gate=False, bias=False),
    dict(dtype=F32, N=4, T=1, E=33, S=16, flags=True, init=True),
    dict(dtype=F32, N=2, T=15, E=8, S=8, init=True),
    dict(dtype=F32, N=2, T=16, E=8, S=8, flags=True, init=True),
    dict(dtype=BF16, N=1, T=300, E=128, S=16, flags=True),
    dict(dtype=F32, N=40, T=9, E=5, S=3, flags=True, ragged=True),
    dict(dtype=F32, N=1, T=700, E=16, S=16, init=True),
    dict(dtype=FP16, N=2, T=523, E=40, S=16, flags=True, ragged=True, init=True),
]


def _id(c):
    return "-".join(f"{k}{str(v).replace('torch.', '')}" for k, v in c.items())


@pytest.mark.parametrize("cfg", SCANS, ids=_id)
def test_scan_forward_and_backward(cuda_device, cfg):
    case = ScanCase(**cfg)
    dtype = cfg["dtype"]
    out, final, saved = case.forward(want_state=True, want_saved=True)
    ro, rf, rg = case.reference(grads=True)
    check("out", out, ro)
    check("final", final, rf)
    c, r = case.args()
    init = c.pop("init_state")
    dx, ddt, dA, dB, dC, dD, dz, dbias, dinit = rlca.selective_scan_backward(
        case.dout.cuda(), saved=saved, **c, **r, dt_softplus=case.softplus,
        d_final_state=case.d_final.cuda(), want_d_init=init is not None)
    for name, got in (("x", dx), ("dt", ddt), ("A", dA), ("B", dB), ("C", dC), ("D", dD),
                      ("z", dz), ("dt_bias", dbias), ("init_state", dinit)):
        if rg[name] is None:
            assert got is None
        else:
            check("d" + name, got, rg[name], dtype if got.dtype == dtype else F32)


def test_scan_no_steps_carries_the_state(cuda_device):
    case = ScanCase(F32, 3, 0, 20, 16, init=True)
    out, final, saved = case.forward(want_state=True, want_saved=True)
    assert out.shape == (3, 0, 20) and torch.equal(final.cpu(), case.v["init_state"])
    c, r = case.args()
    c.pop("init_state")
    grads = rlca.selective_scan_backward(case.dout.cuda(), saved=saved, **c, **r,
                                         d_final_state=case.d_final.cuda(), want_d_init=True)
    assert not grads[2].any() and not grads[5].any() and not grads[7].any()
    assert torch.equal(grads[8].cpu(), case.d_final)


def test_scan_no_rows_gives_zero_parameter_gradients(cuda_device):
    case = ScanCase(F32, 0, 5, 20, 16)
    out, final, saved = case.forward(want_state=True, want_saved=True)
    assert out.shape == (0, 5, 20) and final.shape == (0, 20, 16)
    c, r = case.args()
    c.pop("init_state")
    grads = rlca.selective_scan_backward(case.dout.cuda(), saved=saved, **c, **r)
    for k in (2, 5, 7):
        assert not grads[k].any()


def test_scan_windows_and_steps_continue_one_another(cuda_device):
    """One window, two windows and single tokens give the same outputs and states."""
    case = ScanCase(F32, 3, 45, 36, 16, flags=True, init=True, seed=5)
    c, r = case.args()
    whole, final, _ = rlca.selective_scan(**c, **r, want_state=True)
    state, parts = c["init_state"], []
    for a, b in ((0, 19), (19, 45)):
        cut = {k: v[:, a:b] if k in ("x", "dt", "B", "C", "z") else v for k, v in c.items()}
        cut["init_state"] = state
        rows = {k: None if v is None else v[:, a:b] for k, v in r.items()}
        o, state, _ = rlca.selective_scan(**cut, **rows, want_state=True)
        parts.append(o)
    check("windows", torch.cat(parts, 1), whole.double().cpu())
    check("window state", state, final.double().cpu())
    ended = r["terminated"] | r["truncated"]
    state, steps = c["init_state"].clone(), []
    for t in range(45):
        reset = ended[:, t - 1].contiguous() if t else None
        o, same = rlca.selective_scan_step(c["x"][:, t], c["dt"][:, t], c["A"], c["B"][:, t],
                                           c["C"][:, t], state, D=c["D"], z=c["z"][:, t],
                                           dt_bias=c["dt_bias"], reset=reset)
        assert same is state
        steps.append(o)
    check("steps", torch.stack(steps, 1), whole.double().cpu())
    state[ended[:, -1]] = 0
    check("step state", state, final.double().cpu())


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("N,E,S,G,gate", [(1, 8, 16, 1, True), (5, 130, 16, 2, True),
                                          (3, 33, 5, 1, False), (2, 20, 64, 1, True),
                                          (300, 64, 16, 1, True), (2, 7, 1, 1, True)])
def test_scan_step(cuda_device, dtype, N, E, S, G, gate):
    case = ScanCase(dtype, N, 1, E, S, G, init=True, gate=gate, seed=N + E)
    c, _ = case.args()
    reset = torch.rand(N, generator=_gen(1)) < 0.4
    row = {k: None if c[k] is None else c[k][:, 0] for k in ("x", "dt", "B", "C", "z")}
    state = c["init_state"]
    new = torch.empty_like(state)
    before = state.clone()
    out, got = rlca.selective_scan_step(**row, A=c["A"], D=c["D"], dt_bias=c["dt_bias"],
                                        state=state, reset=reset.cuda(), new_state=new)
    assert got is new and torch.equal(state, before)
    case.v["init_state"] = torch.where(reset[:, None, None], 0.0, case.v["init_state"])
    ro, rf = case.reference()
    check("out", out, ro[:, 0])
    check("state", new, rf)
    out2, same = rlca.selective_scan_step(**row, A=c["A"], D=c["D"], dt_bias=c["dt_bias"],
                                          state=state, reset=reset.cuda())
    assert same is state and torch.equal(state, new) and torch.equal(out, out2)


def test_scan_step_reset_drops_nan_states(cuda_device):
    case = ScanCase(F32, 4, 1, 40, 16, init=True)
    case.v["init_state"][1] = float("nan")
    case.v["init_state"][2] = float("inf")
    c, _ = case.args()
    row = {k: c[k][:, 0] for k in ("x", "dt", "B", "C", "z")}
    reset = torch.tensor([0, 1, 1, 0], dtype=torch.uint8, device="cuda")
    out, _ = rlca.selective_scan_step(**row, A=c["A"], D=c["D"], dt_bias=c["dt_bias"],
                                      state=c["init_state"], reset=reset)
    case.v["init_state"][1:3] = 0
    check("out", out, case.reference()[0][:, 0])


def test_scan_ignores_what_lies_past_a_row_and_before_an_episode(cuda_device):
    """NaN and Inf past the lengths and in an earlier episode change nothing after it."""
    case = ScanCase(F32, 3, 60, 40, 16, seed=9)
    case.rows["lengths"] = torch.tensor([60, 21, 0], dtype=torch.int32)
    term = torch.zeros(3, 60, dtype=torch.bool)
    term[0, 24] = True
    case.rows["terminated"] = term
    ro, rf, rg = case.reference(grads=True)
    for k in ("x", "dt", "B", "C", "z"):
        case.v[k][1, 21:] = float("nan")
        case.v[k][2] = float("inf")
    case.dout[1, 21:] = float("nan")
    case.dout[2] = float("nan")
    out, final, saved = case.forward(want_state=True, want_saved=True)
    check("out", out, ro)
    check("final", final, rf)
    c, r = case.args()
    c.pop("init_state")
    grads = rlca.selective_scan_backward(case.dout.cuda(), saved=saved, **c, **r,
                                         d_final_state=case.d_final.cuda())
    for name, got in zip(("x", "dt", "A", "B", "C", "D", "z", "dt_bias"), grads):
        check("d" + name, got, rg[name])
    # An earlier episode full of NaN.
    case.v["x"][0, :25] = float("nan")
    out2, final2, _ = case.forward(want_state=True)
    assert torch.equal(out2[0, 25:], out[0, 25:]) and torch.equal(final2, final)


def _strided(t, how):
    """The same values at other strides."""
    if t.dim() < 3:
        return t
    if how == "slice":
        wide = torch.zeros(*t.shape[:2], 2, *t.shape[2:], dtype=t.dtype, device=t.device)
        wide[:, :, 1] = t
        return wide[:, :, 1]
    if how == "time_major":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if how == "odd_base":
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)
    return t


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("how", ["slice", "time_major", "odd_base"])
def test_strides_change_nothing(cuda_device, dtype, how):
    case = ScanCase(dtype, 3, 37, 64, 16, flags=True, ragged=True)
    c, r = case.args()
    c.pop("init_state")
    dout = case.dout.cuda()
    base = rlca.selective_scan(**c, **r, want_state=True, want_saved=True)
    bg = rlca.selective_scan_backward(dout, saved=base[2], **c, **r)
    s = {k: v if k in ("A", "D", "dt_bias") else _strided(v, how) for k, v in c.items()}
    outs = {k: _strided(torch.zeros_like(c[k]), how) for k in ("x", "dt", "z", "B", "C")}
    out = _strided(torch.zeros_like(c["x"]), how)
    got = rlca.selective_scan(**s, **r, want_state=True, want_saved=True, out=out)
    gg = rlca.selective_scan_backward(_strided(dout, how), saved=got[2], **s, **r,
                                      dx=outs["x"], ddt=outs["dt"], dz=outs["z"],
                                      dB=outs["B"], dC=outs["C"])
    # Wide and element-wise accesses share the arithmetic but not the order of dD's sums.
    for a, b in zip(got[:2] + gg, base[:2] + bg):
        if a is not None:
            check(how, a, b.double().cpu())
    w, b = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    co, cf = rlca.causal_conv(c["x"], w, b, **r, want_state=True)
    cg = rlca.causal_conv_backward(dout, c["x"], w, b, **r)
    do, df = rlca.causal_conv(s["x"], w, b, **r, want_state=True,
                              out=_strided(torch.zeros_like(c["x"]), how))
    dg = rlca.causal_conv_backward(_strided(dout, how), s["x"], w, b, **r,
                                   dx=_strided(torch.zeros_like(c["x"]), how))
    for a, b in zip((do, df) + dg, (co, cf) + cg):
        check("conv " + how, a, b.double().cpu())


def test_scan_broadcast_rows_and_side_by_side_gradients(cuda_device):
    """B and C shared by all rows (stride 0), dx and dz halves of one gradient."""
    case = ScanCase(F32, 3, 20, 24, 8)
    for k in ("B", "C"):
        case.v[k] = case.v[k][:1].expand(3, -1, -1, -1)
    c, r = case.args()
    c["B"], c["C"] = (c[k][:1].expand(3, -1, -1, -1) for k in ("B", "C"))
    c.pop("init_state")
    out, _, saved = rlca.selective_scan(**c, **r, want_saved=True)
    case.d_final.zero_()
    ro, _, rg = case.reference(grads=True)
    check("out", out, ro)
    dxz = torch.empty(3, 20, 48, device="cuda")
    grads = rlca.selective_scan_backward(case.dout.cuda(), saved=saved, **c, **r,
                                         dx=dxz[..., :24], dz=dxz[..., 24:])
    check("dxz", dxz, torch.cat([rg["x"], rg["z"]], -1))
    check("dB", grads[3], rg["B"])


def test_scan_gradient_against_differences(cuda_device):
    """Directional derivatives of the forward kernel in fp32 against its backward kernel. The
    step's truncation error is of order 1e-6, rounding of the loss of order 1e-7 / 1e-2."""
    case = ScanCase(F32, 2, 24, 20, 16, flags=True, init=True, seed=3)
    c, r = case.args()
    dout, dfin = case.dout.cuda(), case.d_final.cuda()
    out, _, saved = rlca.selective_scan(**c, **r, want_saved=True)
    args = dict(c)
    args.pop("init_state")
    dx, ddt, dA, dB, dC, dD, dz, dbias, dinit = rlca.selective_scan_backward(
        dout, saved=saved, **args, **r, d_final_state=dfin, want_d_init=True)
    grads = dict(x=dx, dt=ddt, A=dA, B=dB, C=dC, D=dD, z=dz, dt_bias=dbias, init_state=dinit)
    g = _gen(7)

    def loss(shift):
        o, f, _ = rlca.selective_scan(**{k: c[k] + shift.get(k, 0) for k in c}, **r,
                                      want_state=True)
        return (o.double() * dout).sum() + (f.double() * dfin).sum()

    for k, grad in grads.items():
        v = torch.randn(c[k].shape, generator=g).cuda()
        want = (grad.double() * v).sum().item()
        eps = 1e-2 / v.norm().item()
        got = (loss({k: eps * v}) - loss({k: -eps * v})).item() / (2 * eps)
        scale = grad.double().norm().item() * v.norm().item()
        assert abs(got - want) <= 1e-3 * scale, f"d{k}: {got} for {want}"


def test_repeated_calls_give_the_same_bits(cuda_device):
    case = ScanCase(BF16, 4, 130, 256, 16, flags=True, ragged=True)
    c, r = case.args()
    c.pop("init_state")
    tokens = torch.randint(0, 50, (4, 130), generator=_gen(2)).cuda()
    w, b = torch.randn(256, 4, device="cuda"), torch.randn(256, device="cuda")
    dout = case.dout.cuda()

    def run():
        f = rlca.selective_scan(**c, **r, want_state=True, want_saved=True)
        g = rlca.selective_scan_backward(dout, saved=f[2], **c, **r)
        k = rlca.causal_conv_backward(dout, c["x"], w, b, **r)
        e = rlca.embed_tokens_backward(dout, tokens, 50)
        return [t for t in (*f[:2], *g, *k, e) if t is not None]

    first = run()
    for _ in range(3):
        for a, b2 in zip(run(), first):
            assert torch.equal(a, b2)


def test_side_stream(cuda_device):
    case = ScanCase(F32, 2, 40, 64, 16)
    want = case.forward()[0]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c, r = case.args()
        got = rlca.selective_scan(**c, **r)[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_graph_capture_of_a_step(cuda_device):
    """One token's work captured once and replayed: the state moves on in place."""
    case = ScanCase(F32, 3, 1, 64, 16, init=True)
    c, _ = case.args()
    row = {k: c[k][:, 0].contiguous() for k in ("x", "dt", "B", "C", "z")}
    kw = dict(**row, A=c["A"], D=c["D"], dt_bias=c["dt_bias"])
    want, state = c["init_state"].clone(), c["init_state"].clone()
    out = torch.empty(3, 64, device="cuda")
    for _ in range(3):
        wo, _ = rlca.selective_scan_step(**kw, state=want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        rlca.selective_scan_step(**kw, state=state, out=out)
    state.copy_(c["init_state"])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, want) and torch.equal(out, wo)


# ----------------------------------------------------------------------------- convolution

CONVS = [
    dict(dtype=F32, N=2, T=40, E=24, K=4),
    dict(dtype=BF16, N=2, T=70, E=264, K=4, flags=True),
    dict(dtype=FP16, N=3, T=37, E=129, K=3, flags=True, ragged=True, init=True),
    dict(dtype=F32, N=3, T=33, E=65, K=2, flags=True, ragged=True, init=True),
    dict(dtype=F32, N=2, T=31, E=8, K=1, flags=True),
    dict(dtype=BF16, N=2, T=32, E=16, K=8, init=True),
    dict(dtype=F32, N=2, T=200, E=20, K=5, flags=True, silu=False),
    dict(dtype=F32, N=4, T=1, E=12, K=4, flags=True, init=True),
    dict(dtype=F32, N=3, T=2, E=12, K=4, init=True, ragged=True),
    dict(dtype=F32, N=2, T=129, E=4, K=4, init=True, bias=False),
    dict(dtype=FP16, N=5, T=300, E=40, K=4, flags=True, ragged=True, init=True),
]


@pytest.mark.parametrize("cfg", CONVS, ids=_id)
def test_conv_forward_and_backward(cuda_device, cfg):
    cfg = dict(cfg)
    dtype, N, T, E, K = (cfg[k] for k in ("dtype", "N", "T", "E", "K"))
    g = _gen(11)
    rn = lambda *s: torch.randn(*s, generator=g)
    x, dout = rn(N, T, E).to(dtype), rn(N, T, E).to(dtype)
    w = rn(E, K) / math.sqrt(K)
    b = rn(E) if cfg.get("bias", True) else None
    init = rn(N, K - 1, E).to(dtype) if cfg.get("init") else None
    rows = dict(terminated=_flags(N, T, g) if cfg.get("flags") else None,
                truncated=_flags(N, T, g, 0.05) if cfg.get("flags") else None,
                lengths=_lengths(N, T, g) if cfg.get("ragged") else None)
    silu = cfg.get("silu", True)
    cu = lambda t: None if t is None else t.cuda()
    r = {k: cu(v) for k, v in rows.items()}
    out, final = rlca.causal_conv(cu(x), cu(w), cu(b), **r, init_state=cu(init), silu=silu,
                                  want_state=True)
    dx, dw, db = rlca.causal_conv_backward(cu(dout), cu(x), cu(w), cu(b), **r,
                                           init_state=cu(init), silu=silu)
    x6, w6 = x.double().requires_grad_(), w.double().requires_grad_()
    b6 = None if b is None else b.double().requires_grad_()
    ro, rf = ref.conv(x6, w6, b6, **rows, init_state=None if init is None else init.double(),
                      silu=silu)
    ro.backward(dout.double())
    check("out", out, ro)
    check("final", final, rf)
    check("dx", dx, x6.grad)
    check("dw", dw, w6.grad)
    if b is None:
        assert db is None
    else:
        check("db", db, b6.grad)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("N,E,K", [(1, 8, 4), (5, 131, 3), (300, 64, 4), (3, 16, 1), (2, 24, 8)])
def test_conv_step(cuda_device, dtype, N, E, K):
    g = _gen(N + E)
    rn = lambda *s: torch.randn(*s, generator=g)
    x, state = rn(N, 2 * E).to(dtype)[:, :E], rn(N, K - 1, E).to(dtype)
    w, b = rn(E, K), rn(E)
    reset = torch.rand(N, generator=g) < 0.4
    if N > 1:
        state[1] = float("nan")
        reset[1] = True
    args = (x.cuda(), state.cuda(), w.cuda(), b.cuda())
    new = torch.empty_like(args[1])
    out, got = rlca.causal_conv_step(*args, reset=reset.cuda(), new_state=new)
    assert got is new
    kept = torch.where(reset[:, None, None], torch.zeros((), dtype=dtype), state)
    ro, rf = ref.conv(x.double()[:, None], w.double(), b.double(), init_state=kept.double())
    check("out", out, ro[:, 0])
    assert torch.equal(new.double().cpu(), rf)
    out2, same = rlca.causal_conv_step(*args, reset=reset.cuda())
    assert same is args[1] and torch.equal(same, new) and torch.equal(out2, out)


def test_conv_windows_and_steps_continue_one_another(cuda_device):
    g = _gen(21)
    x = torch.randn(3, 50, 40, generator=g).cuda()
    w, b = torch.randn(40, 4, generator=g).cuda(), torch.randn(40, generator=g).cuda()
    term = _flags(3, 50, g).cuda()
    whole, final = rlca.causal_conv(x, w, b, terminated=term, want_state=True)
    state, parts = None, []
    for a, e in ((0, 2), (2, 33), (33, 50)):
        o, state = rlca.causal_conv(x[:, a:e], w, b, terminated=term[:, a:e], init_state=state,
                                    want_state=True)
        parts.append(o)
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, final)
    state = torch.zeros(3, 3, 40, device="cuda")
    for t in range(50):
        o, _ = rlca.causal_conv_step(x[:, t], state, w, b,
                                     reset=term[:, t - 1].contiguous() if t else None)
        assert torch.equal(o, whole[:, t])


def test_conv_ignores_masked_inputs(cuda_device):
    g = _gen(22)
    x, dout = torch.randn(2, 40, 16, generator=g), torch.randn(2, 40, 16, generator=g)
    w, b = torch.randn(16, 4, generator=g), torch.randn(16, generator=g)
    term = torch.zeros(2, 40, dtype=torch.bool)
    term[0, 9] = True
    lengths = torch.tensor([40, 13], dtype=torch.int32)
    cu = lambda: (x.cuda(), w.cuda(), b.cuda(), term.cuda(), None, lengths.cuda())
    out, _ = rlca.causal_conv(*cu())
    dx, dw, db = rlca.causal_conv_backward(dout.cuda(), *cu())
    x[1, 13:] = float("nan")
    dout[1, 13:] = float("inf")
    out2, _ = rlca.causal_conv(*cu())
    for a, c in zip(rlca.causal_conv_backward(dout.cuda(), *cu()), (dx, dw, db)):
        assert torch.equal(a, c)
    assert torch.equal(out2, out)
    x[0, :10] = float("nan")
    out3, _ = rlca.causal_conv(*cu())
    dx3 = rlca.causal_conv_backward(dout.cuda(), *cu())[0]
    assert torch.equal(out3[0, 10:], out[0, 10:]) and torch.equal(dx3[0, 10:], dx[0, 10:])


def test_conv_without_rows_or_steps(cuda_device):
    w, b = torch.randn(16, 4, device="cuda"), torch.randn(16, device="cuda")
    init = torch.randn(2, 3, 16, device="cuda")
    x = torch.empty(2, 0, 16, device="cuda")
    out, final = rlca.causal_conv(x, w, b, init_state=init, want_state=True)
    assert out.numel() == 0 and torch.equal(final, init)
    dx, dw, db = rlca.causal_conv_backward(x, x, w, b)
    assert not dw.any() and not db.any()
    none = torch.empty(0, 5, 16, device="cuda")
    dx, dw, db = rlca.causal_conv_backward(none, none, w, b)
    assert not dw.any() and not db.any()


# ------------------------------------------------------------------------------- embedding

def _token_sets(V, M, g):
    return {
        "uniform": torch.randint(0, V, (M,), generator=g),
        "one": torch.full((M,), V - 1),
        "padding": torch.full((M,), -1),
        "mixed": torch.randint(-2, V + 3, (M,), generator=g),
        "skewed": (torch.rand(M, generator=g) ** 6 * V).long(),
    }


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("V,D", [(1, 8), (50, 33), (300, 64), (70000, 16)])
@pytest.mark.parametrize("M", [1, 31, 32, 33, 700, 5000])
def test_embedding(cuda_device, dtype, V, D, M):
    g = _gen(V + M)
    table = torch.randn(V, D, generator=g).to(dtype)
    dout = torch.randn(M, D, generator=g).to(dtype)
    for i, (name, tokens) in enumerate(_token_sets(V, M, g).items()):
        tok = tokens.to(torch.int32 if i % 2 else torch.int64).cuda()
        out = rlca.embed_tokens(tok, table.cuda(), scale=3.0)
        inside = (tokens >= 0) & (tokens < V)
        want = torch.where(inside[:, None], table.double()[tokens.clamp(0, V - 1)] * 3.0, 0.0)
        check(f"{name} rows", out, want)
        grad = rlca.embed_tokens_backward(dout.cuda(), tok, V, scale=0.5)
        want = torch.zeros(V, D, dtype=torch.float64)
        want.index_add_(0, tokens[inside], dout.double()[inside] * 0.5)
        check(f"{name} gradient", grad, want)


def test_embedding_of_many_tokens(cuda_device):
    """More tokens than the sort takes in one sweep of its CTAs, a frequent one among them."""
    g = _gen(4)
    V, D, M = 40000, 24, 70001
    tokens = torch.where(torch.rand(M, generator=g) < 0.3, 7, torch.randint(-1, V, (M,),
                                                                            generator=g))
    dout = torch.randn(M, D, generator=g)
    grad = rlca.embed_tokens_backward(dout.cuda(), tokens.cuda(), V)
    want = torch.zeros(V + 1, D, dtype=torch.float64)
    want.index_add_(0, torch.where(tokens < 0, V, tokens), dout.double())
    check("gradient", grad, want[:V])


def test_embedding_strides_and_empty(cuda_device):
    table = torch.randn(30, 40, device="cuda")
    tokens = torch.randint(0, 30, (3, 7), device="cuda")
    wide = torch.zeros(3, 7, 80, device="cuda")
    out = rlca.embed_tokens(tokens, table[:, 8:24], out=wide[..., 33:49])
    assert out.data_ptr() == wide[..., 33:49].data_ptr()
    assert torch.equal(wide[..., 33:49], table[tokens][..., 8:24])
    assert not wide[..., :33].any() and not wide[..., 49:].any()
    a = rlca.embed_tokens_backward(wide[..., 33:49], tokens, 30)
    b = rlca.embed_tokens_backward(wide[..., 33:49].contiguous(), tokens, 30)
    check("strided", a, b.double().cpu())
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert rlca.embed_tokens(none, table).shape == (0, 40)
    grad = rlca.embed_tokens_backward(torch.empty(0, 40, device="cuda"), none, 30)
    assert grad.shape == (30, 40) and not grad.any()


def test_embedding_gradient_ignores_padded_rows(cuda_device):
    tokens = torch.tensor([3, -1, 3, 99, 0], device="cuda")
    dout = torch.ones(5, 8, device="cuda")
    dout[1], dout[3] = float("nan"), float("inf")
    grad = rlca.embed_tokens_backward(dout, tokens, 5)
    want = torch.zeros(5, 8, dtype=torch.float64)
    want[3], want[0] = 2, 1
    check("gradient", grad, want)


# -------------------------------------------------------------------- offsets past 32 bits

def test_offsets_past_32_bits(cuda_device):
    """Rows that lie more than 2^31 elements apart, and table rows past 2^31 elements."""
    far = (1 << 31) + 64
    big = torch.zeros(far + 40 * 64, dtype=BF16, device="cuda")
    case = ScanCase(BF16, 2, 40, 64, 16, flags=True)
    c, r = case.args()
    c.pop("init_state")
    dout = case.dout.cuda()
    view = big.as_strided((2, 40, 64), (far, 64, 1))
    view.copy_(c["x"])
    base = rlca.selective_scan(**c, **r, want_saved=True)
    bg = rlca.selective_scan_backward(dout, saved=base[2], **c, **r)
    moved = dict(c, x=view)
    got = rlca.selective_scan(**moved, **r)
    assert torch.equal(got[0], base[0])
    gg = rlca.selective_scan_backward(dout, saved=base[2], **moved, **r)
    assert torch.equal(gg[0], bg[0]) and torch.equal(gg[2], bg[2])
    w, b = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    assert torch.equal(rlca.causal_conv(view, w, b, **r)[0],
                       rlca.causal_conv(c["x"], w, b, **r)[0])
    for a, e in zip(rlca.causal_conv_backward(dout, view, w, b, **r),
                    rlca.causal_conv_backward(dout, c["x"], w, b, **r)):
        assert torch.equal(a, e)
    V = far // 64
    table = big[:V * 64].view(V, 64)
    tokens = torch.tensor([0, V - 1, V - 2, V], device="cuda")
    table[V - 1], table[V - 2] = 5.0, 7.0
    out = rlca.embed_tokens(tokens, table).float().cpu()
    assert (out[1] == 5).all() and (out[2] == 7).all() and not out[3].any()
    del big, view, table, moved
    torch.cuda.empty_cache()
    # States past 2^31 elements.
    N, E, S = 1030, 131072, 16
    assert N * E * S > 1 << 31
    state = torch.full((N, E, S), 2.0, device="cuda")
    x = torch.ones(1, E, device="cuda").expand(N, E)
    bc = torch.ones(1, S, device="cuda").expand(N, S)
    dt = torch.zeros(1, E, device="cuda").expand(N, E)
    A = torch.zeros(E, S, device="cuda")
    out, _ = rlca.selective_scan_step(x, dt, A, bc, bc, state, dt_softplus=False)
    assert (out == 2.0 * S).all() and state[-1, -1, -1] == 2.0
    del state, out
    torch.cuda.empty_cache()


# --------------------------------------------------------------- borders between variants

@pytest.mark.parametrize("K", [5, 6, 7, 8])
def test_conv_with_many_taps(cuda_device, K):
    g = _gen(K)
    x, dout = torch.randn(2, 75, 37, generator=g), torch.randn(2, 75, 37, generator=g)
    w, b = torch.randn(37, K, generator=g) / K, torch.randn(37, generator=g)
    init = torch.randn(2, K - 1, 37, generator=g)
    term = _flags(2, 75, g)
    out, final = rlca.causal_conv(x.cuda(), w.cuda(), b.cuda(), term.cuda(),
                                  init_state=init.cuda(), want_state=True)
    dx, dw, db = rlca.causal_conv_backward(dout.cuda(), x.cuda(), w.cuda(), b.cuda(), term.cuda(),
                                           init_state=init.cuda())
    x6, w6, b6 = (v.double().requires_grad_() for v in (x, w, b))
    ro, rf = ref.conv(x6, w6, b6, term, init_state=init.double())
    ro.backward(dout.double())
    for name, got, want in (("out", out, ro), ("final", final, rf), ("dx", dx, x6.grad),
                            ("dw", dw, w6.grad), ("db", db, b6.grad)):
        check(name, got, want)


@pytest.mark.parametrize("M", [2047, 2048, 2049, 4096, 65535, 65536, 65537, 131073])
@pytest.mark.parametrize("V", [255, 256, 65536])
def test_embedding_gradient_at_the_sorts_borders(cuda_device, M, V):
    """One CTA or the cluster, one sweep or several, one pass of 8 bits or two or three."""
    g = _gen(M + V)
    tokens = torch.randint(-1, V + 1, (M,), generator=g)
    dout = torch.randn(M, 4, generator=g)
    grad = rlca.embed_tokens_backward(dout.cuda(), tokens.cuda(), V)
    want = torch.zeros(V + 1, 4, dtype=torch.float64)
    want.index_add_(0, torch.where(tokens < 0, V, tokens), dout.double())
    check("gradient", grad, want[:V])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_an_episode_in_a_later_span_sees_nothing_before_it(cuda_device, dtype):
    """A long row cut into spans: NaN in an earlier episode reaches no output, state or
    gradient of the next one, and no later dout reaches the steps before it."""
    case = ScanCase(dtype, 1, 400, 64, 16, seed=31)
    term = torch.zeros(1, 400, dtype=torch.bool)
    term[0, 149] = True
    case.rows["terminated"] = term
    dout = case.dout.cuda()

    def run():
        out, final, saved = case.forward(want_state=True, want_saved=True)
        c, r = case.args()
        c.pop("init_state")
        return out, final, rlca.selective_scan_backward(dout, saved=saved, **c, **r)

    out, final, grads = run()
    case.v["x"][0, :150] = float("nan")
    out2, final2, grads2 = run()
    assert torch.equal(out2[0, 150:], out[0, 150:]) and torch.equal(final2, final)
    for k in (0, 1, 3, 4, 6):
        assert torch.equal(grads2[k][0, 150:], grads[k][0, 150:])
    case.v["x"][0, :150] = 0.5
    out, final, grads = run()
    dout[0, 150:] = float("nan")
    _, _, grads2 = run()
    for k in (0, 1, 3, 4, 6):
        assert torch.equal(grads2[k][0, :150], grads[k][0, :150])


@pytest.mark.parametrize("N,E", [(300, 2048), (153, 1024), (608, 64), (913, 64)])
def test_scan_backward_variants_agree(cuda_device, N, E):
    """Grids of few, many and very many CTAs take other register cuts: a row's gradients are
    the same in all of them, bit for bit."""
    case = ScanCase(BF16, N, 16, E, 16, flags=True, seed=N)
    c, r = case.args()
    c.pop("init_state")
    dout = case.dout.cuda()
    _, _, saved = rlca.selective_scan(**c, **r, want_saved=True)
    many = rlca.selective_scan_backward(dout, saved=saved, **c, **r)
    one = {k: v if k in ("A", "D", "dt_bias") else v[5:6] for k, v in c.items()}
    rows = {k: None if v is None else v[5:6] for k, v in r.items()}
    few = rlca.selective_scan_backward(dout[5:6], saved=saved[5:6].contiguous(), **one, **rows)
    for k in (0, 1, 3, 4, 6):
        assert torch.equal(many[k][5:6], few[k])


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
def test_scan_of_one_step_of_a_wider_buffer(cuda_device, dtype):
    """Windows of one step, channels cut out of odd rows: the step's stride is nobody's."""
    case = ScanCase(dtype, 4, 1, 64, 16, flags=True, init=True, seed=41)
    c, r = case.args()

    def cut(t):
        base = torch.zeros(4, 8, 67, dtype=dtype, device="cuda")
        base[:, :1, :64] = t
        return base[:, :1, :64]

    # Rows lie 8 x 67 elements apart: a multiple of 8, unlike the stride of the steps.
    for k in ("x", "dt", "z"):
        c[k] = cut(c[k])
    assert c["x"].stride() == (536, 67, 1)
    out, final, saved = rlca.selective_scan(**c, **r, want_state=True, want_saved=True,
                                            out=cut(torch.zeros_like(c["x"])))
    ro, rf, rg = case.reference(grads=True)
    check("out", out, ro)
    check("final", final, rf)
    c.pop("init_state")
    d = {k: cut(torch.zeros_like(c["x"])) for k in ("dx", "ddt", "dz")}
    grads = rlca.selective_scan_backward(cut(case.dout.cuda()), saved=saved, **c, **r, **d,
                                         d_final_state=case.d_final.cuda(), want_d_init=True)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init_state")
    for name, got in zip(names, grads):
        check("d" + name, got, rg[name], dtype if got.dtype == dtype else F32)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("S", [5, 16])
def test_steps_leave_the_windows_states_bit_for_bit(cuda_device, dtype, S):
    """A window that is not cut into spans (fewer than 128 steps) and its tokens one by one do
    the same operations on a state in the same order: no tolerance. Small step sizes, whose
    decays' errors add up over all of the window."""
    T = 120
    case = ScanCase(dtype, 3, T, 40, S, flags=True, init=True, seed=43)
    case.v["dt_bias"] -= 4.0
    c, r = case.args()
    _, final, _ = rlca.selective_scan(**c, **r, want_state=True)
    ended = r["terminated"] | r["truncated"]
    state = c["init_state"].clone()
    for t in range(T):
        reset = ended[:, t - 1].contiguous() if t else None
        rlca.selective_scan_step(c["x"][:, t], c["dt"][:, t], c["A"], c["B"][:, t], c["C"][:, t],
                                 state, D=c["D"], z=c["z"][:, t], dt_bias=c["dt_bias"],
                                 reset=reset)
    state[ended[:, -1]] = 0
    assert torch.equal(state, final)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("steps", [True, False])
def test_decays_have_no_bias_that_adds_up(cuda_device, dtype, steps):
    """500 tokens at a step size near 0.01 and no input: a decay that is off by e on average leaves
    the state off by 500 e. CUDA's expf is off by up to 1.5e-8 on average (measured over -0.5..0):
    no more is allowed. Roundings that add up at random do not show in the mean over 2048 states
    (1e-8); the step size is exact."""
    N, E, S, T = 2, 64, 16, 500
    g = _gen(47)
    A = -(0.7 + 0.7 * torch.rand(E, S, generator=g))
    start = 1 + torch.rand(N, E, S, generator=g)
    dt = torch.full((N, T, E), 0.01).to(dtype)
    x, bc = torch.zeros_like(dt).cuda(), torch.zeros(N, T, S).to(dtype).cuda()
    want = start.double() * torch.exp(T * dt[0, 0, 0].double() * A.double())
    if steps:
        state = start.cuda()
        args = (x[:, 0], dt[:, 0].cuda(), A.cuda(), bc[:, 0], bc[:, 0], state)
        for _ in range(T):
            rlca.selective_scan_step(*args, dt_softplus=False)
    else:
        _, state, _ = rlca.selective_scan(x, dt.cuda(), A.cuda(), bc, bc, init_state=start.cuda(),
                                          dt_softplus=False, want_state=True)
    off = (state.double().cpu() / want - 1).mean().abs().item()
    assert off <= 1.5e-8 * T, off


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,T", [(5, 37), (2, 300)])
def test_states_without_memory(cuda_device, dtype, N, T):
    """A = -inf is a decay of 0, a state that holds the last input only: the steps past a row (the
    rest of a tile, whole spans of a long window) leave it as it is."""
    case = ScanCase(dtype, N, T, 40, 16, ragged=True, init=True, seed=51)
    case.rows["lengths"] = torch.tensor([T, 0, 1, 18, 30][:N], dtype=torch.int32)
    if N == 2:
        case.rows["lengths"][0] = 130
    case.v["A"][:, 3] = -float("inf")
    out, final, _ = case.forward(want_state=True)
    ro, rf = case.reference()
    check("out", out, ro)
    check("final", final, rf)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,T", [(5, 37), (2, 300)])
def test_gradients_of_states_without_memory(cuda_device, dtype, N, T):
    """A = -inf and a rate that no step size of the data survives give the same bits: the limit,
    where A exp(d A) by itself would be NaN."""
    case = ScanCase(dtype, N, T, 40, 16, ragged=True, init=True, seed=51)
    dout, d_final = case.dout.cuda(), case.d_final.cuda()

    def run(rate):
        case.v["A"][:, 3] = rate
        _, _, saved = case.forward(want_saved=True)
        c, r = case.args()
        c.pop("init_state")
        return rlca.selective_scan_backward(dout, saved=saved, **c, **r, d_final_state=d_final,
                                            want_d_init=True)

    for a, b in zip(run(-float("inf")), run(-1e30)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_a_span_passes_nothing_on_where_nothing_comes_in(cuda_device):
    """States that grow by exp(3.5) a step and hold 0 until the last step, over a window that is
    cut into spans of 32 steps: exp of a span's sum of exponents is Inf, times 0."""
    N, T, E, S = 1, 1024, 16, 16
    dt = torch.full((N, T, E), 3.5, device="cuda")
    x = torch.zeros(N, T, E, device="cuda")
    x[:, -1] = 2.0
    b = torch.ones(N, T, S, device="cuda")
    A = torch.ones(E, S, device="cuda")
    out, final, _ = rlca.selective_scan(x, dt, A, b, b, dt_softplus=False, want_state=True)
    assert (out[:, :-1] == 0).all() and (out[:, -1] == 7.0 * S).all()
    assert (final == 7.0).all()


# Spans at every number of lanes to a channel: 1 (S <= 8), 2, 4 and 8 (S > 32) forward, twice that
# backward. Windows this long on so few channels are cut into spans of 32 steps.
@pytest.mark.parametrize("dtype,S,G,gate,E", [
    (F32, 1, 1, True, 24), (BF16, 4, 1, False, 24), (FP16, 8, 2, True, 34), (F32, 7, 1, False, 9),
    (BF16, 17, 1, True, 24), (F32, 24, 3, False, 12), (FP16, 32, 1, True, 19),
    (F32, 33, 1, True, 9), (BF16, 64, 1, False, 16), (FP16, 48, 2, True, 10),
])
@pytest.mark.parametrize("ragged", [False, True])
def test_spans_at_every_state_size(cuda_device, dtype, S, G, gate, E, ragged):
    test_scan_forward_and_backward(
        cuda_device, dict(dtype=dtype, N=2, T=231, E=E, S=S, G=G, gate=gate, flags=ragged,
                          ragged=ragged, init=True, seed=S))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S", [4, 16, 33])
def test_a_row_cut_into_spans_is_the_row_walked_whole(cuda_device, dtype, S):
    """A row beside enough others is walked in one piece, alone in spans: states that leave a span
    are joined through exp(A sum d), a rounding of the exponent in place of the decays' own."""
    T, E, many = 192, 64, 2600
    case = ScanCase(dtype, 1, T, E, S, flags=True, init=True, seed=61)
    c, r = case.args()
    dout, d_final = case.dout.cuda(), case.d_final.cuda()
    rows = lambda t, n: t.expand(n, *t.shape[1:]).contiguous()

    def run(n):
        v = {k: t if k in ("A", "D", "dt_bias") else rows(t, n) for k, t in c.items()}
        f = {k: None if t is None else rows(t, n) for k, t in r.items()}
        out, final, saved = rlca.selective_scan(**v, **f, want_state=True, want_saved=True)
        v.pop("init_state")
        g = rlca.selective_scan_backward(rows(dout, n), saved=saved, **v, **f, want_d_init=True,
                                         d_final_state=rows(d_final, n))
        return [t[:1] for t in (out, final, g[0], g[1], g[3], g[4], g[6], g[8])]

    for name, a, b in zip(("out", "final", "dx", "ddt", "dB", "dC", "dz", "d_init"), run(1),
                          run(many)):
        check(name, a, b.double().cpu())


@pytest.mark.parametrize("dtype,S,per_row", [(F32, 8, 32), (F32, 16, 64), (F32, 64, 256),
                                             (BF16, 8, 32), (BF16, 64, 256)])
@pytest.mark.parametrize("ctas", [1024, 1280])
def test_scan_backward_variants_agree_in_every_form(cuda_device, dtype, S, per_row, ctas):
    """On both sides of one wave of the CTAs that shared memory lets in, against one row alone: the
    same bits."""
    N = ctas // per_row
    case = ScanCase(dtype, N, 16, 2048, S, flags=True, seed=S)
    c, r = case.args()
    c.pop("init_state")
    dout = case.dout.cuda()
    _, _, saved = rlca.selective_scan(**c, **r, want_saved=True)
    many = rlca.selective_scan_backward(dout, saved=saved, **c, **r)
    one = {k: v if k in ("A", "D", "dt_bias") else v[2:3] for k, v in c.items()}
    rows = {k: None if v is None else v[2:3] for k, v in r.items()}
    few = rlca.selective_scan_backward(dout[2:3], saved=saved[2:3].contiguous(), **one, **rows)
    for k in (0, 1, 3, 4, 6):
        assert torch.equal(many[k][2:3], few[k])
