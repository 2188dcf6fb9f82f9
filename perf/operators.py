"""The sequence-model operators of the framework as measurable cases: a segmented selective
state space scan, the short causal convolution in front of it, and the token embedding,
each in its plain form (elementary torch operations in 32 bits) and through the
framework's entry points, with a 64-bit definition to compare both with.

Rows are environments (or prompts), steps are tokens, `start` marks a step whose previous
step ended an episode: neither the state nor the convolution's window crosses it.
"""
import math

import torch

own = False

_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


def _scan(name, op, N, T, E, S, dtype, G=1, gate=True, flags=False, ragged=False, init=False):
    return dict(name=name, op=op, N=N, T=T, E=E, S=S, G=G, dtype=dtype, gate=gate,
                flags=flags, ragged=ragged, init=init)


def _conv(name, op, N, T, E, K, dtype, flags=False, ragged=False, init=False):
    return dict(name=name, op=op, N=N, T=T, E=E, K=K, dtype=dtype, flags=flags,
                ragged=ragged, init=init)


def _embed(name, op, N, T, V, D, dtype):
    return dict(name=name, op=op, N=N, T=T, V=V, D=D, dtype=dtype)


def listed():
    return [
        # One long prompt read into a state: few channels in all, a long axis.
        _scan("scan_prompt_1x8192", "scan", 1, 8192, 2048, 16, "bf16"),
        # A batch of prompts of unlike lengths (one of them empty) continued from earlier
        # states, episodes ending inside, a channel count that is no multiple of anything.
        _scan("scan_prompt_ragged", "scan", 33, 517, 1027, 16, "fp16", flags=True,
              ragged=True, init=True),
        # A training window: forward and all gradients, with episode ends.
        _scan("scan_train_16x1024", "scan_train", 16, 1024, 2048, 16, "bf16", flags=True),
        # A small model in fp32 without the gate: two groups, an odd state size, a
        # learned initial state.
        _scan("scan_train_odd", "scan_train", 7, 300, 518, 10, "fp32", G=2, gate=False,
              flags=True, ragged=True, init=True),
        # Acting: one token for each of a few environments; latency counts.
        _scan("scan_step_16", "scan_step", 16, 1, 1024, 16, "bf16", flags=True),
        # Acting in 4096 environments at once: the states are the traffic.
        _scan("scan_step_4096", "scan_step", 4096, 1, 1024, 16, "bf16", flags=True),
        # The convolution of the same training window, forward and gradients.
        _conv("conv_train_16x1024", "conv_train", 16, 1024, 2048, 4, "bf16", flags=True),
        # A small model in fp32: three taps, odd sizes, a window carried in.
        _conv("conv_train_odd", "conv_train", 5, 333, 1001, 3, "fp32", flags=True,
              ragged=True, init=True),
        # Acting: one token for each of 256 environments.
        _conv("conv_step_256", "conv_step", 256, 1, 2048, 4, "fp16", flags=True),
        # The embedding rows of a batch of token windows.
        _embed("embed_16x1024", "embed", 16, 1024, 32768, 1024, "bf16"),
        # The table's gradient for a large batch: few frequent tokens, many rare ones.
        _embed("embed_grad_64x1024", "embed_grad", 64, 1024, 50000, 1024, "bf16"),
        # The gradient of a small table of discrete observations.
        _embed("embed_grad_16x128", "embed_grad", 16, 128, 512, 64, "fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["scan", "scan_train", "scan_step", "conv_train", "conv_step", "embed",
                     "embed_grad"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    flags, ragged, init = (rng.random() < 0.5 for _ in range(3))
    if op in ("scan", "scan_train"):
        G = rng.choice([1, 1, 2])
        E = G * _log(rng, 64 // G, 2048 // G)
        S = rng.choice([16, 16, 8, 13, 32])
        T = _log(rng, 1, 8192 if op == "scan" else 1024)
        top = 33 if op == "scan" else 16
        N = min(_log(rng, 1, 64), max(1, top * 524288 // (T * E * max(1, S // 16))))
        return dict(op=op, N=N, T=T, E=E, S=S, G=G, dtype=dtype, gate=rng.random() < 0.75,
                    flags=flags, ragged=ragged, init=init)
    if op == "scan_step":
        E = _log(rng, 64, 2048)
        N = min(_log(rng, 1, 4096), 4194304 // E)
        return dict(op=op, N=N, T=1, E=E, S=rng.choice([16, 16, 8, 13]), G=1, dtype=dtype,
                    gate=rng.random() < 0.75, flags=flags, ragged=False, init=False)
    if op == "conv_train":
        E = _log(rng, 64, 2048)
        T = _log(rng, 1, 8192)
        N = min(_log(rng, 1, 64), max(1, 16777216 // (T * E)))
        return dict(op=op, N=N, T=T, E=E, K=rng.choice([4, 4, 3, 2]), dtype=dtype,
                    flags=flags, ragged=ragged, init=init)
    if op == "conv_step":
        return dict(op=op, N=_log(rng, 1, 4096), T=1, E=_log(rng, 64, 2048),
                    K=rng.choice([4, 4, 3, 2]), dtype=dtype, flags=flags, ragged=False,
                    init=False)
    T = _log(rng, 1, 1024)
    return dict(op=op, N=_log(rng, 1, 64), T=T, V=_log(rng, 16, 50000),
                D=_log(rng, 32, 1024), dtype=dtype)


# ------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    op, N, T = case["op"], case["N"], case["T"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device=dev, generator=gen) * std

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen)

    s = {"case": case}
    if op.startswith("embed"):
        V, D = case["V"], case["D"]
        # Token frequencies fall as one over their rank; a few steps hold padding (-1).
        tokens = (float(V) ** uniform(N, T)).long().clamp_(1, V) - 1
        s["tokens"] = torch.where(uniform(N, T) < 0.02, -1, tokens)
        s["scale"] = math.sqrt(D)
        if op == "embed":
            s["table"] = normal(V, D, std=0.02).to(dt)
        else:
            s["dout"] = normal(N, T, D, std=0.1).to(dt)
        return s

    # Episode ends and truncations of a rollout; `reset` is their form for one token.
    for k in ("terminated", "truncated", "lengths", "init", "reset"):
        s[k] = None
    if op.endswith("_step"):
        if case["flags"]:
            s["reset"] = uniform(N) < 0.05
    else:
        if case["flags"]:
            s["terminated"] = uniform(N, T) < 1 / 128
            s["truncated"] = uniform(N, T) < 1 / 256
        if case["ragged"]:
            lengths = (uniform(N) * (T + 1)).int().clamp_(0, T)
            lengths[0] = T
            if N > 2:
                lengths[N // 2] = 0
            s["lengths"] = lengths
    E = case["E"]
    if op.startswith("conv"):
        K = case["K"]
        # The input projection gives the convolution's half and the gate's half side by
        # side, so the rows of x are strided.
        if op == "conv_step":
            s["x"] = normal(N, 2 * E).to(dt)[:, :E]
            s["state"] = normal(N, K - 1, E).to(dt)
            s["new_state"] = torch.empty_like(s["state"])
        else:
            s["x"] = normal(N, T, 2 * E).to(dt)[..., :E]
            s["dout"] = normal(N, T, E).to(dt)
            if case["init"]:
                s["init"] = normal(N, K - 1, E).to(dt)
        s["weight"] = (uniform(E, K) * 2 - 1) / math.sqrt(K)
        s["bias"] = normal(E, std=0.1)
        return s

    S, G = case["S"], case["G"]
    lead = (N,) if op == "scan_step" else (N, T)
    s["x"] = torch.nn.functional.silu(normal(*lead, E)).to(dt)
    s["z"] = normal(*lead, 2 * E).to(dt)[..., E:] if case["gate"] else None
    s["dt"] = normal(*lead, E, std=0.5).to(dt)
    bc = normal(*lead, 2, G, S).to(dt)  # one projection gives B and C side by side
    s["B"], s["C"] = bc.select(-3, 0), bc.select(-3, 1)
    s["A"] = -torch.arange(1, S + 1, device=dev, dtype=torch.float32).expand(E, S) \
        * (1 + 0.1 * uniform(E, S))
    s["D"] = 1 + normal(E, std=0.1)
    # Step sizes start log-uniform in [0.001, 0.1] behind the softplus.
    step = torch.exp(uniform(E) * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    if op == "scan_step":
        s["state"] = normal(N, E, S)
        s["new_state"] = torch.empty_like(s["state"])
    elif case["init"]:
        s["init"] = normal(N, E, S)
    if op == "scan_train":
        s["dout"] = normal(N, T, E).to(dt)
    return s


# --------------------------------------------------------------------------- plain form


def _starts(s, N, T):
    """Steps whose previous step ended an episode, and steps inside the row's length."""
    dev = s["x"].device
    start = torch.zeros(N, T, dtype=torch.bool, device=dev)
    ended = torch.zeros(N, T, dtype=torch.bool, device=dev)
    if s["terminated"] is not None:
        ended = s["terminated"] | s["truncated"]
        start[:, 1:] = ended[:, :-1]
    valid = torch.ones(N, T, dtype=torch.bool, device=dev)
    if s["lengths"] is not None:
        valid = torch.arange(T, device=dev) < s["lengths"][:, None]
    return start & valid, ended & valid, valid


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_scan(s, train):
    c = s["case"]
    N, T, E, S, G = c["N"], c["T"], c["E"], c["S"], c["G"]
    g4 = (N, G, E // G, S)
    start, ended, valid = _starts(s, N, T)
    x = s["x"].float()
    raw = s["dt"].float() + s["dt_bias"]
    d = _softplus(raw)
    A = s["A"].view(1, G, E // G, S)
    h = torch.zeros(g4, device=x.device) if s["init"] is None else s["init"].reshape(g4)
    segments, partial = s["terminated"] is not None, s["lengths"] is not None
    dx_, d_ = (d * x).view(N, T, G, E // G, 1), d.view(N, T, G, E // G, 1)
    B, C = s["B"].float(), s["C"].float()
    y = torch.empty(N, T, E, device=x.device)
    before = []
    zero = torch.zeros((), device=x.device)
    for t in range(T):
        if segments:
            h = torch.where(start[:, t].view(N, 1, 1, 1), zero, h)
        if train:
            before.append(h)
        new = torch.exp(d_[:, t] * A) * h + dx_[:, t] * B[:, t].unsqueeze(2)
        y[:, t] = (new * C[:, t].unsqueeze(2)).sum(-1).view(N, E)
        h = torch.where(valid[:, t].view(N, 1, 1, 1), new, h) if partial else new
    y = y + s["D"] * x
    z = None if s["z"] is None else s["z"].float()
    out = y if z is None else y * z * _sigmoid(z)
    if partial:
        out = torch.where(valid[..., None], out, zero)
    if segments:
        last = valid.sum(1) - 1
        done = (last >= 0) & ended.gather(1, last.clamp(min=0)[:, None])[:, 0]
        h = torch.where(done.view(N, 1, 1, 1), zero, h)
    dtype = s["x"].dtype
    out, final = out.to(dtype), h.reshape(N, E, S)
    if not train:
        return out, final

    dout = s["dout"].float()
    dz = None
    q = dout
    if z is not None:
        sg = _sigmoid(z)
        q = dout * z * sg
        dz = dout * y * sg * (1 + z * (1 - sg))
    if partial:
        q = torch.where(valid[..., None], q, zero)
        dz = None if dz is None else torch.where(valid[..., None], dz, zero)
    q_ = q.view(N, T, G, E // G, 1)
    x_ = x.view(N, T, G, E // G, 1)
    adj = torch.zeros(g4, device=x.device)  # the state's adjoint from later steps
    dA = torch.zeros(g4, device=x.device)
    dB, dC = torch.zeros(N, T, G, S, device=x.device), torch.zeros(N, T, G, S, device=x.device)
    dd, sB = torch.empty(N, T, E, device=x.device), torch.empty(N, T, E, device=x.device)
    for t in reversed(range(T)):
        Bt, Ct = B[:, t].unsqueeze(2), C[:, t].unsqueeze(2)
        ah = torch.exp(d_[:, t] * A)
        if partial:
            ok = valid[:, t].view(N, 1, 1, 1)
            g = torch.where(ok, adj + q_[:, t] * Ct, zero)
        else:
            g = adj + q_[:, t] * Ct
        hp = before[t]
        dC[:, t] = (q_[:, t] * (ah * hp + dx_[:, t] * Bt)).sum(2)
        dB[:, t] = (g * dx_[:, t]).sum(2)
        gah = g * ah * hp
        dA += gah * d_[:, t]
        gB = (g * Bt).sum(-1)
        sB[:, t] = gB.view(N, E)
        dd[:, t] = ((gah * A).sum(-1) + gB * x_[:, t, ..., 0]).view(N, E)
        back = ah * g
        if partial:
            back = torch.where(ok, back, adj)
        adj = torch.where(start[:, t].view(N, 1, 1, 1), zero, back) if segments else back
    draw_ = dd * _sigmoid(raw)
    dx = s["D"] * q + d * sB
    grads = dict(dx=dx.to(dtype), ddt=draw_.to(dtype), dA=dA.sum(0).reshape(E, S),
                 dB=dB.to(dtype), dC=dC.to(dtype), dD=(q * x).sum((0, 1)),
                 dz=None if dz is None else dz.to(dtype), ddt_bias=draw_.sum((0, 1)),
                 d_init=adj.reshape(N, E, S) if s["init"] is not None else None)
    return dict(out=out, final=final, **grads)


def _plain_scan_step(s):
    c = s["case"]
    N, E, S, G = c["N"], c["E"], c["S"], c["G"]
    x = s["x"].float()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    h = s["state"]
    if s["reset"] is not None:
        h = torch.where(s["reset"][:, None, None], torch.zeros((), device=h.device), h)
    h = h.view(N, G, E // G, S)
    B, C = s["B"].float().unsqueeze(2), s["C"].float().unsqueeze(2)
    h = torch.exp(d.view(N, G, -1, 1) * s["A"].view(1, G, -1, S)) * h \
        + (d * x).view(N, G, -1, 1) * B
    y = (h * C).sum(-1).view(N, E) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return y.to(s["x"].dtype), h.reshape(N, E, S)


def _plain_conv(s):
    c = s["case"]
    N, T, E, K = c["N"], c["T"], c["E"], c["K"]
    start, ended, valid = _starts(s, N, T)
    episode = start.int().cumsum(1)
    x = s["x"].float()
    w = s["weight"]
    zero = torch.zeros((), device=x.device)
    carried = torch.zeros(N, K - 1, E, device=x.device)
    if s["init"] is not None:
        carried = s["init"].float()
    padded = torch.cat([carried, x], 1)
    number = torch.cat([torch.zeros(N, K - 1, device=x.device, dtype=torch.int32),
                        episode], 1)
    p = s["bias"].expand(N, T, E)
    for k in range(K):
        same = (number[:, k:k + T] == episode)[..., None]
        p = p + w[:, k] * torch.where(same, padded[:, k:k + T], zero)
    sg = _sigmoid(p)
    out = torch.where(valid[..., None], p * sg, zero)
    # The window carried out: the last K - 1 inputs of the running episode.
    n = valid.sum(1)
    rows = n[:, None] + torch.arange(K - 1, device=x.device)
    last = (n - 1).clamp(min=0)[:, None]
    done = (n > 0) & ended.gather(1, last)[:, 0]
    current = torch.where(n[:, None] > 0, episode.gather(1, last), 0)
    keep = (number.gather(1, rows) == current) & ~done[:, None]
    final = torch.where(keep[..., None], padded.gather(1, rows[..., None].expand(-1, -1, E)),
                        zero)
    dp = torch.where(valid[..., None], s["dout"].float() * sg * (1 + p * (1 - sg)), zero)
    dx = torch.zeros(N, T + K - 1, E, device=x.device)
    dw = torch.empty(E, K, device=x.device)
    for k in range(K):
        part = torch.where((number[:, k:k + T] == episode)[..., None], dp, zero)
        dx[:, k:k + T] += w[:, k] * part
        dw[:, k] = (part * padded[:, k:k + T]).sum((0, 1))
    dtype = s["x"].dtype
    return dict(out=out.to(dtype), final=final.to(dtype), dx=dx[:, K - 1:].to(dtype), dw=dw,
                db=dp.sum((0, 1)))


def _plain_conv_step(s):
    x, state = s["x"].float(), s["state"].float()
    if s["reset"] is not None:
        state = torch.where(s["reset"][:, None, None], torch.zeros((), device=x.device), state)
    window = torch.cat([state, x[:, None]], 1)
    p = s["bias"] + (window * s["weight"].t()).sum(1)
    return (p * _sigmoid(p)).to(s["x"].dtype), window[:, 1:].to(s["x"].dtype)


def _plain_embed(s):
    table, tokens = s["table"], s["tokens"]
    inside = (tokens >= 0) & (tokens < table.shape[0])
    rows = table[torch.where(inside, tokens, 0)].float() * s["scale"]
    return torch.where(inside[..., None], rows, torch.zeros((), device=rows.device)) \
        .to(table.dtype)


def _plain_embed_grad(s):
    V, D = s["case"]["V"], s["case"]["D"]
    tokens = s["tokens"].reshape(-1)
    inside = (tokens >= 0) & (tokens < V)
    rows = torch.where(inside[:, None], s["dout"].reshape(-1, D).float() * s["scale"], 0.0)
    grad = torch.zeros(V, D, device=rows.device)
    grad.index_add_(0, torch.where(inside, tokens, 0), rows)
    return grad


# ------------------------------------------------------------------------ the framework


def _own(s):
    import segmented_associative_scan_gb300 as rlca

    c = s["case"]
    op = c["op"]
    if op == "embed":
        return rlca.embed_tokens(s["tokens"], s["table"], scale=s["scale"])
    if op == "embed_grad":
        return rlca.embed_tokens_backward(s["dout"], s["tokens"], c["V"], scale=s["scale"])
    if op == "conv_step":
        return rlca.causal_conv_step(s["x"], s["state"], s["weight"], s["bias"],
                                     reset=s["reset"], new_state=s["new_state"])
    if op == "scan_step":
        return rlca.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"],
                                        D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                        reset=s["reset"], new_state=s["new_state"])
    rows = dict(terminated=s["terminated"], truncated=s["truncated"], lengths=s["lengths"])
    if op == "conv_train":
        out, final = rlca.causal_conv(s["x"], s["weight"], s["bias"], **rows,
                                      init_state=s["init"], want_state=True)
        dx, dw, db = rlca.causal_conv_backward(s["dout"], s["x"], s["weight"], s["bias"],
                                               **rows, init_state=s["init"])
        return dict(out=out, final=final, dx=dx, dw=dw, db=db)
    extra = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], **rows)
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    if op == "scan":
        out, final, _ = rlca.selective_scan(*args, **extra, init_state=s["init"],
                                            want_state=True)
        return out, final
    out, final, saved = rlca.selective_scan(*args, **extra, init_state=s["init"],
                                            want_state=True, want_saved=True)
    dx, ddt, dA, dB, dC, dD, dz, ddt_bias, d_init = rlca.selective_scan_backward(
        s["dout"], *args, saved, **extra, want_d_init=s["init"] is not None)
    return dict(out=out, final=final, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, dz=dz,
                ddt_bias=ddt_bias, d_init=d_init)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "scan":
        return _plain_scan(state, train=False)
    if op == "scan_train":
        return _plain_scan(state, train=True)
    return {"scan_step": _plain_scan_step, "conv_train": _plain_conv,
            "conv_step": _plain_conv_step, "embed": _plain_embed,
            "embed_grad": _plain_embed_grad}[op](state)


# --------------------------------------------------------------------------------- work


def work(case):
    w = _BYTES[case["dtype"]]
    op, N, T = case["op"], case["N"], case["T"]
    if op == "embed":
        M, D = N * T, case["D"]
        return {"bytes": 2 * w * M * D + 8 * M, "flops": M * D}
    if op == "embed_grad":
        M, D = N * T, case["D"]
        return {"bytes": w * M * D + 8 * M + 4 * case["V"] * D, "flops": 2 * M * D}
    E = case["E"]
    flags = 2 * N * T if case["flags"] else 0
    if op.startswith("conv"):
        K = case["K"]
        carried = w * N * (K - 1) * E
        if op == "conv_step":
            return {"bytes": 2 * w * N * E + 2 * carried + 4 * E * (K + 1),
                    "flops": N * E * (2 * K + 4)}
        return {"bytes": 4 * w * N * T * E + carried * (2 if case["init"] else 1) + flags
                + 8 * E * (K + 1), "flops": N * T * E * (6 * K + 12)}
    S, G = case["S"], case["G"]
    state = 4 * N * E * S
    params = 4 * E * (S + 2)
    gate = 1 if case["gate"] else 0
    if op == "scan_step":
        return {"bytes": w * N * ((3 + gate) * E + 2 * G * S) + 2 * state + params,
                "flops": N * E * (7 * S + 12)}
    forward = w * N * T * ((3 + gate) * E + 2 * G * S) + flags + params \
        + state * (2 if case["init"] else 1)
    if op == "scan":
        return {"bytes": forward, "flops": N * T * E * (7 * S + 12)}
    # The gradients read dout besides and write dx, ddt, dz, dB and dC; nothing that the
    # forward pass saves is counted.
    return {"bytes": forward + w * N * T * ((3 + gate) * E + 2 * G * S) + params
            + (state if case["init"] else 0), "flops": N * T * E * (27 * S + 40)}


# ------------------------------------------------------------------- 64-bit definitions


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits; gradients by automatic
    differentiation of those definitions."""
    s = prepare(case, seed)
    op, N = case["op"], case["N"]
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
         for k, v in s.items()}
    with torch.enable_grad():
        if op.startswith("embed"):
            tokens, V, D = s["tokens"], case["V"], case["D"]
            pad = torch.zeros(1, D, dtype=torch.float64, device=tokens.device)
            row = torch.where((tokens < 0) | (tokens >= V), V, tokens)
            if op == "embed":
                return torch.cat([f["table"] * s["scale"], pad])[row]
            table = torch.zeros(V, D, dtype=torch.float64, device=tokens.device,
                                requires_grad=True)
            out = torch.cat([table * s["scale"], pad])[row]
            return torch.autograd.grad(out, table, f["dout"])[0]
        if op == "conv_step" or op == "scan_step":
            keep = torch.ones(N, dtype=torch.float64, device=f["x"].device)
            if s["reset"] is not None:
                keep = 1 - s["reset"].double()
            carried = f["state"] * keep[:, None, None]
            if op == "conv_step":
                taps = [*carried.unbind(1), f["x"]]
                p = sum((w * t for w, t in zip(f["weight"].unbind(1), taps)), f["bias"])
                return torch.nn.functional.silu(p), torch.stack(taps[1:], 1)
            seq = {k: None if f[k] is None else f[k].unsqueeze(1)
                   for k in ("x", "dt", "B", "C", "z")}
            out, final = _exact_scan({**f, **seq, "init": carried}, case)
            return out[:, 0], final
        train = op.endswith("_train")
        names = ("x", "weight", "bias") if op == "conv_train" else \
            ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")
        leaves = {k: f[k].detach().requires_grad_() for k in names
                  if train and f[k] is not None}
        if op == "conv_train":
            out, final = _exact_conv({**f, **leaves}, case)
        else:
            out, final = _exact_scan({**f, **leaves}, case)
        if not train:
            return out, final
        grads = dict(zip(leaves, torch.autograd.grad(out, list(leaves.values()), f["dout"],
                                                     allow_unused=True)))
    grads = {k: torch.zeros_like(leaves[k]) if v is None else v for k, v in grads.items()}
    out, final = out.detach(), final.detach()
    if op == "conv_train":
        return dict(out=out, final=final, dx=grads["x"], dw=grads["weight"], db=grads["bias"])
    return dict(out=out, final=final, dx=grads["x"], ddt=grads["dt"], dA=grads["A"],
                dB=grads["B"], dC=grads["C"], dD=grads["D"], dz=grads.get("z"),
                ddt_bias=grads["dt_bias"], d_init=grads.get("init"))


def _rows(f, case):
    """Per row: its length and the list of flags, as 0/1 factors [N] for every step."""
    N, T = case["N"], case["T"]
    dev = f["x"].device
    length = torch.full((N,), T, device=dev) if f["lengths"] is None else f["lengths"].long()
    ends = torch.zeros(N, T, dtype=torch.float64, device=dev)
    if f["terminated"] is not None:
        ends = (f["terminated"].int() + f["truncated"].int() > 0).double()
    inside = [(t < length).double() for t in range(T)]
    return inside, ends.unbind(1)


def _exact_scan(f, case):
    N, E, S = case["N"], case["E"], case["S"]
    dev = f["x"].device
    group = torch.arange(E, device=dev) // (E // case["G"])
    state = torch.zeros(N, E, S, dtype=torch.float64, device=dev) if f["init"] is None \
        else f["init"]
    flat = {**f, "terminated": f.get("terminated"), "lengths": f.get("lengths")}
    inside, ends = _rows(flat, case)
    delta = torch.nn.functional.softplus(f["dt"] + f["dt_bias"], threshold=700)
    outs = []
    for t, xt in enumerate(f["x"].unbind(1)):
        dt = delta[:, t, :, None]
        new = torch.exp(dt * f["A"]) * state + dt * xt[..., None] * f["B"][:, t][:, group]
        y = torch.einsum("nes,nes->ne", new, f["C"][:, t][:, group]) + f["D"] * xt
        if f["z"] is not None:
            y = y * torch.nn.functional.silu(f["z"][:, t])
        i = inside[t]
        outs.append(y * i[:, None])
        live = (i * (1 - ends[t]))[:, None, None]
        state = new * live + state * (1 - i)[:, None, None]
    return torch.stack(outs, 1), state


def _exact_conv(f, case):
    N, E, K = case["N"], case["E"], case["K"]
    dev = f["x"].device
    inside, ends = _rows(f, case)
    window = [torch.zeros(N, E, dtype=torch.float64, device=dev) for _ in range(K - 1)]
    if f["init"] is not None:
        window = list(f["init"].unbind(1))
    outs = []
    for t, xt in enumerate(f["x"].unbind(1)):
        taps = window + [xt]
        p = f["bias"]
        for k in range(K):
            p = p + f["weight"][:, k] * taps[k]
        i = inside[t][:, None]
        outs.append(torch.nn.functional.silu(p) * i)
        live = i * (1 - ends[t])[:, None]
        window = [new * live + old * (1 - i) for new, old in zip(taps[1:], window)]
    return torch.stack(outs, 1), torch.stack(window, 1)
