"""The sequence-model operators from their definitions, in 64 bits on the CPU, one step at a
time; gradients by automatic differentiation. Used by the tests only.

Masked steps (past a row's length) and what lies before an episode's start are left out by
selection, never by multiplying with 0, so an Inf or NaN there cannot come through."""
import torch

# Rounding of a result to its type, relative (2^-p for a significand of p bits), and the smallest subnormal's half.
ROUNDING = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
# Arithmetic in 32 bits: the recurrence and the sums carry some tens of roundings of 2^-24
# (exponentials of 2 ulp, a memory of tens of steps), relative to the largest value.
ARITHMETIC = 128 * 2.0 ** -24


def check(name, got, want, dtype=None):
    """|got - want| <= rounding * |want| + arithmetic * max|want|, every element."""
    dtype = dtype or got.dtype
    got = got.detach().double().cpu()
    want = want.detach()
    assert got.shape == want.shape, f"{name}: shape {tuple(got.shape)} != {tuple(want.shape)}"
    if not want.numel():
        return
    bound = ROUNDING[dtype] * want.abs() + TINY[dtype] + ARITHMETIC * want.abs().max()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = int(((got - want).abs() - bound).flatten().nan_to_num(nan=1e30).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst "
                             f"{got.flatten()[i]} for {want.flatten()[i]} (at {i})")


def rows_of(N, T, terminated, truncated, lengths):
    """Python lists: the length of each row and the flag of each step."""
    length = [T] * N if lengths is None else [min(max(int(v), 0), T) for v in lengths]
    ended = [[False] * T for _ in range(N)]
    for flags in (terminated, truncated):
        if flags is not None:
            for n in range(N):
                for t in range(T):
                    ended[n][t] |= bool(flags[n, t])
    return length, ended


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, terminated=None, truncated=None,
         lengths=None, init_state=None, dt_softplus=True):
    """(out [N, T, E], final_state [N, E, S]) in float64; B and C [N, T, G, S]."""
    N, T, E = x.shape
    S, G = A.shape[1], B.shape[2]
    group = torch.arange(E) // (E // G)
    length, ended = rows_of(N, T, terminated, truncated, lengths)
    outs, finals = [], []
    for n in range(N):
        h = init_state[n] if init_state is not None else torch.zeros(E, S, dtype=x.dtype)
        row = []
        for t in range(length[n]):
            if t > 0 and ended[n][t - 1]:
                h = torch.zeros(E, S, dtype=x.dtype)
            d = dt[n, t] if dt_bias is None else dt[n, t] + dt_bias
            if dt_softplus:
                d = torch.logaddexp(d, torch.zeros_like(d))
            h = torch.exp(d[:, None] * A) * h + (d * x[n, t])[:, None] * B[n, t][group]
            y = (h * C[n, t][group]).sum(1)
            if D is not None:
                y = y + D * x[n, t]
            if z is not None:
                y = y * z[n, t] * torch.sigmoid(z[n, t])
            row.append(y)
        row += [torch.zeros(E, dtype=x.dtype)] * (T - length[n])
        outs.append(torch.stack(row) if row else torch.zeros(0, E, dtype=x.dtype))
        if length[n] and ended[n][length[n] - 1]:
            h = torch.zeros(E, S, dtype=x.dtype)
        finals.append(h)
    return torch.stack(outs), torch.stack(finals)


def conv(x, weight, bias=None, terminated=None, truncated=None, lengths=None, init_state=None,
         silu=True):
    """(out [N, T, E], final_state [N, K-1, E]) in float64."""
    N, T, E = x.shape
    K = weight.shape[1]
    zero = torch.zeros(E, dtype=x.dtype)
    length, ended = rows_of(N, T, terminated, truncated, lengths)
    outs, finals = [], []
    for n in range(N):
        window = [zero] * (K - 1) if init_state is None else list(init_state[n])
        row = []
        for t in range(length[n]):
            if t > 0 and ended[n][t - 1]:
                window = [zero] * (K - 1)
            window = window + [x[n, t]]
            p = zero if bias is None else bias
            for k in range(K):
                p = p + weight[:, k] * window[k]
            window = window[1:]
            row.append(p * torch.sigmoid(p) if silu else p)
        row += [zero] * (T - length[n])
        outs.append(torch.stack(row) if row else torch.zeros(0, E, dtype=x.dtype))
        if length[n] and ended[n][length[n] - 1]:
            window = [zero] * (K - 1)
        finals.append(torch.stack(window) if K > 1 else torch.zeros(0, E, dtype=x.dtype))
    return torch.stack(outs), torch.stack(finals)


def embed(tokens, table, scale):
    rows = [table[int(t)] * scale if 0 <= int(t) < table.shape[0]
            else torch.zeros(table.shape[1], dtype=table.dtype) for t in tokens.flatten()]
    if not rows:
        return torch.zeros(tuple(tokens.shape) + (table.shape[1],), dtype=table.dtype)
    return torch.stack(rows).view(*tokens.shape, -1)
