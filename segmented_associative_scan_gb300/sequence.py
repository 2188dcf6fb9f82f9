"""Binding of the sequence-model operators of librlca (``include/rlca_sequence.h``): token
embedding, short causal convolution and selective state space scan, each with its gradient,
the last two also for one token at a time.

Argument marshalling only, like the rest of the package. Activations are [N, T, channels]
CUDA tensors of one data type (float32, bfloat16 or float16), unit stride over the
channels, any stride over rows and steps; parameters, the scan's states and gradients of
parameters are contiguous float32. `terminated` / `truncated` [N, T] (uint8 or bool) end
episodes, `lengths` int32 [N] cuts rows short. Outputs and workspaces are allocated unless
passed in; work is enqueued on the current stream and nothing synchronises.
"""
from __future__ import annotations

import ctypes

import torch

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_F = ctypes.c_float

SCAN_CHUNK = 8  # RLCA_SCAN_CHUNK


class Steps(ctypes.Structure):
    _fields_ = [("ptr", _P), ("row", _I64), ("step", _I64)]


class Rows(ctypes.Structure):
    _fields_ = [("terminated", _P), ("truncated", _P), ("flag_ld", _I64), ("lengths", _P)]


class Scan(ctypes.Structure):
    _fields_ = [("N", _I64), ("T", _I64), ("E", _I64), ("S", _I64), ("G", _I64), ("x", Steps),
                ("dt", Steps), ("z", Steps), ("B", Steps), ("C", Steps), ("A", _P), ("D", _P),
                ("dt_bias", _P), ("rows", Rows), ("init_state", _P), ("dt_softplus", _I32)]


class ScanGrads(ctypes.Structure):
    _fields_ = [("dout", Steps), ("d_final_state", _P), ("saved", _P), ("dx", Steps),
                ("ddt", Steps), ("dz", Steps), ("dB", Steps), ("dC", Steps), ("dA", _P),
                ("dD", _P), ("ddt_bias", _P), ("d_init_state", _P)]


class Conv(ctypes.Structure):
    _fields_ = [("N", _I64), ("T", _I64), ("E", _I64), ("K", _I64), ("x", Steps),
                ("weight", _P), ("bias", _P), ("rows", Rows), ("init_state", _P),
                ("silu", _I32)]


SIGNATURES = {
    "rlca_selective_scan_workspace_bytes": ([_I64] * 5, _SZ),
    "rlca_selective_scan_saved_bytes": ([_I64] * 4, _SZ),
    "rlca_causal_conv_workspace_bytes": ([_I64] * 4, _SZ),
    "rlca_embed_tokens_workspace_bytes": ([_I64] * 3, _SZ),
}
for _suffix in ("", "_bf16", "_fp16"):
    SIGNATURES["rlca_selective_scan" + _suffix] = (
        [ctypes.POINTER(Scan), Steps, _P, _P, _P, _SZ, _P], ctypes.c_int)
    SIGNATURES["rlca_selective_scan_backward" + _suffix] = (
        [ctypes.POINTER(Scan), ctypes.POINTER(ScanGrads), _P, _SZ, _P], ctypes.c_int)
    SIGNATURES["rlca_selective_scan_step" + _suffix] = (
        [ctypes.POINTER(Scan), _P, Steps, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_causal_conv" + _suffix] = (
        [ctypes.POINTER(Conv), Steps, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_causal_conv_backward" + _suffix] = (
        [ctypes.POINTER(Conv), Steps, Steps, _P, _P, _P, _SZ, _P], ctypes.c_int)
    SIGNATURES["rlca_causal_conv_step" + _suffix] = (
        [ctypes.POINTER(Conv), _P, Steps, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_embed_tokens" + _suffix] = (
        [_P, _I32, _P, _I64, _F, _I64, _I64, _I64, _P, _I64, _P], ctypes.c_int)
    SIGNATURES["rlca_embed_tokens_backward" + _suffix] = (
        [_P, _I64, _P, _I32, _F, _I64, _I64, _I64, _P, _P, _SZ, _P], ctypes.c_int)

_SUFFIX = {torch.float32: "", torch.bfloat16: "_bf16", torch.float16: "_fp16"}
_FLAG = (torch.uint8, torch.bool)


def _base():
    import segmented_associative_scan_gb300 as rlca
    return rlca


def _suffix_of(t, name):
    if t.dtype not in _SUFFIX:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_SUFFIX)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return _SUFFIX[t.dtype]


def _run(name, *args, device):
    rlca = _base()
    stream = ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    rlca._check(name, getattr(rlca.lib(), name)(*args, stream))


def _like(t, name, ref, shape):
    """Checks an activation against the call's device, data type and shape."""
    if t.dtype != ref.dtype:
        raise TypeError(f"{name}: dtype {t.dtype} is not the call's {ref.dtype}")
    if t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {shape}")


def _steps(t, name, ref, shape):
    """The rlca_steps of an activation [N, T, ...] whose trailing dimensions are dense."""
    _like(t, name, ref, shape)
    dense = 1
    for size, stride in zip(reversed(shape[2:]), reversed(t.stride()[2:])):
        if size > 1 and stride != dense:
            raise ValueError(f"{name}: channels must be contiguous (unit stride)")
        dense *= size
    return Steps(t.data_ptr() or None, t.stride(0), t.stride(1))


def _row(t, name, ref, shape):
    """The same for one step: [N, ...]."""
    _like(t, name, ref, shape)
    dense = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != dense:
            raise ValueError(f"{name}: channels must be contiguous (unit stride)")
        dense *= size
    return Steps(t.data_ptr() or None, t.stride(0), 0)


def _flat(t, name, ref, shape, dtypes=(torch.float32,)):
    """Pointer of a contiguous tensor (parameters, states, lengths), None for None."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _rows(terminated, truncated, lengths, ref, N, T):
    ld = T
    ptrs = []
    first = None
    for t, name in ((terminated, "terminated"), (truncated, "truncated")):
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype not in _FLAG:
            raise TypeError(f"{name}: dtype {t.dtype} not in {_FLAG}")
        if t.device != ref.device:
            raise ValueError(f"{name} must be on {ref.device}")
        if tuple(t.shape) != (N, T):
            raise ValueError(f"{name}: shape {tuple(t.shape)} != {(N, T)}")
        if T > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: steps must be contiguous (stride(1) == 1)")
        row = t.stride(0) if N > 1 else T
        if first is not None and row != first:
            raise ValueError(f"{name}: row stride {row} != {first}")
        first = ld = row
        ptrs.append(t.data_ptr() or None)
    return Rows(ptrs[0], ptrs[1], ld, _flat(lengths, "lengths", ref, (N,), (torch.int32,)))


def _out(t, shape, dtype, ref):
    return torch.empty(shape, dtype=dtype, device=ref.device) if t is None else t


def _workspace(workspace, need, ref):
    """(pointer, bytes, tensor) of a workspace of at least `need` bytes."""
    if workspace is None:
        workspace = torch.empty(max(1, need), dtype=torch.uint8, device=ref.device)
    elif not workspace.is_cuda or workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a CUDA uint8 tensor")
    return workspace.data_ptr() or None, workspace.numel(), workspace


# ------------------------------------------------------------------------ selective scan


def _scan(x, dt, A, B, C, D, z, dt_bias, rows, dt_softplus, one_step):
    """The rlca_scan of a call (init_state left out); `one_step`: no dimension T."""
    lead = 1 if one_step else 2
    if x.dim() != lead + 1:
        raise ValueError("x must be [N, E]" if one_step else "x must be [N, T, E]")
    steps = _row if one_step else _steps
    N, E = x.shape[0], x.shape[-1]
    T = 1 if one_step else x.shape[1]
    if A.dim() != 2:
        raise ValueError("A must be [E, S]")
    S = A.shape[1]
    if B.dim() not in (lead + 1, lead + 2):
        raise ValueError("B and C must be [..., G, S], or [..., S] for one group")
    G = B.shape[lead] if B.dim() == lead + 2 else 1
    wide = tuple(x.shape[:lead]) + ((G, S) if B.dim() == lead + 2 else (S,))
    shape = tuple(x.shape)
    p = Scan(N, T, E, S, G, steps(x, "x", x, shape), steps(dt, "dt", x, shape),
             Steps() if z is None else steps(z, "z", x, shape), steps(B, "B", x, wide),
             steps(C, "C", x, wide), _flat(A, "A", x, (E, S)), _flat(D, "D", x, (E,)),
             _flat(dt_bias, "dt_bias", x, (E,)), rows, None, 1 if dt_softplus else 0)
    return p, wide


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, terminated=None,
                   truncated=None, lengths=None, init_state=None, dt_softplus=True, out=None,
                   final_state=None, saved=None, want_state=False, want_saved=False,
                   workspace=None):
    """Segmented selective state space scan over whole windows (rlca_selective_scan):
    returns (out, final_state, saved). `saved` (want_saved) is what
    `selective_scan_backward` reads; final_state (want_state) continues the rows."""
    name = "rlca_selective_scan" + _suffix_of(x, "x")
    N, T = x.shape[0], x.shape[1] if x.dim() == 3 else 0
    p, _ = _scan(x, dt, A, B, C, D, z, dt_bias,
                 _rows(terminated, truncated, lengths, x, N, T), dt_softplus, False)
    E, S = p.E, p.S
    p.init_state = _flat(init_state, "init_state", x, (N, E, S))
    out = _out(out, (N, T, E), x.dtype, x)
    if final_state is None and want_state:
        final_state = torch.empty((N, E, S), dtype=torch.float32, device=x.device)
    saved_shape = (N, (T + SCAN_CHUNK - 1) // SCAN_CHUNK, E, S)
    if saved is None and want_saved:
        saved = torch.empty(saved_shape, dtype=torch.float32, device=x.device)
    lib = _base().lib()
    need = lib.rlca_selective_scan_workspace_bytes(N, T, E, S, p.G)
    ws, ws_bytes, keep = _workspace(workspace, need, x)
    _run(name, ctypes.byref(p), _steps(out, "out", x, (N, T, E)),
         _flat(final_state, "final_state", x, (N, E, S)),
         _flat(saved, "saved", x, saved_shape), ws, ws_bytes, device=x.device)
    return out, final_state, saved


def selective_scan_backward(dout, x, dt, A, B, C, saved, D=None, z=None, dt_bias=None,
                            terminated=None, truncated=None, lengths=None, dt_softplus=True,
                            d_final_state=None, dx=None, ddt=None, dz=None, dB=None, dC=None,
                            want_d_init=False, workspace=None):
    """Gradients of `selective_scan`: returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias,
    d_init_state), None for what the call has no argument of (d_init_state: want_d_init).
    dx, ddt, dz, dB and dC may be given, as slices of a wider gradient for instance."""
    name = "rlca_selective_scan_backward" + _suffix_of(x, "x")
    N, T = x.shape[0], x.shape[1] if x.dim() == 3 else 0
    p, wide = _scan(x, dt, A, B, C, D, z, dt_bias,
                    _rows(terminated, truncated, lengths, x, N, T), dt_softplus, False)
    E, S = p.E, p.S
    shape = (N, T, E)
    dx, ddt = _out(dx, shape, x.dtype, x), _out(ddt, shape, x.dtype, x)
    dz = None if z is None else _out(dz, shape, x.dtype, x)
    dB, dC = _out(dB, wide, x.dtype, x), _out(dC, wide, x.dtype, x)
    f32 = dict(dtype=torch.float32, device=x.device)
    dA = torch.empty((E, S), **f32)
    dD = None if D is None else torch.empty(E, **f32)
    ddt_bias = None if dt_bias is None else torch.empty(E, **f32)
    d_init = torch.empty((N, E, S), **f32) if want_d_init else None
    g = ScanGrads(_steps(dout, "dout", x, shape),
                  _flat(d_final_state, "d_final_state", x, (N, E, S)),
                  _flat(saved, "saved", x, (N, (T + SCAN_CHUNK - 1) // SCAN_CHUNK, E, S)),
                  _steps(dx, "dx", x, shape), _steps(ddt, "ddt", x, shape),
                  Steps() if dz is None else _steps(dz, "dz", x, shape),
                  _steps(dB, "dB", x, wide), _steps(dC, "dC", x, wide), dA.data_ptr() or None,
                  None if dD is None else dD.data_ptr() or None,
                  None if ddt_bias is None else ddt_bias.data_ptr() or None,
                  None if d_init is None else d_init.data_ptr() or None)
    need = _base().lib().rlca_selective_scan_workspace_bytes(N, T, E, S, p.G)
    ws, ws_bytes, keep = _workspace(workspace, need, x)
    _run(name, ctypes.byref(p), ctypes.byref(g), ws, ws_bytes, device=x.device)
    return dx, ddt, dA, dB, dC, dD, dz, ddt_bias, d_init


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, reset=None,
                        dt_softplus=True, out=None, new_state=None):
    """One step of N rows (no dimension T): returns (out, new_state). Rows with `reset`
    ([N] uint8 or bool) start from 0. The state is updated in place unless new_state is
    given."""
    name = "rlca_selective_scan_step" + _suffix_of(x, "x")
    p, _ = _scan(x, dt, A, B, C, D, z, dt_bias, Rows(), dt_softplus, True)
    shape = (p.N, p.E, p.S)
    p.init_state = _flat(state, "state", x, shape)
    new_state = state if new_state is None else new_state
    out = torch.empty((p.N, p.E), dtype=x.dtype, device=x.device) if out is None else out
    _run(name, ctypes.byref(p), _flat(reset, "reset", x, (p.N,), _FLAG),
         _row(out, "out", x, (p.N, p.E)), _flat(new_state, "new_state", x, shape),
         device=x.device)
    return out, new_state


# -------------------------------------------------------------------- causal convolution


def _conv(x, weight, bias, rows, silu, one_step):
    lead = 1 if one_step else 2
    if x.dim() != lead + 1:
        raise ValueError("x must be [N, E]" if one_step else "x must be [N, T, E]")
    if weight.dim() != 2:
        raise ValueError("weight must be [E, K]")
    N, E, K = x.shape[0], x.shape[-1], weight.shape[1]
    steps = _row if one_step else _steps
    return Conv(N, 1 if one_step else x.shape[1], E, K, steps(x, "x", x, tuple(x.shape)),
                _flat(weight, "weight", x, (E, K)), _flat(bias, "bias", x, (E,)), rows, None,
                1 if silu else 0)


def causal_conv(x, weight, bias=None, terminated=None, truncated=None, lengths=None,
                init_state=None, silu=True, out=None, final_state=None, want_state=False):
    """Short causal convolution over whole windows (rlca_causal_conv): returns (out,
    final_state). final_state [N, K-1, E] (want_state) continues the rows."""
    name = "rlca_causal_conv" + _suffix_of(x, "x")
    N, T = x.shape[0], x.shape[1] if x.dim() == 3 else 0
    p = _conv(x, weight, bias, _rows(terminated, truncated, lengths, x, N, T), silu, False)
    states = (N, p.K - 1, p.E)
    p.init_state = _flat(init_state, "init_state", x, states, (x.dtype,))
    out = _out(out, (N, T, p.E), x.dtype, x)
    if final_state is None and want_state:
        final_state = torch.empty(states, dtype=x.dtype, device=x.device)
    _run(name, ctypes.byref(p), _steps(out, "out", x, (N, T, p.E)),
         _flat(final_state, "final_state", x, states, (x.dtype,)), device=x.device)
    return out, final_state


def causal_conv_backward(dout, x, weight, bias=None, terminated=None, truncated=None,
                         lengths=None, init_state=None, silu=True, dx=None, workspace=None):
    """Gradients of `causal_conv`: returns (dx, dweight, dbias), dbias None without bias."""
    name = "rlca_causal_conv_backward" + _suffix_of(x, "x")
    N, T = x.shape[0], x.shape[1] if x.dim() == 3 else 0
    p = _conv(x, weight, bias, _rows(terminated, truncated, lengths, x, N, T), silu, False)
    E, K = p.E, p.K
    p.init_state = _flat(init_state, "init_state", x, (N, K - 1, E), (x.dtype,))
    dx = _out(dx, (N, T, E), x.dtype, x)
    dweight = torch.empty((E, K), dtype=torch.float32, device=x.device)
    dbias = None if bias is None else torch.empty(E, dtype=torch.float32, device=x.device)
    need = _base().lib().rlca_causal_conv_workspace_bytes(N, T, E, K)
    ws, ws_bytes, keep = _workspace(workspace, need, x)
    _run(name, ctypes.byref(p), _steps(dout, "dout", x, (N, T, E)),
         _steps(dx, "dx", x, (N, T, E)), dweight.data_ptr() or None,
         None if dbias is None else dbias.data_ptr() or None, ws, ws_bytes, device=x.device)
    return dx, dweight, dbias


def causal_conv_step(x, state, weight, bias=None, reset=None, silu=True, out=None,
                     new_state=None):
    """One step of N rows: x [N, E], state [N, K-1, E]; returns (out, new_state). The state
    is updated in place unless new_state is given."""
    name = "rlca_causal_conv_step" + _suffix_of(x, "x")
    p = _conv(x, weight, bias, Rows(), silu, True)
    states = (p.N, p.K - 1, p.E)
    p.init_state = _flat(state, "state", x, states, (x.dtype,))
    new_state = state if new_state is None else new_state
    out = torch.empty((p.N, p.E), dtype=x.dtype, device=x.device) if out is None else out
    _run(name, ctypes.byref(p), _flat(reset, "reset", x, (p.N,), _FLAG),
         _row(out, "out", x, (p.N, p.E)), _flat(new_state, "new_state", x, states, (x.dtype,)),
         device=x.device)
    return out, new_state


# ------------------------------------------------------------------------ token embedding


def _tokens(tokens, ref):
    if tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError("tokens must be int32 or int64")
    if tokens.device != ref.device:
        raise ValueError(f"tokens must be on {ref.device}")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return tokens.data_ptr() or None, tokens.element_size()


def _matrix(t, name, M, D):
    """Pointer and row stride of a tensor [..., D] seen as [M, D]."""
    if D > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: channels must be contiguous (unit stride)")
    if M <= 1 or t.dim() == 1:
        return t.data_ptr() or None, D
    ld, size = None, 1
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * size:
            raise ValueError(f"{name}: rows must lie at one stride")
        size *= n
    return t.data_ptr() or None, D if ld is None else ld


def embed_tokens(tokens, table, scale=1.0, out=None):
    """scale * table[tokens] (rlca_embed_tokens) for int32 / int64 tokens of any shape; a
    token outside the table gives a row of zeros."""
    if table.dim() != 2:
        raise ValueError("table must be [V, D]")
    name = "rlca_embed_tokens" + _suffix_of(table, "table")
    V, D = table.shape
    M = tokens.numel()
    tok, tok_bytes = _tokens(tokens, table)
    shape = tuple(tokens.shape) + (D,)
    out = _out(out, shape, table.dtype, table)
    _like(out, "out", table, shape)
    tab, tab_ld = _matrix(table, "table", V, D)
    dst, dst_ld = _matrix(out, "out", M, D)
    _run(name, tok, tok_bytes, tab, tab_ld, scale, M, V, D, dst, dst_ld, device=table.device)
    return out


def embed_tokens_backward(dout, tokens, vocab, scale=1.0, dtable=None, workspace=None):
    """The table's gradient [vocab, D] in float32, every row written: scale times the sum of
    dout over the positions of each token."""
    name = "rlca_embed_tokens_backward" + _suffix_of(dout, "dout")
    D, M = dout.shape[-1], tokens.numel()
    if tuple(dout.shape[:-1]) != tuple(tokens.shape):
        raise ValueError(f"dout: shape {tuple(dout.shape)} does not fit tokens "
                         f"{tuple(tokens.shape)}")
    tok, tok_bytes = _tokens(tokens, dout)
    dtable = _out(dtable, (vocab, D), torch.float32, dout)
    src, ld = _matrix(dout, "dout", M, D)
    need = _base().lib().rlca_embed_tokens_workspace_bytes(M, vocab, D)
    ws, ws_bytes, keep = _workspace(workspace, need, dout)
    _run(name, src, ld, tok, tok_bytes, scale, M, vocab, D,
         _flat(dtable, "dtable", dout, (vocab, D)), ws, ws_bytes, device=dout.device)
    return dtable
