"""Binding of the sequence-model operators of librlca (``include/rlca_sequence.h``): token
embedding, short causal convolution and selective state space scan, each with its gradient,
the last two also for one token at a time.

Argument marshalling only, like the rest of the package. Activations are [N, T, channels]
CUDA tensors of one data type (float32, bfloat16 or float16), unit stride over the
channels, any stride over rows and steps; parameters, the scan's states and gradients of
parameters are contiguous float32. `terminated` / `truncated` [N, T] (uint8 or bool) end
episodes, `lengths` int32 [N] cuts rows short. Outputs and workspaces are allocated unless
passed in; work is enqueued on the current stream and nothing synchronises.

The calls build no autograd graph, like the estimators': results of tensors that require
gradients come without one, and gradients are calls of their own (``*_backward``).
"""
from __future__ import annotations

import ctypes
import struct

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


# The structs as the calls below pass them: packed in one go from plain numbers, which takes a
# fraction of the time of filling a ctypes structure (a step's call is all host time).
_STEPS = "Pqq"
_ROWS = "PPqP"
_PACK_SCAN = struct.Struct("@5q" + 5 * _STEPS + "PPP" + _ROWS + "Pi4x").pack
_PACK_GRADS = struct.Struct("@" + _STEPS + "PP" + 5 * _STEPS + "PPPP").pack
_PACK_CONV = struct.Struct("@4q" + _STEPS + "PP" + _ROWS + "Pi4x").pack

SIGNATURES = {
    "rlca_selective_scan_workspace_bytes": ([_I64] * 5, _SZ),
    "rlca_selective_scan_forward_workspace_bytes": ([_I64] * 5, _SZ),
    "rlca_selective_scan_saved_bytes": ([_I64] * 4, _SZ),
    "rlca_causal_conv_workspace_bytes": ([_I64] * 4, _SZ),
    "rlca_embed_tokens_workspace_bytes": ([_I64] * 3, _SZ),
}
for _suffix in ("", "_bf16", "_fp16"):
    SIGNATURES["rlca_selective_scan" + _suffix] = (
        [_P, Steps, _P, _P, _P, _SZ, _P], ctypes.c_int)
    SIGNATURES["rlca_selective_scan_backward" + _suffix] = (
        [_P, _P, _P, _SZ, _P], ctypes.c_int)
    SIGNATURES["rlca_selective_scan_step" + _suffix] = (
        [_P, _P, Steps, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_causal_conv" + _suffix] = (
        [_P, Steps, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_causal_conv_backward" + _suffix] = (
        [_P, Steps, Steps, _P, _P, _P, _SZ, _P], ctypes.c_int)
    SIGNATURES["rlca_causal_conv_step" + _suffix] = (
        [_P, _P, Steps, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_embed_tokens" + _suffix] = (
        [_P, _I32, _P, _I64, _F, _I64, _I64, _I64, _P, _I64, _P], ctypes.c_int)
    SIGNATURES["rlca_embed_tokens_backward" + _suffix] = (
        [_P, _I64, _P, _I32, _F, _I64, _I64, _I64, _P, _P, _SZ, _P], ctypes.c_int)

_SUFFIX = {torch.float32: "", torch.bfloat16: "_bf16", torch.float16: "_fp16"}
_FLAG = (torch.uint8, torch.bool)
_NO_STEPS = (0, 0, 0)
_NO_ROWS = (0, 0, 0, 0)

_functions = {}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _base():
    import segmented_associative_scan_gb300 as rlca
    return rlca


def _function(name):
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_base().lib(), name)
    return fn


def _suffix_of(t, name):
    suffix = _SUFFIX.get(t.dtype)
    if suffix is None:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_SUFFIX)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return suffix


def _run(name, suffix, dev, *args):
    stream = (_raw_stream(dev) if _raw_stream is not None
              else torch.cuda.current_stream(dev).cuda_stream)
    fn = _functions.get(name + suffix)
    status = (_function(name + suffix) if fn is None else fn)(*args, stream)
    if status:
        _base()._check(name + suffix, status)


# The checks below compare in one expression and sort out what is wrong only where something is:
# a one-token call is little else than these checks.


def _refuse(t, name, dtypes, dev, shape):
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _steps(t, name, dtype, dev, shape, lead=2):
    """(pointer, row stride, step stride) of an activation of `lead` leading dimensions (1: one
    step, no dimension T), the one or two trailing ones dense."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, (dtype,), dev, shape)
    s = t.stride()
    if (s[-1] != 1 and shape[-1] > 1) or (len(s) == lead + 2 and shape[-2] > 1
                                          and s[-2] != shape[-1]):
        raise ValueError(f"{name}: channels must be contiguous (unit stride)")
    return t.data_ptr(), s[0], s[1] if lead == 2 else 0


def _flat(t, name, dev, shape, dtype=torch.float32):
    """Pointer of a contiguous tensor (parameters, states, lengths), 0 for None."""
    if t is None:
        return 0
    if (t.dtype is not dtype or t.get_device() != dev or t.shape != shape
            or not t.is_contiguous()):
        _refuse(t, name, (dtype,), dev, shape)
    return t.data_ptr()


def _reset(t, dev, N):
    if t is None:
        return 0
    if t.dtype not in _FLAG or t.get_device() != dev or t.shape != (N,) or not t.is_contiguous():
        _refuse(t, "reset", _FLAG, dev, (N,))
    return t.data_ptr()


def _rows(terminated, truncated, lengths, dev, N, T):
    if terminated is None and truncated is None and lengths is None:
        return _NO_ROWS
    ld = T
    ptrs = [0, 0]
    first = None
    for i, t in enumerate((terminated, truncated)):
        if t is None:
            continue
        name = "truncated" if i else "terminated"
        if t.dtype not in _FLAG or t.get_device() != dev or t.shape != (N, T):
            _refuse(t, name, _FLAG, dev, (N, T))
        s = t.stride()
        if T > 1 and s[1] != 1:
            raise ValueError(f"{name}: steps must be contiguous (stride(1) == 1)")
        row = s[0] if N > 1 else T
        if first is not None and row != first:
            raise ValueError(f"{name}: row stride {row} != {first}")
        first = ld = row
        ptrs[i] = t.data_ptr()
    return ptrs[0], ptrs[1], ld, _flat(lengths, "lengths", dev, (N,), torch.int32)


def _out(t, shape, ref):
    return ref.new_empty(shape) if t is None else t


def _f32(ref, shape):
    return torch.empty(shape, dtype=torch.float32, device=ref.device)


def _workspace(workspace, need, ref):
    """A workspace of at least `need` bytes (the library checks one that is given)."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=ref.device) if need else None
    if not workspace.is_cuda or workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a CUDA uint8 tensor")
    return workspace


def _ws(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())


# ------------------------------------------------------------------------ selective scan


def _scan(x, dev, dt, A, B, C, D, z, dt_bias, rows, init_state, dt_softplus, lead):
    """The packed rlca_scan of a call, (N, T, E, S, G) and the shape of B and C; lead 1: one
    step (no dimension T)."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != lead + 1:
        raise ValueError("x must be [N, E]" if lead == 1 else "x must be [N, T, E]")
    N, E = shape[0], shape[-1]
    T = 1 if lead == 1 else shape[1]
    if A.dim() != 2:
        raise ValueError("A must be [E, S]")
    S = A.shape[1]
    wide = B.shape
    if len(wide) == lead + 2:
        G = wide[lead]
    elif len(wide) == lead + 1:
        G = 1
    else:
        raise ValueError("B and C must be [..., G, S], or [..., S] for one group")
    if wide[:lead] != shape[:lead] or wide[-1] != S:
        raise ValueError(f"B: shape {tuple(wide)} does not fit x {tuple(shape)} and S = {S}")
    packed = _PACK_SCAN(
        N, T, E, S, G, *_steps(x, "x", dtype, dev, shape, lead),
        *_steps(dt, "dt", dtype, dev, shape, lead),
        *(_NO_STEPS if z is None else _steps(z, "z", dtype, dev, shape, lead)),
        *_steps(B, "B", dtype, dev, wide, lead), *_steps(C, "C", dtype, dev, wide, lead),
        _flat(A, "A", dev, (E, S)), _flat(D, "D", dev, (E,)),
        _flat(dt_bias, "dt_bias", dev, (E,)), *rows,
        _flat(init_state, "init_state", dev, (N, E, S)), 1 if dt_softplus else 0)
    return packed, (N, T, E, S, G), wide


def _window(x):
    if x.dim() != 3:
        raise ValueError("x must be [N, T, E]")
    return x.shape[0], x.shape[1]


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, terminated=None,
                   truncated=None, lengths=None, init_state=None, dt_softplus=True, out=None,
                   final_state=None, saved=None, want_state=False, want_saved=False,
                   workspace=None):
    """Segmented selective state space scan over whole windows (rlca_selective_scan):
    returns (out, final_state, saved). `saved` (want_saved) is what
    `selective_scan_backward` reads; final_state (want_state) continues the rows."""
    suffix, dev, dtype = _suffix_of(x, "x"), x.get_device(), x.dtype
    rows = _rows(terminated, truncated, lengths, dev, *_window(x))
    p, (N, T, E, S, G), _ = _scan(x, dev, dt, A, B, C, D, z, dt_bias, rows, init_state,
                                  dt_softplus, 2)
    out = _out(out, x.shape, x)
    if final_state is None and want_state:
        final_state = _f32(x, (N, E, S))
    saved_shape = (N, (T + SCAN_CHUNK - 1) // SCAN_CHUNK, E, S)
    if saved is None and want_saved:
        saved = _f32(x, saved_shape)
    workspace = _workspace(workspace,
                           _function("rlca_selective_scan_forward_workspace_bytes")(N, T, E, S,
                                                                                    G), x)
    _run("rlca_selective_scan", suffix, dev, p, Steps(*_steps(out, "out", dtype, dev, x.shape)),
         _flat(final_state, "final_state", dev, (N, E, S)),
         _flat(saved, "saved", dev, saved_shape), *_ws(workspace))
    return out, final_state, saved


def selective_scan_backward(dout, x, dt, A, B, C, saved, D=None, z=None, dt_bias=None,
                            terminated=None, truncated=None, lengths=None, dt_softplus=True,
                            d_final_state=None, dx=None, ddt=None, dz=None, dB=None, dC=None,
                            want_d_init=False, workspace=None):
    """Gradients of `selective_scan`: returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias,
    d_init_state), None for what the call has no argument of (d_init_state: want_d_init).
    dx, ddt, dz, dB and dC may be given, as slices of a wider gradient for instance."""
    suffix, dev, dtype = _suffix_of(x, "x"), x.get_device(), x.dtype
    rows = _rows(terminated, truncated, lengths, dev, *_window(x))
    p, (N, T, E, S, G), wide = _scan(x, dev, dt, A, B, C, D, z, dt_bias, rows, None,
                                     dt_softplus, 2)
    shape = x.shape
    dx, ddt = _out(dx, shape, x), _out(ddt, shape, x)
    dz = None if z is None else _out(dz, shape, x)
    dB, dC = _out(dB, wide, x), _out(dC, wide, x)
    dA = _f32(x, (E, S))
    dD = None if D is None else _f32(x, (E,))
    ddt_bias = None if dt_bias is None else _f32(x, (E,))
    d_init = _f32(x, (N, E, S)) if want_d_init else None
    ptr = lambda t: 0 if t is None else t.data_ptr()
    g = _PACK_GRADS(
        *_steps(dout, "dout", dtype, dev, shape),
        _flat(d_final_state, "d_final_state", dev, (N, E, S)),
        _flat(saved, "saved", dev, (N, (T + SCAN_CHUNK - 1) // SCAN_CHUNK, E, S)),
        *_steps(dx, "dx", dtype, dev, shape), *_steps(ddt, "ddt", dtype, dev, shape),
        *(_NO_STEPS if dz is None else _steps(dz, "dz", dtype, dev, shape)),
        *_steps(dB, "dB", dtype, dev, wide), *_steps(dC, "dC", dtype, dev, wide), ptr(dA),
        ptr(dD), ptr(ddt_bias),
        ptr(d_init))
    workspace = _workspace(workspace,
                           _function("rlca_selective_scan_workspace_bytes")(N, T, E, S, G), x)
    _run("rlca_selective_scan_backward", suffix, dev, p, g, *_ws(workspace))
    return dx, ddt, dA, dB, dC, dD, dz, ddt_bias, d_init


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, reset=None,
                        dt_softplus=True, out=None, new_state=None):
    """One step of N rows (no dimension T): returns (out, new_state). Rows with `reset`
    ([N] uint8 or bool) start from 0. The state is updated in place unless new_state is
    given."""
    suffix, dev, dtype = _suffix_of(x, "x"), x.get_device(), x.dtype
    p, (N, _, E, S, _), _ = _scan(x, dev, dt, A, B, C, D, z, dt_bias, _NO_ROWS, state,
                                  dt_softplus, 1)
    new_state = state if new_state is None else new_state
    out = _out(out, x.shape, x)
    _run("rlca_selective_scan_step", suffix, dev, p, _reset(reset, dev, N),
         Steps(*_steps(out, "out", dtype, dev, x.shape, 1)),
         _flat(new_state, "new_state", dev, (N, E, S)))
    return out, new_state


# -------------------------------------------------------------------- causal convolution


def _conv(x, dev, weight, bias, rows, init_state, silu, lead):
    """The packed rlca_conv of a call, (N, T, E, K) and the state's shape."""
    if x.dim() != lead + 1:
        raise ValueError("x must be [N, E]" if lead == 1 else "x must be [N, T, E]")
    if weight.dim() != 2:
        raise ValueError("weight must be [E, K]")
    shape = x.shape
    N, E, K = shape[0], shape[-1], weight.shape[1]
    T = 1 if lead == 1 else shape[1]
    states = (N, K - 1, E)
    packed = _PACK_CONV(
        N, T, E, K, *_steps(x, "x", x.dtype, dev, shape, lead),
        _flat(weight, "weight", dev, (E, K)), _flat(bias, "bias", dev, (E,)), *rows,
        _flat(init_state, "init_state", dev, states, x.dtype), 1 if silu else 0)
    return packed, (N, T, E, K), states


def causal_conv(x, weight, bias=None, terminated=None, truncated=None, lengths=None,
                init_state=None, silu=True, out=None, final_state=None, want_state=False):
    """Short causal convolution over whole windows (rlca_causal_conv): returns (out,
    final_state). final_state [N, K-1, E] (want_state) continues the rows."""
    suffix, dev, dtype = _suffix_of(x, "x"), x.get_device(), x.dtype
    rows = _rows(terminated, truncated, lengths, dev, *_window(x))
    p, _, states = _conv(x, dev, weight, bias, rows, init_state, silu, 2)
    out = _out(out, x.shape, x)
    if final_state is None and want_state:
        final_state = x.new_empty(states)
    _run("rlca_causal_conv", suffix, dev, p, Steps(*_steps(out, "out", dtype, dev, x.shape)),
         _flat(final_state, "final_state", dev, states, dtype))
    return out, final_state


def causal_conv_backward(dout, x, weight, bias=None, terminated=None, truncated=None,
                         lengths=None, init_state=None, silu=True, dx=None, workspace=None):
    """Gradients of `causal_conv`: returns (dx, dweight, dbias), dbias None without bias."""
    suffix, dev, dtype = _suffix_of(x, "x"), x.get_device(), x.dtype
    rows = _rows(terminated, truncated, lengths, dev, *_window(x))
    p, (N, T, E, K), _ = _conv(x, dev, weight, bias, rows, init_state, silu, 2)
    dx = _out(dx, x.shape, x)
    dweight = _f32(x, (E, K))
    dbias = None if bias is None else _f32(x, (E,))
    workspace = _workspace(workspace,
                           _function("rlca_causal_conv_workspace_bytes")(N, T, E, K), x)
    _run("rlca_causal_conv_backward", suffix, dev, p,
         Steps(*_steps(dout, "dout", dtype, dev, x.shape)),
         Steps(*_steps(dx, "dx", dtype, dev, x.shape)), dweight.data_ptr(),
         None if dbias is None else dbias.data_ptr(), *_ws(workspace))
    return dx, dweight, dbias


def causal_conv_step(x, state, weight, bias=None, reset=None, silu=True, out=None,
                     new_state=None):
    """One step of N rows: x [N, E], state [N, K-1, E]; returns (out, new_state). The state
    is updated in place unless new_state is given."""
    suffix, dev, dtype = _suffix_of(x, "x"), x.get_device(), x.dtype
    p, (N, _, _, _), states = _conv(x, dev, weight, bias, _NO_ROWS, state, silu, 1)
    new_state = state if new_state is None else new_state
    out = _out(out, x.shape, x)
    _run("rlca_causal_conv_step", suffix, dev, p, _reset(reset, dev, N),
         Steps(*_steps(out, "out", dtype, dev, x.shape, 1)),
         _flat(new_state, "new_state", dev, states, dtype))
    return out, new_state


# ------------------------------------------------------------------------ token embedding


def _tokens(tokens, dev):
    if tokens.dtype is not torch.int64 and tokens.dtype is not torch.int32:
        raise TypeError("tokens must be int32 or int64")
    if tokens.get_device() != dev:
        raise ValueError(f"tokens must be on cuda:{dev}")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return tokens.data_ptr(), tokens.element_size()


def _matrix(t, name, M, D):
    """Pointer and row stride of a tensor [..., D] seen as [M, D]."""
    if t.is_contiguous():
        return t.data_ptr(), D
    if D > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: channels must be contiguous (unit stride)")
    if M <= 1 or t.dim() == 1:
        return t.data_ptr(), D
    ld, size = None, 1
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * size:
            raise ValueError(f"{name}: rows must lie at one stride")
        size *= n
    return t.data_ptr(), D if ld is None else ld


def embed_tokens(tokens, table, scale=1.0, out=None):
    """scale * table[tokens] (rlca_embed_tokens) for int32 / int64 tokens of any shape; a
    token outside the table gives a row of zeros."""
    if table.dim() != 2:
        raise ValueError("table must be [V, D]")
    suffix, dev = _suffix_of(table, "table"), table.get_device()
    V, D = table.shape
    M = tokens.numel()
    tok = _tokens(tokens, dev)
    shape = tokens.shape + (D,)
    if out is None:
        out = table.new_empty(shape)
    elif out.dtype is not table.dtype or out.get_device() != dev or out.shape != shape:
        _refuse(out, "out", (table.dtype,), dev, shape)
    _run("rlca_embed_tokens", suffix, dev, *tok, *_matrix(table, "table", V, D), scale, M, V,
         D, *_matrix(out, "out", M, D))
    return out


def embed_tokens_backward(dout, tokens, vocab, scale=1.0, dtable=None, workspace=None):
    """The table's gradient [vocab, D] in float32, every row written: scale times the sum of
    dout over the positions of each token."""
    suffix, dev = _suffix_of(dout, "dout"), dout.get_device()
    D, M = dout.shape[-1], tokens.numel()
    if dout.shape[:-1] != tokens.shape:
        raise ValueError(f"dout: shape {tuple(dout.shape)} does not fit tokens "
                         f"{tuple(tokens.shape)}")
    tok = _tokens(tokens, dev)
    if dtable is None:
        dtable = _f32(dout, (vocab, D))
    src = _matrix(dout, "dout", M, D)
    workspace = _workspace(workspace,
                           _function("rlca_embed_tokens_workspace_bytes")(M, vocab, D), dout)
    _run("rlca_embed_tokens_backward", suffix, dev, *src, *tok, scale, M, vocab, D,
         _flat(dtable, "dtable", dev, (vocab, D)), *_ws(workspace))
    return dtable
