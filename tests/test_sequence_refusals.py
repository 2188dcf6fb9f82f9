"""The sequence-model entry points reject bad arguments on the host with the documented
status codes before any CUDA call (no GPU needed; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import segmented_associative_scan_gb300 as rlca
from segmented_associative_scan_gb300 import sequence as seq

OK, NULL, SHAPE, ALIAS, WORKSPACE = 0, -1, -2, -4, -5


@pytest.fixture(scope="module")
def lib():
    rlca.build()
    return rlca.lib()


def fake(i):
    return 0x100000000 + i * 0x1000000


def steps(i, row=64 * 32, step=32):
    return seq.Steps(None if i is None else fake(i), row, step)


def scan(**kw):
    v = dict(N=4, T=64, E=32, S=16, G=1, x=steps(1), dt=steps(2), z=steps(3),
             B=steps(4, 64 * 16, 16), C=steps(5, 64 * 16, 16), A=fake(6), D=fake(7),
             dt_bias=fake(8), rows=seq.Rows(fake(9), fake(10), 64, fake(11)),
             init_state=fake(12), dt_softplus=1)
    v.update(kw)
    return seq.Scan(*(v[k] for k, _ in seq.Scan._fields_))


def run_scan(lib, out=None, final=fake(14), saved=fake(15), **kw):
    return lib.rlca_selective_scan_bf16(ctypes.byref(scan(**kw)),
                                        steps(13) if out is None else out, final, saved,
                                        fake(40), 1 << 20, None)


def test_scan_shapes_and_nulls(lib):
    for kw in (dict(N=-1), dict(T=-1), dict(E=-1), dict(S=0), dict(S=65), dict(G=0), dict(G=3),
               dict(T=(1 << 30) + 1), dict(N=1 << 40, T=1 << 20),
               dict(x=steps(1, -1)), dict(rows=seq.Rows(fake(9), None, 63, None))):
        assert run_scan(lib, **kw) == SHAPE, kw
    for k in ("x", "dt", "B", "C"):
        assert run_scan(lib, **{k: steps(None)}) == NULL, k
    assert run_scan(lib, A=None) == NULL
    assert run_scan(lib, out=steps(None)) == NULL
    assert lib.rlca_selective_scan(None, steps(1), None, None, None, 0, None) == NULL
    assert run_scan(lib, N=0, x=steps(None)) == OK
    # Outputs whose elements would share addresses.
    assert run_scan(lib, out=steps(13, 64 * 32, 31)) == SHAPE
    assert run_scan(lib, out=steps(13, 32, 0)) == SHAPE


def test_scan_aliases(lib):
    for i in (1, 2, 3, 4, 5):
        assert run_scan(lib, out=steps(i)) == ALIAS
    assert run_scan(lib, final=fake(6)) == ALIAS
    assert run_scan(lib, final=fake(12)) == ALIAS   # a window's states are not updated in place
    assert run_scan(lib, saved=fake(14)) == ALIAS
    assert run_scan(lib, saved=fake(9) - 16) == ALIAS
    # Overlap inside one stride, and slices that touch.
    wide = lambda off: seq.Steps(fake(20) + 2 * off, 64 * 64, 64)
    assert run_scan(lib, x=wide(0), out=wide(31)) == ALIAS
    assert run_scan(lib, x=wide(32), out=wide(1)) == ALIAS


def run_backward(lib, ws=fake(40), ws_bytes=1 << 24, problem=None, **kw):
    v = dict(dout=steps(20), d_final_state=fake(21), saved=fake(22), dx=steps(23),
             ddt=steps(24), dz=steps(25), dB=steps(26, 64 * 16, 16), dC=steps(27, 64 * 16, 16),
             dA=fake(28), dD=fake(29), ddt_bias=fake(30), d_init_state=fake(31))
    v.update(kw)
    g = seq.ScanGrads(*(v[k] for k, _ in seq.ScanGrads._fields_))
    return lib.rlca_selective_scan_backward(ctypes.byref(scan(**(problem or {}))),
                                            ctypes.byref(g), ws, ws_bytes, None)


def test_scan_backward_refusals(lib):
    for k in ("dout", "dx", "ddt", "dz", "dB", "dC"):
        assert run_backward(lib, **{k: steps(None)}) == NULL, k
    for k in ("saved", "dA"):
        assert run_backward(lib, **{k: None}) == NULL, k
    assert run_backward(lib, dx=steps(24)) == ALIAS
    assert run_backward(lib, dC=steps(26, 64 * 16, 16)) == ALIAS
    assert run_backward(lib, dA=fake(22)) == ALIAS
    need = lib.rlca_selective_scan_workspace_bytes(4, 64, 32, 16, 1)
    assert need > 0
    assert run_backward(lib, ws_bytes=need - 1) == WORKSPACE
    assert run_backward(lib, ws=None) == WORKSPACE
    assert run_backward(lib, ws=fake(40) + 16) == WORKSPACE
    assert run_backward(lib, ws=fake(23)) == ALIAS
    assert lib.rlca_selective_scan_backward(None, None, None, 0, None) == NULL
    assert lib.rlca_selective_scan_workspace_bytes(-1, 64, 32, 16, 1) == 0
    assert lib.rlca_selective_scan_saved_bytes(4, 65, 32, 16) == 4 * 4 * 9 * 32 * 16


def test_scan_step_refusals(lib):
    def f(new=fake(14), out=None, **kw):
        return lib.rlca_selective_scan_step(ctypes.byref(scan(**{"T": 1, **kw})), fake(9),
                                            out or steps(13), new, None)
    assert f(T=2) == SHAPE and f(S=0) == SHAPE
    assert f(new=None) == NULL and f(x=steps(None)) == NULL
    assert f(new=fake(12) + 64) == ALIAS  # part of the state, not all of it
    assert f(out=steps(1)) == ALIAS
    assert f(N=0) == OK


def conv(**kw):
    v = dict(N=4, T=64, E=32, K=4, x=steps(1), weight=fake(2), bias=fake(3),
             rows=seq.Rows(fake(4), fake(5), 64, fake(6)), init_state=fake(7), silu=1)
    v.update(kw)
    return seq.Conv(*(v[k] for k, _ in seq.Conv._fields_))


def test_conv_refusals(lib):
    f = lambda out=None, final=fake(9), **kw: lib.rlca_causal_conv(
        ctypes.byref(conv(**kw)), out or steps(8), final, None)
    for kw in (dict(K=0), dict(K=9), dict(N=-1), dict(T=-1), dict(E=-1),
               dict(x=steps(1, 5, -1)), dict(out=steps(8, 31, 31))):
        assert f(**kw) == SHAPE, kw
    assert f(x=steps(None)) == NULL and f(weight=None) == NULL and f(out=steps(None)) == NULL
    assert f(out=steps(1)) == ALIAS and f(final=fake(7)) == ALIAS
    assert f(N=0) == OK and f(E=0) == OK
    b = lambda ws=fake(20), n=1 << 24, dw=fake(12), dx=None, **kw: \
        lib.rlca_causal_conv_backward(ctypes.byref(conv(**kw)), steps(10), dx or steps(11), dw,
                                      fake(13), ws, n, None)
    assert b(dw=None) == NULL and b(dx=steps(None)) == NULL
    assert b(dx=steps(10)) == ALIAS
    need = lib.rlca_causal_conv_workspace_bytes(4, 64, 32, 4)
    assert b(n=need - 1) == WORKSPACE and b(ws=None) == WORKSPACE and b(ws=fake(11)) == ALIAS
    s = lambda new=fake(9), **kw: lib.rlca_causal_conv_step(
        ctypes.byref(conv(**{"T": 1, **kw})), None, steps(8), new, None)
    assert s(T=2) == SHAPE and s(new=None) == NULL and s(init_state=None) == NULL
    assert s(new=fake(7) + 4) == ALIAS


def test_embedding_refusals(lib):
    f = lambda tok=fake(1), tb=8, table=fake(2), ld=32, M=100, V=50, D=32, out=fake(3), \
        old=32: lib.rlca_embed_tokens(tok, tb, table, ld, 1.0, M, V, D, out, old, None)
    assert f(tb=2) == SHAPE and f(ld=31) == SHAPE and f(old=31) == SHAPE
    assert f(M=-1) == SHAPE and f(V=-1) == SHAPE and f(D=-1) == SHAPE and f(M=1 << 31) == SHAPE
    assert f(tok=None) == NULL and f(table=None) == NULL and f(out=None) == NULL
    assert f(out=fake(2)) == ALIAS
    assert f(M=0) == OK and f(D=0, ld=0, old=0) == OK
    need = lib.rlca_embed_tokens_workspace_bytes(100, 50, 32)
    b = lambda dt=fake(3), ws=fake(5), n=need, tok=fake(1): lib.rlca_embed_tokens_backward_fp16(
        fake(4), 32, tok, 8, 1.0, 100, 50, 32, dt, ws, n, None)
    assert b(dt=None) == NULL and b(tok=None) == NULL and b(dt=fake(4)) == ALIAS
    assert b(n=need - 1) == WORKSPACE and b(ws=None) == WORKSPACE and b(ws=fake(3)) == ALIAS


def test_binding_refuses_other_devices_and_types():
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError):
        rlca.selective_scan(x, x, x, x, x)
    with pytest.raises(TypeError):
        rlca.causal_conv(x.double(), x)
    with pytest.raises(ValueError):
        rlca.embed_tokens(torch.zeros(2, dtype=torch.int64), torch.zeros(3, 4))


def test_misaligned_pointers(lib):
    MEMORY = -8
    off = lambda i, b: seq.Steps(fake(i) + b, 64 * 32, 32)
    assert run_scan(lib, x=off(1, 1)) == MEMORY            # bf16: 2-byte elements
    assert run_scan(lib, A=fake(6) + 2) == MEMORY          # fp32
    assert lib.rlca_causal_conv(ctypes.byref(conv(x=off(1, 2))), steps(8), fake(9),
                                None) == MEMORY
    assert lib.rlca_embed_tokens(fake(1) + 4, 8, fake(2), 32, 1.0, 100, 50, 32, fake(3), 32,
                                 None) == MEMORY


def test_only_the_state_may_be_the_new_state(lib):
    """An update in place is a pair of the state and its new value: another input at the same
    address is read while the state is overwritten."""
    def scan_step(**kw):
        return lib.rlca_selective_scan_step(ctypes.byref(scan(**{"T": 1, **kw})), None,
                                            steps(13), fake(12), None)

    for k in ("A", "D", "dt_bias"):
        assert scan_step(**{k: fake(12)}) == ALIAS, k
    for k in ("x", "dt", "z", "B", "C"):
        assert scan_step(**{k: steps(12)}) == ALIAS, k

    def conv_step(**kw):
        return lib.rlca_causal_conv_step(ctypes.byref(conv(**{"T": 1, **kw})), None, steps(8),
                                         fake(7), None)

    assert conv_step(x=steps(7)) == ALIAS
    assert conv_step(weight=fake(7)) == ALIAS and conv_step(bias=fake(7)) == ALIAS
    # The update in place itself is no alias (nor is a window of no inputs).
    assert scan_step() != ALIAS and conv_step() != ALIAS and conv_step(K=1) != ALIAS


def test_embedding_takes_every_size_below_two_to_the_31(lib):
    top = (1 << 31) - 1
    f = lambda M, V: lib.rlca_embed_tokens(fake(1), 4, None, 1, 1.0, M, V, 1, None, 1, None)
    assert f(top, 10) == NULL and f(10, top) == NULL
    assert f(top + 1, 10) == SHAPE and f(10, top + 1) == SHAPE
    assert lib.rlca_embed_tokens_workspace_bytes(top, top, 1) > 2 * 8 * top
