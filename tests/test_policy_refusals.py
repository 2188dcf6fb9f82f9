"""The losses' entry points reject bad arguments on the host with the documented status codes
before any CUDA call (no GPU needed; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import segmented_associative_scan_gb300 as rlca
from segmented_associative_scan_gb300 import policy as pol
from segmented_associative_scan_gb300.sequence import Steps

OK, NULL, SHAPE, PARAM, ALIAS, MEMORY = 0, -1, -2, -3, -4, -8
N, T, V, K = 4, 16, 100, 8
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    rlca.build()
    return rlca.lib()


def fake(i):
    return 0x100000000 + i * 0x1000000


def steps(i, width=V):
    return Steps(None if i is None else fake(i), T * width, width)


def line(i, ld=T):
    return pol.Line(None if i is None else fake(i), ld)


def make(struct, defaults, kw):
    return struct(*({**defaults, **kw}[k] for k, _ in struct._fields_))


def choices(**kw):
    return make(pol.Choices, dict(N=N, T=T, V=V, logits=steps(1), tokens=fake(2), token_ld=T,
                                  lengths=fake(3), token_bytes=8, temperature=1.0), kw)


BAD_SHAPES = [dict(N=-1), dict(T=-1), dict(V=0), dict(V=-1), dict(V=(1 << 30) + 1), dict(T=(1 << 30) + 1),
              dict(N=1 << 40, T=1 << 20), dict(N=1 << 20, T=1 << 11, V=1), dict(token_bytes=2), dict(token_ld=-1),
              dict(logits=Steps(fake(1), -1, V))]
BAD_TEMPERATURES = [0.0, -1.0, 0.9e-6, 1.1e6, NAN, INF]


def check_choices(f):
    """What every entry point refuses of its logits and tokens."""
    for kw in BAD_SHAPES:
        assert f(**kw) == SHAPE, kw
    for t in BAD_TEMPERATURES:
        assert f(temperature=t) == PARAM, t
    assert f(logits=steps(None)) == NULL and f(tokens=None) == NULL
    assert f(logits=Steps(fake(1) + 1, T * V, V)) == MEMORY
    assert f(tokens=fake(2) + 4) == MEMORY
    assert f(N=0, logits=steps(None), tokens=None) == OK


def test_token_logprobs(lib):
    def f(logp=fake(4), entropy=fake(5), saved=fake(6), **kw):
        return lib.rlca_token_logprobs_bf16(ctypes.byref(choices(**kw)), logp, entropy, saved, None)
    check_choices(f)
    assert f(T=0, logits=steps(None), logp=None) == OK
    assert f(logp=None) == NULL and lib.rlca_token_logprobs(None, None, None, None, None) == NULL
    assert f(logp=fake(1)) == ALIAS and f(entropy=fake(2)) == ALIAS and f(saved=fake(3)) == ALIAS
    assert f(logp=fake(5) + 4 * N * T - 4) == ALIAS or f(entropy=fake(4) + 4) == ALIAS
    assert f(saved=fake(6) + 4) == MEMORY and f(logp=fake(4) + 2) == MEMORY


def test_token_logprobs_backward(lib):
    def f(dlogp=line(4), dentropy=line(5), entropy=fake(6), saved=fake(7), dlogits=steps(8), **kw):
        return lib.rlca_token_logprobs_backward_fp16(ctypes.byref(choices(**kw)), dlogp, dentropy,
                                                     entropy, saved, dlogits, None)
    check_choices(f)
    assert f(saved=None) == NULL and f(entropy=None) == NULL and f(dlogits=steps(None)) == NULL
    assert f(dlogp=line(4, -1)) == SHAPE and f(dlogits=Steps(fake(8), T * V, V - 1)) == SHAPE
    assert f(dlogits=steps(7)) == ALIAS and f(dlogits=steps(4)) == ALIAS
    # Exactly the logits, and no other overlap with them.
    assert f(dlogits=steps(1), saved=fake(7) + 4) == MEMORY
    assert f(dlogits=Steps(fake(1) + 2, T * V, V)) == ALIAS
    assert f(dlogits=Steps(fake(1), T * V + 8, V)) == ALIAS
    assert f(logits=Steps(fake(1), 0, V), dlogits=steps(1)) == ALIAS
    assert f(dlogits=steps(1), dlogp=line(1)) == ALIAS
    assert f(saved=fake(7) + 4) == MEMORY


def policy(**kw):
    return make(pol.Policy, dict(old_logp=line(10), advantage=line(11), ref_logp=line(12),
                                 weight=line(13), clip_low=0.2, clip_high=0.2, kl_coef=0.1,
                                 entropy_coef=0.1, loss=fake(14), logp=fake(15), entropy=fake(16),
                                 kl=fake(17), dlogits=steps(18)), kw)


def test_policy_loss(lib):
    def f(q=None, **kw):
        return lib.rlca_policy_loss(ctypes.byref(choices(**kw)), ctypes.byref(policy(**(q or {}))),
                                    None)
    check_choices(f)
    assert lib.rlca_policy_loss(None, None, None) == NULL
    for k in ("old_logp", "advantage"):
        assert f({k: line(None)}) == NULL, k
        assert f({k: line(10, -1)}) == SHAPE, k
    assert f(dict(loss=None)) == NULL
    # A KL term, or its values, without a reference.
    assert f(dict(ref_logp=line(None))) == NULL
    assert f(dict(ref_logp=line(None), kl=None)) == NULL
    assert f(dict(ref_logp=line(None), kl_coef=0.0)) == NULL
    for k, bad in (("clip_low", (-0.1, 1.1, NAN)), ("clip_high", (-0.1, NAN, INF)),
                   ("kl_coef", (-0.1, NAN, INF)), ("entropy_coef", (NAN, INF))):
        for v in bad:
            assert f({k: v}) == PARAM, (k, v)
    for k in ("loss", "logp", "entropy", "kl"):
        assert f({k: fake(1)}) == ALIAS and f({k: fake(10)}) == ALIAS, k
        assert f({k: fake(18) + 64}) == ALIAS, k
    assert f(dict(dlogits=steps(13))) == ALIAS
    assert f(dict(dlogits=Steps(fake(18), V, 0))) == SHAPE
    assert f(dict(dlogits=Steps(fake(1), T * V, V), loss=fake(14) + 2)) == MEMORY
    assert f(dict(loss=fake(1), dlogits=steps(1))) == ALIAS


def preference(**kw):
    return make(pol.Preference, dict(ref_logp=line(10), beta=0.1, smoothing=0.1, by_length=0,
                                     loss=fake(11), scores=fake(12), logp=fake(13), saved=fake(14),
                                     slope=fake(15)), kw)


def test_preference_loss(lib):
    def f(q=None, **kw):
        return lib.rlca_preference_loss_bf16(ctypes.byref(choices(**kw)),
                                             ctypes.byref(preference(**(q or {}))), None)
    check_choices(f)
    assert f(N=5) == SHAPE
    for k, bad in (("beta", (0.0, -1.0, NAN, INF)), ("smoothing", (-0.1, 1.1, NAN))):
        for v in bad:
            assert f({k: v}) == PARAM, (k, v)
    for k in ("loss", "scores", "logp", "saved"):
        assert f({k: None}) == NULL, k
    assert f(dict(ref_logp=line(10, -2))) == SHAPE
    assert f(dict(scores=fake(10))) == ALIAS and f(dict(loss=fake(12))) == ALIAS
    assert f(dict(saved=fake(14) + 4)) == MEMORY
    assert f(T=0, q=dict(loss=None)) == NULL  # pairs have a loss without any steps

    def b(dloss=fake(20), slope=fake(15), saved=fake(14), dlogits=steps(21), **kw):
        return lib.rlca_preference_loss_backward(ctypes.byref(choices(**kw)), dloss, slope, saved,
                                                 dlogits, None)
    check_choices(b)
    assert b(N=3) == SHAPE
    assert b(slope=None) == NULL and b(saved=None) == NULL and b(dlogits=steps(None)) == NULL
    assert b(dlogits=steps(14)) == ALIAS and b(saved=fake(14) + 4) == MEMORY


def distill(**kw):
    return make(pol.Distill, dict(K=K, index=steps(10, K), teacher=steps(11, K), index_bytes=8,
                                  teacher_fp32=1, weight=line(12), loss=fake(13),
                                  dlogits=steps(14)), kw)


def test_distill_topk(lib):
    def f(q=None, **kw):
        return lib.rlca_distill_topk_fp16(ctypes.byref(choices(**{"tokens": None, **kw})),
                                          ctypes.byref(distill(**(q or {}))), None)
    for kw in BAD_SHAPES[:8] + BAD_SHAPES[10:]:
        assert f(**kw) == SHAPE, kw
    for t in BAD_TEMPERATURES:
        assert f(temperature=t) == PARAM, t
    for k, bad in (("K", (-1, 257)), ("index_bytes", (2, 0))):
        for v in bad:
            assert f({k: v}) == SHAPE, (k, v)
    assert f(dict(index=steps(None))) == NULL and f(dict(teacher=steps(None))) == NULL
    assert f(dict(loss=None)) == NULL and f(logits=steps(None)) == NULL
    assert f(dict(loss=fake(10))) == ALIAS and f(dict(dlogits=steps(11))) == ALIAS
    assert f(dict(teacher=Steps(fake(11) + 2, T * K, K))) == MEMORY
    assert f(dict(index=Steps(fake(10) + 4, T * K, K))) == MEMORY
    assert f(dict(index=Steps(fake(10), -1, K))) == SHAPE
    assert f(N=0) == OK and f(T=0) == OK


def test_binding_refuses_other_devices_types_and_shapes():
    z, tok, s = torch.zeros(2, 3, 4), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    with pytest.raises(ValueError):
        rlca.token_logprobs(z, tok)
    with pytest.raises(TypeError):
        rlca.policy_loss(z.double(), tok, s, s)
    with pytest.raises(ValueError):
        rlca.preference_loss(z, tok)
    with pytest.raises(TypeError):
        rlca.distill_topk(z.int(), tok, s)


def test_structs_as_they_are_packed():
    """The packed forms are the structures of the header, byte for byte."""
    got = pol._PACK_CHOICES(1, 2, 3, 4, 5, 6, 7, 8, 9, 4, 0.5)
    want = pol.Choices(1, 2, 3, Steps(4, 5, 6), 7, 8, 9, 4, 0.5)
    assert got == bytes(want)
    got = pol._PACK_POLICY(1, 2, 3, 4, 5, 6, 7, 8, 0.1, 0.2, 0.3, 0.4, 9, 10, 11, 12, 13, 14, 15)
    want = pol.Policy(pol.Line(1, 2), pol.Line(3, 4), pol.Line(5, 6), pol.Line(7, 8), 0.1, 0.2, 0.3,
                      0.4, 9, 10, 11, 12, Steps(13, 14, 15))
    assert got == bytes(want)
    got = pol._PACK_PREFERENCE(1, 2, 0.5, 0.25, 1, 3, 4, 5, 6, 7)
    want = pol.Preference(pol.Line(1, 2), 0.5, 0.25, 1, 3, 4, 5, 6, 7)
    assert got == bytes(want)
    got = pol._PACK_DISTILL(1, 2, 3, 4, 5, 6, 7, 8, 1, 9, 10, 11, 12, 13, 14)
    want = pol.Distill(1, Steps(2, 3, 4), Steps(5, 6, 7), 8, 1, pol.Line(9, 10), 11,
                       Steps(12, 13, 14))
    assert got == bytes(want)
