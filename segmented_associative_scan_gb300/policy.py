"""Binding of the losses over a vocabulary of librlca (``include/rlca_policy.h``): token
log-probabilities, the clipped policy loss with its KL term, the preference loss of pairs and
the distillation from a teacher's top logits, each with its gradient.

Argument marshalling only, like the rest of the package. Logits are CUDA tensors [N, T, V] of
one data type (float32, bfloat16 or float16), or [N, V] for one step of N rows, unit stride
over the vocabulary, any stride over rows and steps; tokens are int32 or int64, values per step
float32, both [N, T] ([N]) with unit stride over the steps. A step whose token lies outside the
vocabulary or which lies past its row's length (`lengths`, int32 [N]) does not count: its
outputs and gradients are 0. Outputs are allocated unless passed in; work is enqueued on the
current stream and nothing synchronises.

The calls build no autograd graph, like the estimators': gradients come from calls of their own
(``*_backward``), or, where one read of the logits gives both, with the loss (`want_grad`).
`dlogits` may be the logits themselves, which it then replaces.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from .sequence import (_F, _I32, _I64, _NO_STEPS, _P, _STEPS, Steps, _flat, _refuse, _run,
                       _steps, _suffix_of)

_LINE = "Pq"
_NO_LINE = (0, 0)


class Line(ctypes.Structure):
    _fields_ = [("ptr", _P), ("ld", _I64)]


class Choices(ctypes.Structure):
    _fields_ = [("N", _I64), ("T", _I64), ("V", _I64), ("logits", Steps), ("tokens", _P),
                ("token_ld", _I64), ("lengths", _P), ("token_bytes", _I32), ("temperature", _F)]


class Policy(ctypes.Structure):
    _fields_ = [("old_logp", Line), ("advantage", Line), ("ref_logp", Line), ("weight", Line),
                ("clip_low", _F), ("clip_high", _F), ("kl_coef", _F), ("entropy_coef", _F),
                ("loss", _P), ("logp", _P), ("entropy", _P), ("kl", _P), ("dlogits", Steps)]


class Preference(ctypes.Structure):
    _fields_ = [("ref_logp", Line), ("beta", _F), ("smoothing", _F), ("by_length", _I32),
                ("loss", _P), ("scores", _P), ("logp", _P), ("saved", _P), ("slope", _P)]


class Distill(ctypes.Structure):
    _fields_ = [("K", _I64), ("index", Steps), ("teacher", Steps), ("index_bytes", _I32),
                ("teacher_fp32", _I32), ("weight", Line), ("loss", _P), ("dlogits", Steps)]


_PACK_CHOICES = struct.Struct("@3q" + _STEPS + "PqPif").pack
_PACK_POLICY = struct.Struct("@" + 4 * _LINE + "4fPPPP" + _STEPS).pack
_PACK_PREFERENCE = struct.Struct("@" + _LINE + "ffi4xPPPPP").pack
_PACK_DISTILL = struct.Struct("@q" + 2 * _STEPS + "ii" + _LINE + "P" + _STEPS).pack

SIGNATURES = {}
for _suffix in ("", "_bf16", "_fp16"):
    SIGNATURES["rlca_token_logprobs" + _suffix] = ([_P, _P, _P, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_token_logprobs_backward" + _suffix] = (
        [_P, Line, Line, _P, _P, Steps, _P], ctypes.c_int)
    SIGNATURES["rlca_policy_loss" + _suffix] = ([_P, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_preference_loss" + _suffix] = ([_P, _P, _P], ctypes.c_int)
    SIGNATURES["rlca_preference_loss_backward" + _suffix] = (
        [_P, _P, _P, _P, Steps, _P], ctypes.c_int)
    SIGNATURES["rlca_distill_topk" + _suffix] = ([_P, _P, _P], ctypes.c_int)

_F32 = (torch.float32,)
_INDEX = (torch.int32, torch.int64)


def _line(t, name, dtypes, dev, shape):
    """(pointer, row stride) of one value per step, (0, 0) for None."""
    if t is None:
        return _NO_LINE
    if t.dtype not in dtypes or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, dtypes, dev, shape)
    s = t.stride()
    if len(s) == 1:  # one step of each row
        return t.data_ptr(), s[0] if shape[0] > 1 else 1
    if shape[1] > 1 and s[1] != 1:
        raise ValueError(f"{name}: steps must be contiguous (stride(1) == 1)")
    return t.data_ptr(), s[0] if shape[0] > 1 else shape[1]


def _choices(logits, tokens, lengths, temperature):
    """The packed rlca_choices of a call, its suffix, device, the shape of a value per step and
    the number of leading dimensions."""
    suffix, dev = _suffix_of(logits, "logits"), logits.get_device()
    shape = logits.shape
    lead = len(shape) - 1
    if lead != 2 and lead != 1:
        raise ValueError("logits must be [N, T, V], or [N, V] for one step")
    if shape[-1] == 0:
        raise ValueError("logits must have a vocabulary (V >= 1)")
    rows = shape[:-1]
    if tokens is None:
        ptr, ld, size = 0, 0, 8
    else:
        ptr, ld = _line(tokens, "tokens", _INDEX, dev, rows)
        size = tokens.element_size()
    N, T = rows[0], rows[1] if lead == 2 else 1
    packed = _PACK_CHOICES(N, T, shape[-1],
                           *_steps(logits, "logits", logits.dtype, dev, shape, lead), ptr, ld,
                           _flat(lengths, "lengths", dev, (N,), torch.int32), size, temperature)
    return packed, suffix, dev, rows, lead


def _gradient(dlogits, want, logits, dev, lead):
    """The gradient's tensor (None: not wanted) and its steps."""
    if dlogits is None:
        if not want:
            return None, _NO_STEPS
        shape = logits.shape
        dlogits = torch.empty(shape, dtype=logits.dtype, device=logits.device)
        V = shape[-1]
        return dlogits, (dlogits.data_ptr(), shape[1] * V if lead == 2 else V,
                         V if lead == 2 else 0)
    return dlogits, _steps(dlogits, "dlogits", logits.dtype, dev, logits.shape, lead)


def _scalar(t, name, want, device, dev, shape):
    """An fp32 result (None: not wanted) and its pointer; one that is allocated here needs no
    check."""
    if t is not None:
        return t, _flat(t, name, dev, shape)
    if not want:
        return None, 0
    t = torch.empty(shape, dtype=torch.float32, device=device)
    return t, t.data_ptr()


# ------------------------------------------------------------- token log-probabilities


def token_logprobs(logits, tokens, lengths=None, temperature=1.0, want_entropy=False,
                   want_saved=False, logp=None, entropy=None, saved=None):
    """log softmax(logits / temperature)[token] of every step (rlca_token_logprobs): returns
    (logp, entropy, saved), the last two None unless wanted. `saved` is what
    `token_logprobs_backward` reads."""
    p, suffix, dev, rows, _ = _choices(logits, tokens, lengths, temperature)
    device = logits.device
    logp, to = _scalar(logp, "logp", True, device, dev, rows)
    entropy, to_entropy = _scalar(entropy, "entropy", want_entropy, device, dev, rows)
    saved, to_saved = _scalar(saved, "saved", want_saved, device, dev, rows + (2,))
    _run("rlca_token_logprobs", suffix, dev, p, to, to_entropy, to_saved)
    return logp, entropy, saved


def token_logprobs_backward(dlogp, logits, tokens, saved, lengths=None, temperature=1.0,
                            entropy=None, dentropy=None, dlogits=None):
    """Gradient of sum(logp * dlogp) + sum(entropy * dentropy) by the logits. dlogp may be None;
    dentropy needs the `entropy` of the forward call."""
    p, suffix, dev, rows, lead = _choices(logits, tokens, lengths, temperature)
    dlogits, steps = _gradient(dlogits, True, logits, dev, lead)
    _run("rlca_token_logprobs_backward", suffix, dev, p,
         Line(*_line(dlogp, "dlogp", _F32, dev, rows)),
         Line(*_line(dentropy, "dentropy", _F32, dev, rows)),
         _flat(entropy, "entropy", dev, rows), _flat(saved, "saved", dev, rows + (2,)),
         Steps(*steps))
    return dlogits


# --------------------------------------------------------------------- clipped policy loss


def policy_loss(logits, tokens, old_logp, advantages, ref_logp=None, weight=None, lengths=None,
                clip_low=0.2, clip_high=0.2, kl_coef=0.0, entropy_coef=0.0, temperature=1.0,
                want_entropy=False, want_grad=False, loss=None, logp=None, entropy=None, kl=None,
                dlogits=None):
    """Clipped policy loss of every step (rlca_policy_loss): returns (loss, logp, entropy, kl,
    dlogits); entropy and dlogits None unless wanted, kl None without ref_logp. dlogits is the
    gradient of sum(weight * loss) (weight None: 1)."""
    p, suffix, dev, rows, lead = _choices(logits, tokens, lengths, temperature)
    device = logits.device
    loss, to = _scalar(loss, "loss", True, device, dev, rows)
    logp, to_logp = _scalar(logp, "logp", True, device, dev, rows)
    entropy, to_entropy = _scalar(entropy, "entropy", want_entropy, device, dev, rows)
    kl, to_kl = _scalar(kl, "kl", ref_logp is not None, device, dev, rows)
    dlogits, steps = _gradient(dlogits, want_grad, logits, dev, lead)
    q = _PACK_POLICY(*_line(old_logp, "old_logp", _F32, dev, rows),
                     *_line(advantages, "advantages", _F32, dev, rows),
                     *_line(ref_logp, "ref_logp", _F32, dev, rows),
                     *_line(weight, "weight", _F32, dev, rows), clip_low, clip_high, kl_coef,
                     entropy_coef, to, to_logp, to_entropy, to_kl, *steps)
    _run("rlca_policy_loss", suffix, dev, p, q)
    return loss, logp, entropy, kl, dlogits


# ------------------------------------------------------------------------ preference loss


def _pairs_saved(rows):
    return (2 * rows.numel() + rows[0],)


def preference_loss(logits, tokens, ref_logp=None, lengths=None, beta=0.1, smoothing=0.0,
                    by_length=False, temperature=1.0, want_saved=False, loss=None, scores=None,
                    logp=None):
    """Preference loss of N / 2 pairs (rlca_preference_loss): rows n and N / 2 + n are the
    preferred and the other answer of pair n. Returns (loss [N / 2], scores [N], logp, saved);
    `saved` (want_saved) is what `preference_loss_backward` reads."""
    p, suffix, dev, rows, _ = _choices(logits, tokens, lengths, temperature)
    N, device = rows[0], logits.device
    loss, to = _scalar(loss, "loss", True, device, dev, (N // 2,))
    scores, to_scores = _scalar(scores, "scores", True, device, dev, (N,))
    logp, to_logp = _scalar(logp, "logp", True, device, dev, rows)
    # (a logit at or near the largest, the sum relative to it) of every step, and behind them the slope
    # of every row.
    saved, to_saved = _scalar(None, "saved", True, device, dev, _pairs_saved(rows))
    q = _PACK_PREFERENCE(*_line(ref_logp, "ref_logp", _F32, dev, rows), beta, smoothing,
                         1 if by_length else 0, to, to_scores, to_logp, to_saved,
                         to_saved + 8 * rows.numel() if want_saved else 0)
    _run("rlca_preference_loss", suffix, dev, p, q)
    return loss, scores, logp, saved if want_saved else None


def preference_loss_backward(dloss, logits, tokens, saved, lengths=None, temperature=1.0,
                             dlogits=None):
    """Gradient of sum(loss * dloss) by the logits; dloss [N / 2], or None for ones."""
    p, suffix, dev, rows, lead = _choices(logits, tokens, lengths, temperature)
    stats = _flat(saved, "saved", dev, _pairs_saved(rows))
    dlogits, steps = _gradient(dlogits, True, logits, dev, lead)
    _run("rlca_preference_loss_backward", suffix, dev, p,
         _flat(dloss, "dloss", dev, (rows[0] // 2,)), stats + 8 * rows.numel(), stats,
         Steps(*steps))
    return dlogits


# --------------------------------------------------------------------------- distillation


def distill_topk(logits, teacher_index, teacher_logits, weight=None, lengths=None,
                 temperature=1.0, want_grad=False, loss=None, dlogits=None):
    """Distillation from a teacher's K largest logits (rlca_distill_topk): teacher_index int32 /
    int64 and teacher_logits (float32 or the logits' type) [N, T, K]. Returns (loss, dlogits);
    dlogits (want_grad) is the gradient of sum(weight * loss) (weight None: 1)."""
    p, suffix, dev, rows, lead = _choices(logits, None, lengths, temperature)
    shape, dtype = teacher_index.shape, teacher_logits.dtype
    if len(shape) != lead + 1 or shape[:-1] != rows:
        raise ValueError(f"teacher_index: shape {tuple(shape)} does not fit logits "
                         f"{tuple(logits.shape)}")
    if teacher_index.dtype not in _INDEX:
        raise TypeError("teacher_index must be int32 or int64")
    if dtype is not torch.float32 and dtype is not logits.dtype:
        raise TypeError("teacher_logits must be float32 or of the logits' type")
    loss, to = _scalar(loss, "loss", True, logits.device, dev, rows)
    dlogits, steps = _gradient(dlogits, want_grad, logits, dev, lead)
    q = _PACK_DISTILL(shape[-1],
                      *_steps(teacher_index, "teacher_index", teacher_index.dtype, dev, shape,
                              lead),
                      *_steps(teacher_logits, "teacher_logits", dtype, dev, shape, lead),
                      teacher_index.element_size(), 1 if dtype is torch.float32 else 0,
                      *_line(weight, "weight", _F32, dev, rows), to, *steps)
    _run("rlca_distill_topk", suffix, dev, p, q)
    return loss, dlogits
