"""The router as operators of their own: selection with gates, the balance loss
with per-expert counts, and the gradient of both.

Argument marshalling like ``block.py``, whose conventions hold here too: CUDA
tensors of one device, that device's current stream or `stream`, no
synchronisation, :class:`MoeError` with MOE_ERR_INVALID_ARG for bad arguments,
gradients as calls of their own.  `score` is "sigmoid" or "softmax", as in a
layer's configuration.  idx may go on to ``sort_by_expert`` or ``w4_matvec``,
which take its -1 as dropped slots.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import SCORE_SIGMOID_BIAS, SCORE_SOFTMAX, _check, lib
from .block import DTYPES, _bad, _current, _device, _empty, _int32, _on, _p, _raw_stream, _rows

SCORES = {"sigmoid": SCORE_SIGMOID_BIAS, "softmax": SCORE_SOFTMAX}


class _SelectArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("ld_logits", C.c_int64)] + \
               [(n, C.c_void_p) for n in ("bias", "mask", "idx", "gates")] + \
               [(n, C.c_int32) for n in ("T", "E", "k", "dtype", "score_fn", "normalize")] + [("scale", C.c_float)]


class _BalanceLossArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("ld_logits", C.c_int64)] + \
               [(n, C.c_void_p) for n in ("idx", "sequences", "loss", "counts", "tokens", "workspace")] + \
               [("workspace_bytes", C.c_size_t)] + [(n, C.c_int32) for n in ("T", "E", "k", "S", "dtype", "score_fn")]


class _RouterBackwardArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("ld_logits", C.c_int64)] + \
               [(n, C.c_void_p) for n in ("idx", "d_gates", "d_loss", "counts", "tokens", "sequences", "d_logits")] + \
               [("ld_d_logits", C.c_int64)] + \
               [(n, C.c_int32) for n in ("T", "E", "k", "S", "dtype", "score_fn", "normalize")] + [("scale", C.c_float)]


def declare(L):
    """Argument types of the entry points below (called once, when libmoe is loaded)."""
    for name, args in (("moe_select", _SelectArgs), ("moe_balance_loss", _BalanceLossArgs),
                       ("moe_router_backward", _RouterBackwardArgs)):
        f = getattr(L, name)
        f.restype = C.c_int
        f.argtypes = [C.POINTER(args), C.c_void_p]
    L.moe_balance_loss_workspace_bytes.restype = C.c_size_t
    L.moe_balance_loss_workspace_bytes.argtypes = [C.c_int32, C.c_int32, C.c_int32]


def _score(score, what):
    if not isinstance(score, str) or score not in SCORES:
        _bad(what + ": score is 'sigmoid' or 'softmax'")
    return SCORES[score]


def _logits(logits, what):
    if logits.dim() != 2 or logits.shape[1] < 1:
        _bad(what + ": logits are [T][E]")
    T, E = logits.shape
    if E > 1024:
        _bad(what + ": at most 1024 experts")
    _int32(T, what)
    rows, ld = _rows(logits, what)
    return rows, ld, T, E


def _slots_of(idx, T, E, dev, what):
    if not isinstance(idx, torch.Tensor) or idx.dtype != torch.int32 or idx.dim() != 2 or idx.shape[0] != T \
            or not 1 <= idx.shape[1] <= min(32, E) or idx.get_device() != dev:
        _bad(what + ": idx is int32 [T][k], k up to 32 and the number of experts, on the same device")
    return idx.contiguous()


def _ints(t, shape, dev, name, what):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or tuple(t.shape) != shape or t.get_device() != dev:
        _bad(what + ": " + name)
    return t.contiguous()


def _floats(t, shape, dev, name, what):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != shape or t.get_device() != dev:
        _bad(what + ": " + name)
    return t.contiguous()


def _sequences(sequences, dev, what):
    """(contiguous offsets or None, their number of sequences)."""
    if sequences is None:
        return None, 1
    if not isinstance(sequences, torch.Tensor) or sequences.dtype != torch.int32 or sequences.dim() != 1 \
            or not 2 <= sequences.shape[0] <= 1 + (1 << 20) or sequences.get_device() != dev:
        _bad(what + ": sequences are int32 offsets [S + 1] on the same device")
    return sequences.contiguous(), sequences.shape[0] - 1


def select_experts(logits: torch.Tensor, k: int, *, bias: Optional[torch.Tensor] = None, score: str = "sigmoid",
                   normalize: bool = True, scale: float = 1.0, mask: Optional[torch.Tensor] = None, stream=None):
    """The k experts of each token of logits [T][E] and their gates (see
    moe_select): (idx int32 [T][k], gates float32 [T][k]), in descending order
    of the keys.  bias float32 [E] goes with sigmoid scores and into the keys
    only; mask bool [T] is False for tokens that are routed nowhere (idx -1,
    gate 0)."""
    what = "select_experts"
    dev = _device(logits, what)
    if dev != _current() or stream is not None:
        return _on(dev, stream, select_experts, logits, k, bias=bias, score=score, normalize=normalize, scale=scale, mask=mask)
    rows, ld, T, E = _logits(logits, what)
    kind, k = _score(score, what), int(k)
    if not 1 <= k <= min(32, E):
        _bad(what + ": 1 <= k <= 32 and the number of experts")
    if bias is not None:
        if kind != SCORE_SIGMOID_BIAS:
            _bad(what + ": a bias goes with sigmoid scores")
        bias = _floats(bias, (E,), dev, "bias is float32 [E] on the same device", what)
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype != torch.bool or tuple(mask.shape) != (T,) or mask.get_device() != dev:
            _bad(what + ": mask is bool [T] on the same device")
        mask = mask.contiguous()
    idx = _empty((T, k), dtype=torch.int32, device=logits.device)
    gates = _empty((T, k), dtype=torch.float32, device=logits.device)
    a = _SelectArgs(rows.data_ptr(), ld, _p(bias), _p(mask), idx.data_ptr(), gates.data_ptr(), T, E, k, DTYPES[rows.dtype],
                    kind, bool(normalize), scale)
    code = lib().moe_select(a, _raw_stream(dev))
    if code:
        _check(code, "moe_select")
    return idx, gates


def balance_loss(logits: torch.Tensor, idx: torch.Tensor, *, score: str = "sigmoid",
                 sequences: Optional[torch.Tensor] = None, stream=None):
    """Balance loss of each sequence and its experts' counts (see
    moe_balance_loss): (loss float32 [S], counts int32 [S][E], tokens int32
    [S]).  sequences: int32 offsets [S + 1] of their rows; None: one sequence of
    all rows."""
    what = "balance_loss"
    dev = _device(logits, what)
    if dev != _current() or stream is not None:
        return _on(dev, stream, balance_loss, logits, idx, score=score, sequences=sequences)
    rows, ld, T, E = _logits(logits, what)
    kind = _score(score, what)
    idx = _slots_of(idx, T, E, dev, what)
    seq, S = _sequences(sequences, dev, what)
    where = logits.device
    loss = _empty(S, dtype=torch.float32, device=where)
    counts = _empty((S, E), dtype=torch.int32, device=where)
    tokens = _empty(S, dtype=torch.int32, device=where)
    L = lib()
    size = L.moe_balance_loss_workspace_bytes(T, E, S)
    work = _empty(size, dtype=torch.uint8, device=where) if size else None
    a = _BalanceLossArgs(rows.data_ptr(), ld, idx.data_ptr(), _p(seq), loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(),
                         _p(work), size, T, E, idx.shape[1], S, DTYPES[rows.dtype], kind)
    code = L.moe_balance_loss(a, _raw_stream(dev))
    if code:
        _check(code, "moe_balance_loss")
    return loss, counts, tokens


def router_backward(logits: torch.Tensor, idx: torch.Tensor, *, d_gates: Optional[torch.Tensor] = None,
                    d_loss: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                    tokens: Optional[torch.Tensor] = None, sequences: Optional[torch.Tensor] = None,
                    score: str = "sigmoid", normalize: bool = True, scale: float = 1.0, stream=None) -> torch.Tensor:
    """Gradient of the logits, [T][E] of their type, from the gradients of
    select_experts' gates (d_gates float32 [T][k], with its score, normalize and
    scale), of balance_loss' losses (d_loss float32 [S], with the counts, tokens
    and sequences of that call), or of both; see moe_router_backward."""
    what = "router_backward"
    dev = _device(logits, what)
    if dev != _current() or stream is not None:
        return _on(dev, stream, router_backward, logits, idx, d_gates=d_gates, d_loss=d_loss, counts=counts, tokens=tokens,
                   sequences=sequences, score=score, normalize=normalize, scale=scale)
    rows, ld, T, E = _logits(logits, what)
    kind = _score(score, what)
    idx = _slots_of(idx, T, E, dev, what)
    k = idx.shape[1]
    if d_gates is None and d_loss is None:
        _bad(what + ": d_gates or d_loss")
    if d_gates is not None:
        d_gates = _floats(d_gates, (T, k), dev, "d_gates is float32 [T][k] on the same device", what)
    seq, S = None, 1
    if d_loss is not None:
        seq, S = _sequences(sequences, dev, what)
        d_loss = _floats(d_loss, (S,), dev, "d_loss is float32 [S] on the same device", what)
        counts = _ints(counts, (S, E), dev, "counts is int32 [S][E] on the same device", what)
        tokens = _ints(tokens, (S,), dev, "tokens is int32 [S] on the same device", what)
    elif counts is not None or tokens is not None or sequences is not None:
        _bad(what + ": counts, tokens and sequences go with d_loss")
    out = _empty((T, E), dtype=rows.dtype, device=logits.device)
    a = _RouterBackwardArgs(rows.data_ptr(), ld, idx.data_ptr(), _p(d_gates), _p(d_loss), _p(counts), _p(tokens), _p(seq),
                            out.data_ptr(), E, T, E, k, S, DTYPES[rows.dtype], kind, bool(normalize), scale)
    code = lib().moe_router_backward(a, _raw_stream(dev))
    if code:
        _check(code, "moe_router_backward")
    return out
