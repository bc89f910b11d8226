"""Operators round the layer: tokens sorted by expert and back, the norms
behind and before a block, four-bit activations with their product, and products
of a few rows with four-bit weights.

Argument marshalling for the stand-alone entry points of ``include/moe.h``;
nothing is computed here.  Every function takes CUDA tensors of one device,
runs on that device's current stream, does not synchronise, and can be captured
in a CUDA graph.  With `stream` (a torch.cuda.Stream of that device) it runs as
inside ``with torch.cuda.stream(stream)``: what it allocates, outputs among it,
belongs to that stream, and the inputs have to be ready there.  Rows may be
strided (a copy is made only where a row's elements are not contiguous).  Bad
arguments raise :class:`MoeError` with MOE_ERR_INVALID_ARG before anything is
enqueued.  Gradients are calls of their own; nothing is recorded for autograd.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import MOE_ERR_INVALID_ARG, MoeError, _check, lib

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2
GATES = {"none": GATE_NONE, "channel": GATE_CHANNEL, "token": GATE_TOKEN}


class _BlockNormArgs(C.Structure):
    _fields_ = [("x", C.c_void_p), ("ld_x", C.c_int64), ("y", C.c_void_p), ("ld_y", C.c_int64),
                ("w_post", C.c_void_p), ("w_pre", C.c_void_p), ("gate", C.c_void_p),
                ("h", C.c_void_p), ("ld_h", C.c_int64), ("u", C.c_void_p), ("ld_u", C.c_int64)] + \
               [(n, C.c_int32) for n in ("T", "D", "x_dtype", "y_dtype", "u_dtype", "w_dtype", "gate_kind")] + \
               [("res_scale", C.c_float), ("eps", C.c_float)]


class _BlockNormBackwardArgs(C.Structure):
    _fields_ = [("dh", C.c_void_p), ("ld_dh", C.c_int64), ("du", C.c_void_p), ("ld_du", C.c_int64),
                ("h", C.c_void_p), ("ld_h", C.c_int64), ("y", C.c_void_p), ("ld_y", C.c_int64),
                ("w_post", C.c_void_p), ("w_pre", C.c_void_p), ("gate", C.c_void_p),
                ("dx", C.c_void_p), ("ld_dx", C.c_int64), ("dy", C.c_void_p), ("ld_dy", C.c_int64),
                ("dw_post", C.c_void_p), ("dw_pre", C.c_void_p), ("d_gate", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)] + \
               [(n, C.c_int32) for n in ("T", "D", "x_dtype", "y_dtype", "u_dtype", "w_dtype", "gate_kind")] + \
               [("res_scale", C.c_float), ("eps", C.c_float)]


class _BlockArgs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("x", "u", "y", "h", "next_u", "w_pre", "w_post", "gate", "next_w_pre")] + \
               [(n, C.c_int32) for n in ("x_dtype", "w_dtype", "gate_kind", "u_ready")] + \
               [("res_scale", C.c_float), ("eps", C.c_float)]


class _W4MatvecArgs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("codes", "scales", "up_codes", "up_scales", "x")] + [("ld_x", C.c_int64)] + \
               [(n, C.c_void_p) for n in ("idx", "weights", "out")] + [("ld_out", C.c_int64)] + \
               [(n, C.c_int32) for n in ("T", "k", "G", "M", "K", "group", "x_per_slot", "format", "scale_dtype", "x_dtype",
                                         "out_dtype")] + [("dev_status", C.c_void_p)]


def declare(L):
    """Argument types of the entry points below (called once, when libmoe is loaded)."""
    P, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    for name, args in (
            ("moe_sort", [P, i32, i32, i32, P, P, P, P, C.c_size_t, P]),
            ("moe_permute", [P, i64, i64, i32, i32, P, i64, P, i64, P]),
            ("moe_unpermute", [P, i64, i32, i64, P, P, i32, i32, i32, P, i64, i32, P]),
            ("moe_unpermute_backward", [P, i64, i32, P, i64, i32, i64, P, P, i32, i32, i32, P, i64, P, P]),
            ("moe_block_norm", [C.POINTER(_BlockNormArgs), P]),
            ("moe_block_norm_backward", [C.POINTER(_BlockNormBackwardArgs), P]),
            ("moe_mxfp4_quantize", [P, i64, i32, i64, i64, P, P, P]),
            ("moe_mxfp4_decode", [P, P, i64, i64, P, i64, i32, P]),
            ("moe_mx4_gemm", [P, P, i32, i32, P, P, i32, i32, P, P, i64, i32, P, P]),
            ("moe_w4_matvec", [C.POINTER(_W4MatvecArgs), P]),
            ("moe_forward_block", [P, C.POINTER(_BlockArgs), i32, P])):
        f = getattr(L, name)
        f.restype = C.c_int
        f.argtypes = args
    L.moe_sort_workspace_bytes.restype = C.c_size_t
    L.moe_sort_workspace_bytes.argtypes = [i32, i32, i32]
    L.moe_block_norm_workspace_bytes.restype = C.c_size_t
    L.moe_block_norm_workspace_bytes.argtypes = [i32, i32]


def _bad(what):
    raise MoeError(MOE_ERR_INVALID_ARG, what)


def _require(ok, what):
    if not ok:
        _bad(what)


# The current stream's handle without a Stream object (2.8 us a call on the
# host of a GB300) and the current device without a check of the context, where
# this PyTorch has those shortcuts.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty = torch.empty


def _device(t, what):
    """Index of the CUDA device that tensor `t` is on."""
    if not isinstance(t, torch.Tensor):
        _bad(what + ": CUDA tensors are needed")
    dev = t.get_device()
    if dev < 0:
        _bad(what + ": CUDA tensors are needed")
    return dev


def _on(dev, stream, f, *args, **kwargs):
    """f with device `dev`, or its stream `stream`, current.  Copies and workspaces then belong to the stream that
    reads them: memory of another stream may be handed out again before the kernels are through with it."""
    if stream is None:
        with torch.cuda.device(dev):
            return f(*args, **kwargs)
    if not isinstance(stream, torch.cuda.Stream) or stream.device_index != dev:
        _bad(f.__name__ + ": stream is a torch.cuda.Stream of the tensors' device")
    with torch.cuda.stream(stream):
        return f(*args, **kwargs)


def _int32(n, what):
    """Sizes go to the entry points as 32-bit integers, which the call would cut off."""
    if n > 0x7fffffff:
        _bad(what + ": sizes below 2^31")


def _rows(t, what):
    """t [..., D] of a known type as rows: (2-D tensor whose rows are contiguous, row stride in elements)."""
    if t.dtype not in DTYPES:
        _bad(what + ": float32, bfloat16 or float16 is needed")
    return _strided(t, what)


def _strided(t, what):
    if t.dim() == 2:
        (T, D), (ld, unit) = t.shape, t.stride()
        if unit == 1 and ld >= D and T > 1:
            return t, ld
    else:
        _require(t.dim() >= 1, what + ": a matrix is needed")
        D = t.shape[-1]
        t = t.reshape(-1, D) if D else t.reshape(0, 0)
        T, (ld, unit) = t.shape[0], t.stride()
    if T <= 1 or D <= 1:
        return t.contiguous(), D              # strides of single rows and columns say nothing
    if unit != 1 or ld < D:
        return t.contiguous(), D
    return t, ld


def _out_rows(out, T, D, dtype, dev, what):
    """Row stride of the output matrix `out`, which has to be [T][D] with contiguous rows."""
    if out.dim() != 2 or out.shape[0] != T or out.shape[1] != D or out.dtype != dtype or out.get_device() != dev:
        _bad(what + ": the output's shape, type or device")
    ld, unit = out.stride()
    if out.numel() == 0 or T == 1:
        ld = D
    elif ld < D:
        _bad(what + ": output rows must lie apart")
    if unit != 1 and D > 1 and out.numel():
        _bad(what + ": output rows must be contiguous")
    return ld


def _slots(slot_pos, dev, what):
    if slot_pos.dtype != torch.int32 or slot_pos.dim() != 2 or not slot_pos.is_contiguous() or slot_pos.get_device() != dev:
        _bad(what + ": slot_pos is a contiguous int32 [T][k] on the same device")
    _int32(slot_pos.numel(), what)
    return slot_pos.shape


def _weights_of(weights, slot_pos, what):
    if weights is None:
        return None
    if not isinstance(weights, torch.Tensor) or weights.dtype != torch.float32 or weights.shape != slot_pos.shape or weights.get_device() != slot_pos.get_device():
        _bad(what + ": weights are float32 [T][k] on the same device")
    return weights.contiguous()


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ tokens by expert and back
def sort_by_expert(idx: torch.Tensor, n_experts: int, stream=None):
    """Sort the (token, slot) pairs of idx int32 [T][k] by expert (see
    moe_sort): (offsets int32 [E + 1], sorted_slot int32 [T * k], slot_pos
    int32 [T][k]).  Entries outside [0, n_experts) are dropped (-1)."""
    dev = _device(idx, "sort_by_expert")
    if idx.dtype != torch.int32 or idx.dim() != 2:
        _bad("sort_by_expert: idx is int32 [T][k]")
    E = int(n_experts)
    if not 1 <= E <= 1024:
        _bad("sort_by_expert: 1 <= n_experts <= 1024")
    _int32(idx.numel(), "sort_by_expert")
    if dev != _current() or stream is not None:
        return _on(dev, stream, sort_by_expert, idx, E)
    idx = idx.contiguous()
    T, k = idx.shape
    where = idx.device
    slot_pos = _empty((T, k), dtype=torch.int32, device=where)
    sorted_slot = _empty(T * k, dtype=torch.int32, device=where)
    offsets = _empty(E + 1, dtype=torch.int32, device=where)
    L = lib()
    size = L.moe_sort_workspace_bytes(T, k, E)
    work = _empty(size, dtype=torch.uint8, device=where) if size else None
    code = L.moe_sort(idx.data_ptr(), T, k, E, offsets.data_ptr(), sorted_slot.data_ptr(), slot_pos.data_ptr(),
                      work.data_ptr() if size else None, size, _raw_stream(dev))
    if code:
        _check(code, "moe_sort")
    return offsets, sorted_slot, slot_pos


def permute(x: torch.Tensor, slot_pos: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rows[slot_pos[t, j]] = x[t] (see moe_permute).  x [T][D] of any type
    (codes and scales too); out [n][D], by default T * k new rows, whose places
    that no slot names are not initialised."""
    dev = _device(x, "permute")
    if dev != _current() or stream is not None:
        return _on(dev, stream, permute, x, slot_pos, out)
    T, k = _slots(slot_pos, dev, "permute")
    if x.dim() != 2 or x.shape[0] != T or x.shape[1] < 1:
        _bad("permute: x is [T][D]")
    x, ld = _strided(x, "permute")
    D, size = x.shape[1], x.element_size()
    if out is None:
        n, ld_rows = T * k, D
        out = _empty((n, D), dtype=x.dtype, device=x.device)
    else:
        n = out.shape[0] if out.dim() == 2 else -1
        ld_rows = _out_rows(out, n, D, x.dtype, dev, "permute")
    code = lib().moe_permute(x.data_ptr(), ld * size, D * size, T, k, slot_pos.data_ptr(), n, out.data_ptr(), ld_rows * size, _raw_stream(dev))
    if code:
        _check(code, "moe_permute")
    return out


def unpermute(rows: torch.Tensor, slot_pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] rows[slot_pos[t, j]] (see moe_unpermute); y [T][D] of out_dtype (default: rows')."""
    dev = _device(rows, "unpermute")
    if dev != _current() or stream is not None:
        return _on(dev, stream, unpermute, rows, slot_pos, weights, out_dtype, out)
    T, k = _slots(slot_pos, dev, "unpermute")
    if rows.dim() != 2 or rows.shape[1] < 1:
        _bad("unpermute: rows is [n][D]")
    rows, ld = _rows(rows, "unpermute")
    n, D = rows.shape
    _int32(D, "unpermute")
    w = _weights_of(weights, slot_pos, "unpermute")
    dtype = out_dtype or (rows.dtype if out is None else out.dtype)
    if dtype not in DTYPES:
        _bad("unpermute: output type")
    if out is None:
        out, ld_y = _empty((T, D), dtype=dtype, device=rows.device), D
    else:
        ld_y = _out_rows(out, T, D, dtype, dev, "unpermute")
    code = lib().moe_unpermute(rows.data_ptr(), ld, DTYPES[rows.dtype], n, slot_pos.data_ptr(),
                               None if w is None else w.data_ptr(), T, k, D, out.data_ptr(), ld_y, DTYPES[dtype], _raw_stream(dev))
    if code:
        _check(code, "moe_unpermute")
    return out


def permute_backward(d_rows: torch.Tensor, slot_pos: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of permute: dx[t] = sum_j d_rows[slot_pos[t, j]]."""
    return unpermute(d_rows, slot_pos, None, out_dtype, out, stream)


def unpermute_backward(dy: torch.Tensor, rows: torch.Tensor, slot_pos: torch.Tensor,
                       weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       need_rows: bool = True, need_weights: bool = True, stream=None):
    """Gradients of unpermute (see moe_unpermute_backward): (d_rows like rows,
    or None; d_weights float32 [T][k], or None).  out: where d_rows goes; a new
    one's places that no slot names are not initialised."""
    dev = _device(dy, "unpermute_backward")
    if dev != _current() or stream is not None:
        return _on(dev, stream, unpermute_backward, dy, rows, slot_pos, weights, out, need_rows, need_weights)
    T, k = _slots(slot_pos, dev, "unpermute_backward")
    if dy.dim() != 2 or dy.shape[0] != T or dy.shape[1] < 1 or rows.dim() != 2 or rows.shape[1] != dy.shape[1] \
            or rows.get_device() != dev:
        _bad("unpermute_backward: dy is [T][D], rows is [n][D] on the same device")
    dy, ld_dy = _rows(dy, "unpermute_backward")
    rows, ld = _rows(rows, "unpermute_backward")
    n, D = rows.shape
    _int32(D, "unpermute_backward")
    w = _weights_of(weights, slot_pos, "unpermute_backward")
    ld_d = D
    if not need_rows:
        out = None
    elif out is None:
        out = _empty((n, D), dtype=rows.dtype, device=rows.device)
    else:
        ld_d = _out_rows(out, n, D, rows.dtype, dev, "unpermute_backward")
    d_w = _empty((T, k), dtype=torch.float32, device=rows.device) if need_weights else None
    code = lib().moe_unpermute_backward(dy.data_ptr(), ld_dy, DTYPES[dy.dtype], rows.data_ptr(), ld, DTYPES[rows.dtype], n,
                                        slot_pos.data_ptr(), _p(w), T, k, D, _p(out), ld_d, _p(d_w), _raw_stream(dev))
    if code:
        _check(code, "moe_unpermute_backward")
    return out, d_w


# ------------------------------------------------------------------ norms round a block
def _gate(gate, gate_per, T, D, dev, what):
    """(contiguous gate, kind): gate [D] or [T], told apart by gate_per or, where T != D, by its length."""
    if gate is None:
        if gate_per not in (None, "none"):
            _bad(what + ": gate_per without a gate")
        return None, GATE_NONE
    n = gate.numel()
    if gate_per is None:
        if T == D or n not in (T, D):
            _bad(what + ": the gate is [D] or [T]; gate_per says which where both fit")
        gate_per = "channel" if n == D else "token"
    if gate_per not in ("channel", "token") or gate.get_device() != dev or n != (D if gate_per == "channel" else T):
        _bad(what + ": gate_per is 'channel' ([D]) or 'token' ([T]), on the same device")
    if gate.dim() != 1:
        gate = gate.reshape(-1)
    return gate.contiguous(), GATES[gate_per]


def _norm_weights(what, dev, D, w_post, w_pre, gate):
    """The code of the weights' common type; each norm weight is a contiguous [D]."""
    kind = None
    for w in (w_post, w_pre):
        if w is not None:
            if w.dim() != 1 or w.shape[0] != D or not w.is_contiguous():
                _bad(what + ": norm weights are contiguous [D]")
            if w.get_device() != dev or (kind is not None and w.dtype != kind):
                _bad(what + ": weights and gate of one type on the same device")
            kind = w.dtype
    if gate is not None:
        if gate.get_device() != dev or (kind is not None and gate.dtype != kind):
            _bad(what + ": weights and gate of one type on the same device")
        kind = gate.dtype
    if kind is None:
        return 0
    if kind not in DTYPES:
        _bad(what + ": float32, bfloat16 or float16 weights are needed")
    return DTYPES[kind]


def _out_like(out, shape, T, dtype, dev, what):
    """Row stride of `out`, which has to be of `shape` with evenly spaced, contiguous rows, and its rows."""
    if out.shape != shape:
        _bad(what + ": the output's shape, type or device")
    r = out
    if out.dim() != 2:
        try:
            r = out.view(T, shape[-1])
        except RuntimeError:
            _bad(what + ": output rows must be evenly spaced")
    return _out_rows(r, T, shape[-1], dtype, dev, what)


def block_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, *, w_post: Optional[torch.Tensor] = None,
               w_pre: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, gate_per: Optional[str] = None,
               res_scale: float = 1.0, eps: float = 1e-6, u_dtype: Optional[torch.dtype] = None, need_u: bool = True,
               out_h: Optional[torch.Tensor] = None, out_u: Optional[torch.Tensor] = None, stream=None):
    """h = res_scale x + gate w_post y / rms(y) and u = w_pre h / rms(h) (see
    moe_block_norm), for x and y [..., D]: (h, u).  Without y, h is x itself;
    need_u=False leaves u out (None).  u has u_dtype (default: x's type).
    out_h (which may be x) and out_u take the results; they are [..., D] with
    contiguous rows."""
    what = "block_norm"
    dev = _device(x, what)
    if dev != _current() or stream is not None:
        return _on(dev, stream, block_norm, x, y, w_post=w_post, w_pre=w_pre, gate=gate, gate_per=gate_per, res_scale=res_scale,
                   eps=eps, u_dtype=u_dtype, need_u=need_u, out_h=out_h, out_u=out_u)
    shape = x.shape
    if not shape or shape[-1] < 1:
        _bad("block_norm: x is [..., D]")
    D = shape[-1]
    xr, ld_x = _rows(x, what)
    T = xr.shape[0]
    _int32(max(T, D), what)
    h, u = x, None
    y_p = h_p = u_p = gate_p = None
    ld_y = ld_h = ld_u = D
    y_type = u_type = kind = 0
    if y is not None:
        if y.shape != shape or y.get_device() != dev:
            _bad("block_norm: y has x's shape and device")
        yr, ld_y = _rows(y, what)
        y_p, y_type = yr.data_ptr(), DTYPES[yr.dtype]
        if out_h is None:
            h = _empty(shape, dtype=x.dtype, device=x.device)
        else:
            h, ld_h = out_h, _out_like(out_h, shape, T, x.dtype, dev, what)
        h_p = h.data_ptr()
        gate, kind = _gate(gate, gate_per, T, D, dev, what)
        gate_p = _p(gate)
    elif gate is not None or w_post is not None or out_h is not None or not need_u:
        _bad("block_norm: gate, w_post and out_h go with y")
    if need_u:
        dt = u_dtype or (x.dtype if out_u is None else out_u.dtype)
        if dt not in DTYPES:
            _bad("block_norm: u_dtype")
        if out_u is None:
            u = _empty(shape, dtype=dt, device=x.device)
        else:
            u, ld_u = out_u, _out_like(out_u, shape, T, dt, dev, what)
        u_p, u_type = u.data_ptr(), DTYPES[dt]
    else:
        w_pre = None
    w_type = _norm_weights(what, dev, D, w_post, w_pre, gate)
    if T:
        a = _BlockNormArgs(xr.data_ptr(), ld_x, y_p, ld_y, _p(w_post), _p(w_pre), gate_p, h_p, ld_h, u_p, ld_u, T, D,
                           DTYPES[xr.dtype], y_type, u_type, w_type, kind, res_scale, eps)
        code = lib().moe_block_norm(a, _raw_stream(dev))
        if code:
            _check(code, "moe_block_norm")
    return h, u


def block_norm_backward(dh: Optional[torch.Tensor], du: Optional[torch.Tensor], h: torch.Tensor,
                        y: Optional[torch.Tensor] = None, *, w_post: Optional[torch.Tensor] = None,
                        w_pre: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                        gate_per: Optional[str] = None, res_scale: float = 1.0, eps: float = 1e-6,
                        need_weights: bool = True, stream=None) -> dict:
    """Gradients of block_norm (see moe_block_norm_backward) from the gradients
    of its outputs (either may be None) and the h and y that it stored: a dict
    of 'dx', 'dy', 'dw_post', 'dw_pre' and 'd_gate' (weights and gate in
    float32; None for what the call does not have).  need_weights=False leaves
    the weights' and the gate's out."""
    what = "block_norm_backward"
    dev = _device(h, what)
    if dev != _current() or stream is not None:
        return _on(dev, stream, block_norm_backward, dh, du, h, y, w_post=w_post, w_pre=w_pre, gate=gate, gate_per=gate_per,
                   res_scale=res_scale, eps=eps, need_weights=need_weights)
    shape, where = h.shape, h.device
    if not shape or shape[-1] < 1 or (dh is None and du is None):
        _bad("block_norm_backward: dh or du, and h [..., D]")
    D = shape[-1]
    for t in (dh, du, y):
        if t is not None and (t.shape != shape or t.get_device() != dev):
            _bad("block_norm_backward: dh, du and y have h's shape and device")
    if dh is not None and dh.dtype != h.dtype:
        _bad("block_norm_backward: dh has h's type")
    hr, ld_h = _rows(h, what)
    T = hr.shape[0]
    _int32(max(T, D), what)
    dh_p = du_p = y_p = dy_p = gate_p = work_p = None
    ld_dh = ld_du = ld_y = D
    u_type = y_type = kind = size = 0
    if dh is not None:
        dhr, ld_dh = _rows(dh, what)
        dh_p = dhr.data_ptr()
    if du is not None:
        dur, ld_du = _rows(du, what)
        du_p, u_type = dur.data_ptr(), DTYPES[dur.dtype]
    else:
        w_pre = None
    dx = _empty(shape, dtype=h.dtype, device=where)
    dy = None
    if y is not None:
        yr, ld_y = _rows(y, what)
        y_p, y_type = yr.data_ptr(), DTYPES[yr.dtype]
        dy = _empty(shape, dtype=y.dtype, device=where)
        dy_p = dy.data_ptr()
        gate, kind = _gate(gate, gate_per, T, D, dev, what)
        gate_p = _p(gate)
    elif gate is not None or w_post is not None:
        _bad("block_norm_backward: gate and w_post go with y")
    w_type = _norm_weights(what, dev, D, w_post, w_pre, gate)
    dw_post = dw_pre = d_gate = None
    if need_weights:
        columns = 0
        if w_post is not None:
            dw_post, columns = _empty(D, dtype=torch.float32, device=where), 1
        if w_pre is not None:
            dw_pre, columns = _empty(D, dtype=torch.float32, device=where), 1
        if kind == GATE_CHANNEL:
            d_gate, columns = _empty(D, dtype=torch.float32, device=where), 1
        elif kind == GATE_TOKEN:
            d_gate = _empty(T, dtype=torch.float32, device=where)
        if columns and T:
            size = lib().moe_block_norm_workspace_bytes(T, D)
            work = _empty(size, dtype=torch.uint8, device=where)
            work_p = work.data_ptr()
    a = _BlockNormBackwardArgs(dh_p, ld_dh, du_p, ld_du, hr.data_ptr(), ld_h, y_p, ld_y, _p(w_post), _p(w_pre), gate_p,
                               dx.data_ptr(), D, dy_p, D, _p(dw_post), _p(dw_pre), _p(d_gate), work_p, size, T, D,
                               DTYPES[hr.dtype], y_type, u_type, w_type, kind, res_scale, eps)
    code = lib().moe_block_norm_backward(a, _raw_stream(dev))
    if code:
        _check(code, "moe_block_norm_backward")
    return dict(dx=dx, dy=dy, dw_post=dw_post, dw_pre=dw_pre, d_gate=d_gate)


# ------------------------------------------------------------------ four bits
def mxfp4_quantize(x: torch.Tensor, stream=None):
    """MXFP4 of x [..., K] (float32, bfloat16 or float16; K a multiple of 32):
    (codes uint8 [..., K/2], scales uint8 [..., K/32]); see moe_mxfp4_quantize."""
    dev = _device(x, "mxfp4_quantize")
    if dev != _current() or stream is not None:
        return _on(dev, stream, mxfp4_quantize, x)
    shape = x.shape
    if not shape or shape[-1] < 32 or shape[-1] % 32:
        _bad("mxfp4_quantize: K is a multiple of 32")
    K = shape[-1]
    xr, ld = _rows(x, "mxfp4_quantize")
    lead = tuple(shape[:-1])
    codes = _empty(lead + (K // 2,), dtype=torch.uint8, device=x.device)
    scales = _empty(lead + (K // 32,), dtype=torch.uint8, device=x.device)
    code = lib().moe_mxfp4_quantize(xr.data_ptr(), ld, DTYPES[xr.dtype], xr.shape[0], K, codes.data_ptr(), scales.data_ptr(), _raw_stream(dev))
    if code:
        _check(code, "moe_mxfp4_quantize")
    return codes, scales


def _mx4(codes, scales, what):
    c, s = tuple(codes.shape), tuple(scales.shape)
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not c or not s or c[:-1] != s[:-1] \
            or c[-1] != 16 * s[-1] or c[-1] < 16 or codes.get_device() != scales.get_device():
        _bad(what + ": codes uint8 [..., K/2] and scales uint8 [..., K/32] of one device")
    return codes.contiguous(), scales.contiguous()


def mxfp4_decode(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The values [..., K] that MXFP4 codes and scales stand for, rounded to `dtype`."""
    dev = _device(codes, "mxfp4_decode")
    if dev != _current() or stream is not None:
        return _on(dev, stream, mxfp4_decode, codes, scales, dtype)
    codes, scales = _mx4(codes, scales, "mxfp4_decode")
    if dtype not in DTYPES:
        _bad("mxfp4_decode: output type")
    K = codes.shape[-1] * 2
    x = _empty(tuple(codes.shape[:-1]) + (K,), dtype=dtype, device=codes.device)
    code = lib().moe_mxfp4_decode(codes.data_ptr(), scales.data_ptr(), x.numel() // K, K, x.data_ptr(), K, DTYPES[dtype], _raw_stream(dev))
    if code:
        _check(code, "moe_mxfp4_decode")
    return x


def mx4_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
             offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             out_dtype: Optional[torch.dtype] = None, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Product of MXFP4 operands (see moe_mx4_gemm): out [N][M] of out_dtype
    (default float32) = B A^T with A [M][K]; or, with A [G][M][K] and offsets
    int32 [G + 1] on the device, rows offsets[g] to offsets[g + 1] of B times
    A[g].  Rows that belong to no group are left as they were."""
    what = "mx4_gemm"
    dev = _device(a_codes, what)
    if dev != _current() or stream is not None:
        return _on(dev, stream, mx4_gemm, a_codes, a_scales, b_codes, b_scales, offsets, out, out_dtype, status)
    a_codes, a_scales = _mx4(a_codes, a_scales, what)
    b_codes, b_scales = _mx4(b_codes, b_scales, what)
    if b_codes.dim() != 2 or b_codes.shape[1] != a_codes.shape[-1] or b_codes.get_device() != dev:
        _bad("mx4_gemm: B is [N][K] of A's K, on A's device")
    if offsets is None:
        if a_codes.dim() != 2:
            _bad("mx4_gemm: one matrix [M][K] without offsets")
        G, M = 1, a_codes.shape[0]
    else:
        if a_codes.dim() != 3 or offsets.dtype != torch.int32 or not offsets.is_contiguous() \
                or offsets.numel() != a_codes.shape[0] + 1 or offsets.get_device() != dev:
            _bad("mx4_gemm: A is [G][M][K], offsets int32 [G + 1] on its device")
        G, M, _ = a_codes.shape
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1 or status.get_device() != dev):
        _bad("mx4_gemm: status is int32 on A's device")
    N, K = b_codes.shape[0], 2 * b_codes.shape[1]
    _int32(max(G, M, N, K), what)
    dtype = out_dtype or (torch.float32 if out is None else out.dtype)
    if dtype not in DTYPES:
        _bad("mx4_gemm: output type")
    if out is None:
        out, ld = _empty((N, M), dtype=dtype, device=a_codes.device), M
    else:
        ld = _out_rows(out, N, M, dtype, dev, what)
    code = lib().moe_mx4_gemm(a_codes.data_ptr(), a_scales.data_ptr(), G, M, b_codes.data_ptr(), b_scales.data_ptr(), N, K,
                              _p(offsets), out.data_ptr(), ld, DTYPES[dtype], _p(status), _raw_stream(dev))
    if code:
        _check(code, "moe_mx4_gemm")
    return out


W4_MXFP4, W4_INT4 = 0, 1


def _w4(codes, scales, dims, dev, what):
    """Contiguous (codes, scales), and the group that a scale is for: codes uint8 [..., K/2], scales [..., K/group]."""
    if not isinstance(codes, torch.Tensor) or not isinstance(scales, torch.Tensor) or codes.dtype != torch.uint8 \
            or (scales.dtype != torch.uint8 and scales.dtype not in DTYPES) or codes.dim() != dims \
            or scales.shape[:-1] != codes.shape[:-1] or scales.dim() != dims or codes.numel() == 0 or scales.shape[-1] < 1 \
            or codes.get_device() != dev or scales.get_device() != dev:
        _bad(what + ": codes uint8 [..., M, K/2] and scales [..., M, K/group] on x's device")
    K, n = 2 * codes.shape[-1], scales.shape[-1]
    if K % n or K // n not in ((32,) if scales.dtype == torch.uint8 else (32, 64, 128)):
        _bad(what + ": a scale for 32 weights (E8M0), or for 32, 64 or 128 (floating scales)")
    return codes.contiguous(), scales.contiguous(), K // n


def w4_matvec(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, *, up=None, idx: Optional[torch.Tensor] = None,
              weights: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Products of a few rows with four-bit weights (see moe_w4_matvec), x not
    quantised.  scales uint8: MXFP4 as mxfp4_quantize writes it; scales float32,
    bfloat16 or float16: codes 0 to 15 that stand for -8 to 7.  One matrix codes
    [M][K/2]: x [N][K] or [K] gives [N][M] or [M].  With idx int32 [T][k] and
    codes [G][M][K/2]: x [T][K], or [T][k][K] with a row for each slot, gives
    [T][k][M], zeros for slots outside [0, G); with weights float32 [T][k] the
    weighted sum over a token's slots, [T][M].  up: a second (codes, scales), for
    SiLU(product) times its product.  The result has out_dtype (default: x's)."""
    what = "w4_matvec"
    dev = _device(x, what)
    if dev != _current() or stream is not None:
        return _on(dev, stream, w4_matvec, x, codes, scales, up=up, idx=idx, weights=weights, out_dtype=out_dtype, out=out,
                   status=status)
    codes, scales, group = _w4(codes, scales, 2 if idx is None else 3, dev, what)
    M, K = codes.shape[-2], 2 * codes.shape[-1]
    if up is not None:
        if not isinstance(up, (tuple, list)) or len(up) != 2:
            _bad(what + ": up is (codes, scales)")
        up_codes, up_scales, _ = _w4(up[0], up[1], codes.dim(), dev, what)
        if up_codes.shape != codes.shape or up_scales.shape != scales.shape or up_scales.dtype != scales.dtype:
            _bad(what + ": up has the sizes and types of the first matrix")
    if not x.dim() or x.shape[-1] != K:
        _bad(what + ": x [..., K]")
    G, k, per_slot = 1, 1, 0
    if idx is None:
        if x.dim() > 2 or weights is not None:
            _bad(what + ": without idx, x is [N][K] or [K] and there are no weights")
        lead = tuple(x.shape[:-1])
        T = lead[0] if lead else 1
    else:
        if not isinstance(idx, torch.Tensor) or idx.dtype != torch.int32 or idx.dim() != 2 or idx.get_device() != dev:
            _bad(what + ": idx is int32 [T][k] on the same device")
        G, (T, k) = codes.shape[0], idx.shape
        _int32(idx.numel(), what)
        per_slot = int(x.dim() == 3)
        if tuple(x.shape[:-1]) not in ((T,), (T, k)):
            _bad(what + ": x is [T][K] or [T][k][K]")
        idx = idx.contiguous()
        weights = _weights_of(weights, idx, what)
        lead = (T,) if weights is not None else (T, k)
        if weights is not None and up is not None:
            _bad(what + ": up and weights do not go together")
    xr, ld = _rows(x, what)
    _int32(max(T, K, G * M), what)
    if out is not None and not isinstance(out, torch.Tensor):
        _bad(what + ": out is a tensor")
    dtype = out_dtype or (x.dtype if out is None else out.dtype)
    if not isinstance(dtype, torch.dtype) or dtype not in DTYPES:
        _bad(what + ": output type")
    if status is not None and (not isinstance(status, torch.Tensor) or status.dtype != torch.int32 or status.numel() < 1 or status.get_device() != dev):
        _bad(what + ": status is int32 on x's device")
    shape = lead + (M,)
    n = T if len(lead) < 2 else T * k
    if out is None:
        out, ld_out = _empty(shape, dtype=dtype, device=x.device), M
    else:
        ld_out = _out_like(out, shape, n, dtype, dev, what)
    if n:
        ints = scales.dtype != torch.uint8
        a = _W4MatvecArgs(codes.data_ptr(), scales.data_ptr(), None if up is None else up_codes.data_ptr(),
                          None if up is None else up_scales.data_ptr(), xr.data_ptr(), ld, _p(idx), _p(weights), out.data_ptr(),
                          ld_out, T, k, G, M, K, group, per_slot, W4_INT4 if ints else W4_MXFP4,
                          DTYPES[scales.dtype] if ints else 0, DTYPES[xr.dtype], DTYPES[dtype], _p(status))
        code = lib().moe_w4_matvec(a, _raw_stream(dev))
        if code:
            _check(code, "moe_w4_matvec")
    return out
