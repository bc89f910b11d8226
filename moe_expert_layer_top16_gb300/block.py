"""Operators round the layer: tokens sorted by expert and back, the norms
behind and before a block, and four-bit activations with their product.

Argument marshalling for the stand-alone entry points of ``include/moe.h``;
nothing is computed here.  Every function takes CUDA tensors of one device,
runs on that device's current stream (or `stream`), does not synchronise, and
can be captured in a CUDA graph.  Rows may be strided (a copy is made only
where a row's elements are not contiguous).  Bad arguments raise
:class:`MoeError` with MOE_ERR_INVALID_ARG before anything is enqueued.
Gradients are calls of their own; nothing is recorded for autograd.
"""
from __future__ import annotations

import ctypes as C
import functools
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


def declare(L):
    """Argument types of the entry points below (called once, when libmoe is loaded)."""
    P, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    for name, args in (
            ("moe_sort", [P, i32, i32, i32, P, P, P, P]),
            ("moe_permute", [P, i64, i64, i32, i32, P, i64, P, i64, P]),
            ("moe_unpermute", [P, i64, i32, i64, P, P, i32, i32, i32, P, i64, i32, P]),
            ("moe_unpermute_backward", [P, i64, i32, P, i64, i32, i64, P, P, i32, i32, i32, P, i64, P, P]),
            ("moe_block_norm", [C.POINTER(_BlockNormArgs), P]),
            ("moe_block_norm_backward", [C.POINTER(_BlockNormBackwardArgs), P]),
            ("moe_mxfp4_quantize", [P, i64, i32, i64, i64, P, P, P]),
            ("moe_mxfp4_decode", [P, P, i64, i64, P, i64, i32, P]),
            ("moe_mx4_gemm", [P, P, i32, i32, P, P, i32, i32, P, P, i64, i32, P, P]),
            ("moe_forward_block", [P, C.POINTER(_BlockArgs), i32, P])):
        f = getattr(L, name)
        f.restype = C.c_int
        f.argtypes = args
    L.moe_block_norm_workspace_bytes.restype = C.c_size_t
    L.moe_block_norm_workspace_bytes.argtypes = [i32, i32]


def _require(ok, what):
    if not ok:
        raise MoeError(MOE_ERR_INVALID_ARG, what)


def _on_device(f):
    """Run with the device of the first tensor among the positional arguments current."""
    @functools.wraps(f)
    def call(*args, **kwargs):
        first = next((t for t in args if isinstance(t, torch.Tensor)), None)
        _require(first is not None and first.is_cuda, f"{f.__name__}: CUDA tensors are needed")
        if first.device.index == torch.cuda.current_device():
            return f(*args, **kwargs)
        with torch.cuda.device(first.device):
            return f(*args, **kwargs)
    return call


def _stream(stream):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _same_device(dev, what, *tensors):
    for t in tensors:
        if t is not None:
            _require(t.device == dev, f"{what}: all tensors on one device")


def _rows(t, what, dtypes=DTYPES):
    """t [..., D] as rows: (2-D tensor whose rows are contiguous, row stride in elements)."""
    _require(t.dim() >= 1 and t.dtype in dtypes, f"{what}: bad shape or type")
    D = t.shape[-1]
    if t.dim() != 2:
        t = t.reshape(-1, D) if D else t.reshape(0, 0)
    T = t.shape[0]
    if T <= 1 or D <= 1:
        if not t.is_contiguous():
            t = t.contiguous()
        return t, D
    if t.stride(1) != 1 or t.stride(0) < D:
        t = t.contiguous()
    return t, t.stride(0)


def _out_rows(out, shape, dtype, dev, what):
    """An output matrix: `out` (2-D, contiguous rows), or a new one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev), shape[1]
    _require(tuple(out.shape) == tuple(shape) and out.dtype == dtype and out.device == dev, f"{what}: bad output")
    if out.numel() == 0 or shape[0] == 1:
        _require(out.numel() == 0 or shape[1] == 1 or out.stride(1) == 1, f"{what}: output rows must be contiguous")
        return out, shape[1]
    _require((shape[1] == 1 or out.stride(1) == 1) and out.stride(0) >= shape[1],
             f"{what}: output rows must be contiguous and apart")
    return out, out.stride(0)


def _slots(slot_pos, dev, what):
    _require(slot_pos.dtype == torch.int32 and slot_pos.dim() == 2 and slot_pos.is_contiguous() and slot_pos.device == dev,
             f"{what}: slot_pos is a contiguous int32 [T][k] on the same device")
    return slot_pos.shape


def _weights_of(weights, slot_pos, what):
    if weights is None:
        return None
    _require(weights.dtype == torch.float32 and weights.shape == slot_pos.shape and weights.device == slot_pos.device,
             f"{what}: weights are float32 [T][k] on the same device")
    return weights.contiguous()


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ tokens by expert and back
@_on_device
def sort_by_expert(idx: torch.Tensor, n_experts: int, stream=None):
    """Sort the (token, slot) pairs of idx int32 [T][k] by expert (see
    moe_sort): (offsets int32 [E + 1], sorted_slot int32 [T * k], slot_pos
    int32 [T][k]).  Entries outside [0, n_experts) are dropped (-1)."""
    _require(idx.dtype == torch.int32 and idx.dim() == 2, "sort_by_expert: idx is int32 [T][k]")
    idx = idx.contiguous()
    T, k = idx.shape
    _require(1 <= int(n_experts) <= 1024, "sort_by_expert: 1 <= n_experts <= 1024")
    tables = torch.empty(2 * T * k + int(n_experts) + 1, dtype=torch.int32, device=idx.device)
    slot_pos, sorted_slot, offsets = tables[:T * k].view(T, k), tables[T * k:2 * T * k], tables[2 * T * k:]
    _check(lib().moe_sort(_p(idx), T, k, int(n_experts), _p(offsets), _p(sorted_slot), _p(slot_pos), _stream(stream)),
           "moe_sort")
    return offsets, sorted_slot, slot_pos


@_on_device
def permute(x: torch.Tensor, slot_pos: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rows[slot_pos[t, j]] = x[t] (see moe_permute).  x [T][D] of any type
    (codes and scales too); out [n][D], by default T * k new rows, whose places
    that no slot names are not initialised."""
    T, k = _slots(slot_pos, x.device, "permute")
    _require(x.dim() == 2 and x.shape[0] == T and x.shape[1] >= 1, "permute: x is [T][D]")
    x, ld = _rows(x, "permute", (x.dtype,))
    D, size = x.shape[1], x.element_size()
    rows, ld_rows = _out_rows(out, (T * k if out is None else out.shape[0], D), x.dtype, x.device, "permute")
    _check(lib().moe_permute(_p(x), ld * size, D * size, T, k, _p(slot_pos), rows.shape[0], _p(rows), ld_rows * size,
                             _stream(stream)), "moe_permute")
    return rows


@_on_device
def unpermute(rows: torch.Tensor, slot_pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] rows[slot_pos[t, j]] (see moe_unpermute); y [T][D] of out_dtype (default: rows')."""
    T, k = _slots(slot_pos, rows.device, "unpermute")
    _require(rows.dim() == 2 and rows.shape[1] >= 1, "unpermute: rows is [n][D]")
    rows, ld = _rows(rows, "unpermute")
    D = rows.shape[1]
    w = _weights_of(weights, slot_pos, "unpermute")
    dtype = out_dtype or (rows.dtype if out is None else out.dtype)
    _require(dtype in DTYPES, "unpermute: output type")
    y, ld_y = _out_rows(out, (T, D), dtype, rows.device, "unpermute")
    _check(lib().moe_unpermute(_p(rows), ld, DTYPES[rows.dtype], rows.shape[0], _p(slot_pos), _p(w), T, k, D, _p(y), ld_y,
                               DTYPES[dtype], _stream(stream)), "moe_unpermute")
    return y


def permute_backward(d_rows: torch.Tensor, slot_pos: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of permute: dx[t] = sum_j d_rows[slot_pos[t, j]]."""
    return unpermute(d_rows, slot_pos, None, out_dtype, out, stream)


@_on_device
def unpermute_backward(dy: torch.Tensor, rows: torch.Tensor, slot_pos: torch.Tensor,
                       weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       need_rows: bool = True, need_weights: bool = True, stream=None):
    """Gradients of unpermute (see moe_unpermute_backward): (d_rows like rows,
    or None; d_weights float32 [T][k], or None).  out: where d_rows goes; a new
    one's places that no slot names are not initialised."""
    T, k = _slots(slot_pos, dy.device, "unpermute_backward")
    _require(dy.dim() == 2 and dy.shape[0] == T and dy.shape[1] >= 1 and rows.dim() == 2 and rows.shape[1] == dy.shape[1],
             "unpermute_backward: dy is [T][D], rows is [n][D]")
    _same_device(dy.device, "unpermute_backward", rows)
    dy, ld_dy = _rows(dy, "unpermute_backward")
    rows, ld = _rows(rows, "unpermute_backward")
    D = dy.shape[1]
    w = _weights_of(weights, slot_pos, "unpermute_backward")
    d_rows, ld_d = (_out_rows(out, tuple(rows.shape), rows.dtype, rows.device, "unpermute_backward")
                    if need_rows else (None, 0))
    d_w = torch.empty(T, k, dtype=torch.float32, device=dy.device) if need_weights else None
    _check(lib().moe_unpermute_backward(_p(dy), ld_dy, DTYPES[dy.dtype], _p(rows), ld, DTYPES[rows.dtype], rows.shape[0],
                                        _p(slot_pos), _p(w), T, k, D, _p(d_rows), ld_d, _p(d_w), _stream(stream)),
           "moe_unpermute_backward")
    return d_rows, d_w


# ------------------------------------------------------------------ norms round a block
def _gate(gate, gate_per, T, D, dev, what):
    """(contiguous gate, kind): gate [D] or [T], told apart by gate_per or, where T != D, by its length."""
    if gate is None:
        _require(gate_per in (None, "none"), f"{what}: gate_per without a gate")
        return None, GATE_NONE
    _require(gate_per in (None, "channel", "token") and gate.device == dev, f"{what}: gate_per is 'channel' or 'token'")
    n = gate.numel()
    if gate_per is None:
        _require(T != D and n in (T, D), f"{what}: the gate is [D] or [T]; gate_per says which where both fit")
        gate_per = "channel" if n == D else "token"
    _require(n == (D if gate_per == "channel" else T), f"{what}: the gate's length")
    return gate.reshape(-1).contiguous(), GATES[gate_per]


def _norm_weights(what, dev, D, w_post, w_pre, gate):
    """The weights' common type code; each weight contiguous [D]."""
    given = [w for w in (w_post, w_pre, gate) if w is not None]
    if not given:
        return 0
    _require(all(w.dtype == given[0].dtype and w.device == dev for w in given) and given[0].dtype in DTYPES,
             f"{what}: weights and gate of one type on the same device")
    _require(all(w is None or (w.dim() == 1 and w.shape[0] == D and w.is_contiguous()) for w in (w_post, w_pre)),
             f"{what}: norm weights are contiguous [D]")
    return DTYPES[given[0].dtype]


@_on_device
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
    _require(x.dim() >= 1 and x.shape[-1] >= 1, "block_norm: x is [..., D]")
    _same_device(x.device, what, y, out_h, out_u)
    shape, D = x.shape, x.shape[-1]
    _require(y is None or y.shape == shape, "block_norm: y has x's shape")
    _require(y is not None or need_u, "block_norm: nothing to compute")
    xr, ld_x = _rows(x, what)
    T = xr.shape[0]
    a = _BlockNormArgs()
    a.T, a.D, a.res_scale, a.eps = T, D, res_scale, eps
    a.x, a.ld_x, a.x_dtype = _p(xr), ld_x, DTYPES[xr.dtype]
    h = x
    if y is not None:
        yr, a.ld_y = _rows(y, what)
        a.y, a.y_dtype = _p(yr), DTYPES[yr.dtype]
        h, hr, a.ld_h = _out_like(out_h, shape, T, x.dtype, x.device, what)
        a.h = _p(hr)
        gate, a.gate_kind = _gate(gate, gate_per, T, D, x.device, what)
        a.w_post, a.gate = _p(w_post), _p(gate)
    else:
        _require(gate is None and w_post is None and out_h is None, "block_norm: gate, w_post and out_h go with y")
    u = None
    if need_u:
        dt = u_dtype or (x.dtype if out_u is None else out_u.dtype)
        _require(dt in DTYPES, "block_norm: u_dtype")
        u, ur, a.ld_u = _out_like(out_u, shape, T, dt, x.device, what)
        a.u, a.u_dtype, a.w_pre = _p(ur), DTYPES[dt], _p(w_pre)
    a.w_dtype = _norm_weights(what, x.device, D, w_post, w_pre if need_u else None, gate)
    if T:
        _check(lib().moe_block_norm(C.byref(a), _stream(stream)), "moe_block_norm")
    return h, u


def _out_like(out, shape, T, dtype, dev, what):
    """(tensor of `shape`, the same as rows, row stride)."""
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
        return out, out, shape[-1]
    _require(out.shape == shape and out.dtype == dtype and out.device == dev, f"{what}: bad output")
    if out.dim() == 2:
        r = out
    else:
        try:
            r = out.view(T, shape[-1])
        except RuntimeError:
            raise MoeError(MOE_ERR_INVALID_ARG, f"{what}: output rows must be evenly spaced") from None
    r, ld = _out_rows(r, (T, shape[-1]), dtype, dev, what)
    return out, r, ld


@_on_device
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
    shape, D, dev = h.shape, h.shape[-1] if h.dim() else 0, h.device
    _require(D >= 1 and (dh is not None or du is not None), "block_norm_backward: dh or du, and h [..., D]")
    for t in (dh, du, y):
        _require(t is None or (t.shape == shape and t.device == dev), "block_norm_backward: dh, du and y have h's shape and device")
    _require(dh is None or dh.dtype == h.dtype, "block_norm_backward: dh has h's type")
    a = _BlockNormBackwardArgs()
    hr, a.ld_h = _rows(h, what)
    T = hr.shape[0]
    a.h, a.x_dtype = _p(hr), DTYPES[hr.dtype]
    a.T, a.D, a.res_scale, a.eps = T, D, res_scale, eps
    if dh is not None:
        dhr, a.ld_dh = _rows(dh, what)
        a.dh = _p(dhr)
    if du is not None:
        dur, a.ld_du = _rows(du, what)
        a.du, a.u_dtype = _p(dur), DTYPES[dur.dtype]
    got = dict.fromkeys(("dx", "dy", "dw_post", "dw_pre", "d_gate"))
    got["dx"] = torch.empty(shape, dtype=h.dtype, device=dev)
    a.dx, a.ld_dx = _p(got["dx"]), D
    columns = 0
    if y is not None:
        yr, a.ld_y = _rows(y, what)
        a.y, a.y_dtype = _p(yr), DTYPES[yr.dtype]
        got["dy"] = torch.empty(shape, dtype=y.dtype, device=dev)
        a.dy, a.ld_dy = _p(got["dy"]), D
        gate, a.gate_kind = _gate(gate, gate_per, T, D, dev, what)
        a.w_post, a.gate = _p(w_post), _p(gate)
    else:
        _require(gate is None and w_post is None, "block_norm_backward: gate and w_post go with y")
    if du is None:
        w_pre = None
    a.w_pre = _p(w_pre)
    a.w_dtype = _norm_weights(what, dev, D, w_post, w_pre, gate)
    if need_weights:
        # the column sums: weights' gradients exist for norms without weights
        # too (of the ones that they stand for), but only given ones are asked for
        names = [n for n, t in (("dw_post", w_post), ("dw_pre", w_pre),
                                ("d_gate", gate if a.gate_kind == GATE_CHANNEL else None)) if t is not None]
        columns = len(names)
        out = torch.empty(columns, D, dtype=torch.float32, device=dev)
        for n, t in zip(names, out):
            got[n] = t
            setattr(a, n, _p(t))
        if a.gate_kind == GATE_TOKEN:
            got["d_gate"] = torch.empty(T, dtype=torch.float32, device=dev)
            a.d_gate = _p(got["d_gate"])
    if columns and T:
        size = lib().moe_block_norm_workspace_bytes(T, D)
        work = torch.empty(size, dtype=torch.uint8, device=dev)
        a.workspace, a.workspace_bytes = _p(work), size
    _check(lib().moe_block_norm_backward(C.byref(a), _stream(stream)), "moe_block_norm_backward")
    return got


# ------------------------------------------------------------------ four bits
@_on_device
def mxfp4_quantize(x: torch.Tensor, stream=None):
    """MXFP4 of x [..., K] (float32, bfloat16 or float16; K a multiple of 32):
    (codes uint8 [..., K/2], scales uint8 [..., K/32]); see moe_mxfp4_quantize."""
    _require(x.dim() >= 1 and x.shape[-1] >= 32 and x.shape[-1] % 32 == 0, "mxfp4_quantize: K is a multiple of 32")
    xr, ld = _rows(x, "mxfp4_quantize")
    K = x.shape[-1]
    codes = torch.empty(*x.shape[:-1], K // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(*x.shape[:-1], K // 32, dtype=torch.uint8, device=x.device)
    _check(lib().moe_mxfp4_quantize(_p(xr), ld, DTYPES[xr.dtype], xr.shape[0], K, _p(codes), _p(scales), _stream(stream)),
           "moe_mxfp4_quantize")
    return codes, scales


def _mx4(codes, scales, what):
    _require(codes.dtype == torch.uint8 and scales.dtype == torch.uint8 and codes.dim() == scales.dim() >= 1
             and codes.shape[:-1] == scales.shape[:-1] and codes.shape[-1] == 16 * scales.shape[-1] >= 16
             and codes.device == scales.device, f"{what}: codes uint8 [..., K/2] and scales uint8 [..., K/32]")
    return codes.contiguous(), scales.contiguous()


@_on_device
def mxfp4_decode(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The values [..., K] that MXFP4 codes and scales stand for, rounded to `dtype`."""
    codes, scales = _mx4(codes, scales, "mxfp4_decode")
    _require(dtype in DTYPES, "mxfp4_decode: output type")
    K = codes.shape[-1] * 2
    x = torch.empty(*codes.shape[:-1], K, dtype=dtype, device=codes.device)
    _check(lib().moe_mxfp4_decode(_p(codes), _p(scales), x.numel() // K, K, _p(x), K, DTYPES[dtype], _stream(stream)),
           "moe_mxfp4_decode")
    return x


@_on_device
def mx4_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
             offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             out_dtype: Optional[torch.dtype] = None, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Product of MXFP4 operands (see moe_mx4_gemm): out [N][M] of out_dtype
    (default float32) = B A^T with A [M][K]; or, with A [G][M][K] and offsets
    int32 [G + 1] on the device, rows offsets[g] to offsets[g + 1] of B times
    A[g].  Rows that belong to no group are left as they were."""
    what = "mx4_gemm"
    a_codes, a_scales = _mx4(a_codes, a_scales, what)
    b_codes, b_scales = _mx4(b_codes, b_scales, what)
    _same_device(a_codes.device, what, b_codes, offsets, out, status)
    _require(b_codes.dim() == 2 and b_codes.shape[1] == a_codes.shape[-1], "mx4_gemm: B is [N][K] of A's K")
    if offsets is None:
        _require(a_codes.dim() == 2, "mx4_gemm: one matrix [M][K] without offsets")
        G, M = 1, a_codes.shape[0]
    else:
        _require(a_codes.dim() == 3 and offsets.dtype == torch.int32 and offsets.is_contiguous()
                 and offsets.numel() == a_codes.shape[0] + 1, "mx4_gemm: A is [G][M][K], offsets int32 [G + 1]")
        G, M = a_codes.shape[:2]
    _require(status is None or (status.dtype == torch.int32 and status.numel() >= 1), "mx4_gemm: status is int32")
    N, K = b_codes.shape[0], 2 * b_codes.shape[1]
    dtype = out_dtype or (torch.float32 if out is None else out.dtype)
    _require(dtype in DTYPES, "mx4_gemm: output type")
    out, ld = _out_rows(out, (N, M), dtype, a_codes.device, what)
    _check(lib().moe_mx4_gemm(_p(a_codes), _p(a_scales), G, M, _p(b_codes), _p(b_scales), N, K, _p(offsets), _p(out), ld,
                              DTYPES[dtype], _p(status), _stream(stream)), "moe_mx4_gemm")
    return out
