"""The norms round a block and their gradients on matrices that lie anyhow:
bases off 16 bytes and strides that differ modulo a window (element by
element), padded rows, rows whose stride is odd; and gradients whose du has
another type than h.  Each against the formulas in 64 bits, and nothing
outside a matrix's rows is written.

Tolerances as derived in test_gpu_block_norm: a row's sum of D squares in fp32
is off by at most (D / threads + 12) 2^-24 relative with at least 32 threads,
half of which reaches the reciprocal root; c covers each normalised value.  An
output adds half a step of its type, column sums T 2^-24 of the magnitudes."""
import ctypes as C

import pytest
import torch

import test_gpu_block_norm as base
import moe_expert_layer_top16_gb300 as moe
from moe_expert_layer_top16_gb300 import block

pytestmark = pytest.mark.gpu

DEV = base.DEV
F32, BF16, F16 = base.F32, base.BF16, base.F16
HALF, TINY, EPS, rms = base.HALF, base.TINY, base.EPS, base.rms
SCALE = 0.75
GUARD = 5.0


class Matrix:
    """[T][D] of type t whose first element lies `off` elements behind a multiple of 16 bytes and whose rows are `ld`
    apart, in memory that is GUARD everywhere else."""

    def __init__(self, T, D, t, off=0, ld=None, data=None):
        ld = D if ld is None else ld
        self.ld = ld
        self.flat = torch.full((off + (T - 1) * ld + D + 67,), GUARD, device=DEV).to(t)
        self.m = self.flat.as_strided((T, D), (ld, 1), off)
        if data is not None:
            self.m.copy_(data)

    def rest_is_untouched(self):
        keep = self.flat.clone()
        keep.as_strided(self.m.shape, self.m.stride(), self.m.storage_offset()).fill_(GUARD)
        return bool((keep == GUARD).all())


# (offset of the base, padding of a row) for each matrix of a call, in turn
LAYOUTS = {
    "bases off 16 bytes": [(1, 0)],
    "one base off 16 bytes": [(0, 0), (1, 0)],
    "strides unequal modulo a window": [(0, 0), (0, 3)],
    "odd bases and strides": [(3, 5), (1, 2), (0, 0)],
    "whole padded rows": [(0, "whole")],
    "odd strides": [(0, 1)],
    "odd strides, apart": [(0, 1), (0, 17)],
}


def place(layout, i, T, D, t, data=None):
    off, pad = LAYOUTS[layout][i % len(LAYOUTS[layout])]
    ld = (D + 15) // 8 * 8 if pad == "whole" else D + pad
    return Matrix(T, D, t, off, ld, data)


CASES = [(3, 72, F32, F32, F32, "channel"), (40, 1001, BF16, BF16, F32, "token"), (700, 96, F16, F32, F16, None),
         (333, 1000, BF16, F32, F32, "channel"), (9, 1032, F32, BF16, F32, "token"), (400, 1031, F16, F16, F16, "channel"),
         (2, 16384, BF16, BF16, BF16, "channel"), (310, 4104, F32, F32, F32, None), (5, 16383, F32, F32, F32, "token"),
         (1, 50, BF16, BF16, F32, "channel"), (320, 2056, F32, F16, F32, "channel")]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,D,tx,ty,tw,gate", CASES)
@pytest.mark.parametrize("tu", [None, BF16, F32])
def test_forward(T, D, tx, ty, tw, gate, tu, layout):
    s = base.make(T, D, tx, ty, tw, gate, seed=T + D)
    tu = tu or tx
    x, y = place(layout, 0, T, D, tx, s["x"]), place(layout, 1, T, D, ty, s["y"])
    h, u = place(layout, 2, T, D, tx), place(layout, 3, T, D, tu)
    got = moe.block_norm(x.m, y.m, w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per=gate, res_scale=SCALE, eps=EPS,
                         out_h=h.m, out_u=u.m)
    assert got[0] is h.m and got[1] is u.m and h.rest_is_untouched() and u.rest_is_untouched()
    assert torch.equal(x.m, s["x"]) and torch.equal(y.m, s["y"])
    c = (D / 64 + 16) * 2.0 ** -24

    def check(h, u, ref, tol):
        assert ((h.double() - ref).abs() <= tol + (ref.abs() + tol) * HALF[tx] + TINY[tx]).all()
        f = h.double()
        ref = s["w_pre"].double() * f / rms(f)
        assert ((u.double() - ref).abs() <= ref.abs() * (c + HALF[tu] * (1 + c)) + TINY[tu]).all()

    add = base.gate64(s, gate) * s["w_post"].double() * s["y"].double() / rms(s["y"].double())
    ref = SCALE * s["x"].double() + add
    check(h.m, u.m, ref, add.abs() * c + ref.abs() * 2.0 ** -23)
    # in place on the residual stream; the norm before a block alone; only h
    moe.block_norm(x.m, y.m, w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per=gate, res_scale=SCALE, eps=EPS,
                   out_h=x.m, out_u=u.m)
    check(x.m, u.m, ref, add.abs() * c + ref.abs() * 2.0 ** -23)
    assert x.rest_is_untouched()
    moe.block_norm(x.m, w_pre=s["w_pre"], eps=EPS, out_u=u.m)
    check(x.m, u.m, x.m.double(), torch.zeros((), device=DEV))
    only = place(layout, 4, T, D, tx)
    x.m.copy_(s["x"])
    moe.block_norm(x.m, y.m, w_post=s["w_post"], gate=s["gate"], gate_per=gate, res_scale=SCALE, eps=EPS, out_h=only.m, need_u=False)
    assert ((only.m.double() - ref).abs() <= add.abs() * c + ref.abs() * 2.0 ** -23 + (ref.abs() * (1 + 2 * c) + add.abs() * c) * HALF[tx] +
            TINY[tx]).all() and only.rest_is_untouched()


def backward(s, T, D, tx, ty, tu, tw, gate, given, where):
    """moe_block_norm_backward itself (the binding's dx and dy are contiguous), checked against the formula."""
    code = block.DTYPES
    dh = where(0, tx, s["dh"]) if given != "du" else None
    du = where(1, tu, s["du"].to(tu)) if given != "dh" else None
    h, y = where(2, tx, s["x"]), where(3, ty, s["y"])
    dx, dy = where(4, tx), where(5, ty)
    post = given != "pre"
    grads = {n: torch.full((D,), float("nan"), device=DEV) for n in ("dw_post", "dw_pre")}
    grads["d_gate"] = torch.full((T if gate == "token" else D,), float("nan"), device=DEV)
    work = torch.empty(moe.lib().moe_block_norm_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    p = lambda m: None if m is None else m.m.data_ptr()  # noqa: E731
    ld = lambda m: D if m is None else m.ld  # noqa: E731
    a = block._BlockNormBackwardArgs(
        p(dh), ld(dh), p(du), ld(du), p(h), h.ld, p(y) if post else None, y.ld, s["w_post"].data_ptr() if post else None,
        s["w_pre"].data_ptr() if du else None, s["gate"].data_ptr() if post and gate else None, p(dx), dx.ld,
        p(dy) if post else None, dy.ld, grads["dw_post"].data_ptr() if post else None, grads["dw_pre"].data_ptr() if du else None,
        grads["d_gate"].data_ptr() if post and gate else None, work.data_ptr(), work.numel(), T, D, code[tx], code[ty], code[tu],
        code[tw], block.GATES[gate or "none"] if post else 0, SCALE, EPS)
    assert moe.lib().moe_block_norm_backward(C.byref(a), torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
    c = (D / 64 + 24) * 2.0 ** -24
    hd = s["x"].double()
    total, mag = torch.zeros_like(hd), torch.zeros_like(hd)
    if dh:
        total, mag = total + s["dh"].double(), mag + s["dh"].double().abs()
    if du:
        g = s["du"].to(tu).double()
        a64, hh = g * s["w_pre"].double(), hd / rms(hd)
        total = total + (a64 - hh * (a64 * hh).mean(-1, keepdim=True)) / rms(hd)
        mag = mag + (a64.abs() + hh.abs() * (a64 * hh).abs().mean(-1, keepdim=True)) / rms(hd)
        col = (g * hh).abs().sum(0)
        assert ((grads["dw_pre"].double() - (g * hh).sum(0)).abs() <= col * (c + (T + 24) * 2.0 ** -24)).all()
    ref = (SCALE if post else 1.0) * total
    assert ((dx.m.double() - ref).abs() <= mag * c + (ref.abs() + mag * c) * HALF[tx] + TINY[tx]).all()
    assert dx.rest_is_untouched() and dy.rest_is_untouched()
    if not post:
        return
    yd, g, w = s["y"].double(), base.gate64(s, gate), s["w_post"].double()
    yh, q, qm = yd / rms(yd), total * g * w, mag * (g * w).abs()
    ref = (q - yh * (q * yh).mean(-1, keepdim=True)) / rms(yd)
    m = (qm + yh.abs() * (qm * yh.abs()).mean(-1, keepdim=True)) / rms(yd)
    assert ((dy.m.double() - ref).abs() <= m * 2 * c + (ref.abs() + m * 2 * c) * HALF[ty] + TINY[ty]).all()
    terms, tm = total * yh, mag * yh.abs()
    tol = (tm * g.abs()).sum(0) * (2 * c + (T + 24) * 2.0 ** -24)
    assert ((grads["dw_post"].double() - (terms * g).sum(0)).abs() <= tol).all()
    if gate == "channel":
        tol = tm.sum(0) * w.abs() * (2 * c + (T + 24) * 2.0 ** -24)
        assert ((grads["d_gate"].double() - (terms * w).sum(0)).abs() <= tol).all()
    elif gate == "token":
        assert ((grads["d_gate"].double() - (terms * w).sum(-1)).abs() <= (tm * w.abs()).sum(-1) * 3 * c).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,D,tx,ty,tw,gate", CASES)
@pytest.mark.parametrize("given", ["both", "dh", "du", "pre"])
def test_backward(T, D, tx, ty, tw, gate, given, layout):
    s = base.make(T, D, tx, ty, tw, gate, seed=T + D + 1)
    backward(s, T, D, tx, ty, tx, tw, gate, given, lambda i, t, data=None: place(layout, i, T, D, t, data))


OTHER = [(40, 264, "channel"), (333, 1001, "token"), (190, 7168, "channel"), (170, 7167, None), (41, 8200, "token"),
         (90, 16384, "channel"), (60, 16383, "token"), (1300, 72, "channel"), (3, 13, None)]


@pytest.mark.parametrize("T,D,gate", OTHER)
@pytest.mark.parametrize("tx,ty,tu", [(F32, F32, BF16), (F32, F32, F16), (F32, BF16, BF16), (BF16, BF16, F32), (BF16, F32, F32),
                                      (F16, F32, BF16), (F16, BF16, F32)])
@pytest.mark.parametrize("given", ["both", "du", "pre"])
def test_backward_with_du_of_another_type(T, D, gate, tx, ty, tu, given):
    """What a block whose input u has another type than its residual stream leads to."""
    s = base.make(T, D, tx, ty, F32, gate, seed=T + D + 2)
    backward(s, T, D, tx, ty, tu, F32, gate, given, lambda i, t, data=None: Matrix(T, D, t, data=data))


def test_views_of_the_bindings_callers():
    """Padded and shifted views as a program has them, through the binding, with the binding's own contiguous outputs."""
    T, D = 300, 1001
    s = base.make(T, D, BF16, BF16, F32, "channel", seed=5)
    kw = dict(w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per="channel", res_scale=SCALE, eps=EPS)
    du = s["du"].to(BF16)
    c = (D / 64 + 24) * 2.0 ** -24
    for off, ld in ((0, 1008), (1, 1001), (0, 1003), (8, 1008)):
        m = {n: Matrix(T, D, BF16, off, ld, t).m for n, t in (("x", s["x"]), ("dh", s["dh"]), ("du", du))}
        h, u = moe.block_norm(m["x"], s["y"], **kw)
        add = s["gate"].double() * s["w_post"].double() * s["y"].double() / rms(s["y"].double())
        ref = SCALE * s["x"].double() + add
        tol = add.abs() * c + ref.abs() * 2.0 ** -23
        assert ((h.double() - ref).abs() <= tol + (ref.abs() + tol) * HALF[BF16]).all()
        f = h.double()
        ref = s["w_pre"].double() * f / rms(f)
        assert ((u.double() - ref).abs() <= ref.abs() * (c + HALF[BF16] * (1 + c))).all()
        got = moe.block_norm_backward(m["dh"], m["du"], m["x"], s["y"], **kw)
        a, hh = du.double() * s["w_pre"].double(), s["x"].double() / rms(s["x"].double())
        total = s["dh"].double() + (a - hh * (a * hh).mean(-1, keepdim=True)) / rms(s["x"].double())
        mag = s["dh"].double().abs() + (a.abs() + hh.abs() * (a * hh).abs().mean(-1, keepdim=True)) / rms(s["x"].double())
        ref = SCALE * total
        assert ((got["dx"].double() - ref).abs() <= mag * c + (ref.abs() + mag * c) * HALF[BF16]).all()
        want = (du.double() * hh).sum(0)
        assert ((got["dw_pre"].double() - want).abs() <= (du.double() * hh).abs().sum(0) * (c + (T + 24) * 2.0 ** -24)).all()
