"""One matrix and a second one with SiLU, as the shared experts' gate and up, for
one to many rows; rows that shared memory does not hold at once; and the ranges
of numbers and the dropped slots that the header allows.

Tolerances are those that test_gpu_w4_matvec.py derives."""
import math

import pytest
import torch

import test_gpu_w4_matvec as mv
import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def pair(M, K, form, seed):
    return mv.weights((M, K), form, seed), mv.weights((M, K), form, seed + 1)


def check(x, gate, up, **kw):
    vg, vu = mv.values(*gate), mv.values(*up)
    a, b, ea, eb = x.double() @ vg.T, x.double() @ vu.T, mv.bound(vg, x), mv.bound(vu, x)
    s = a * torch.sigmoid(a)
    got = moe.w4_matvec(x, *gate, up=up, **kw)
    mv.close(got, s * b, 1.1 * ea * b.abs() + (s.abs() + 1.1 * ea) * eb + 8 * U * (s * b).abs())
    return got


@pytest.mark.parametrize("form", mv.FORMS, ids=str)
@pytest.mark.parametrize("N,M,K", [(1, 1, 128), (1, 50, 384), (2, 33, 896), (3, 17, 1152), (4, 100, 256), (5, 40, 640), (8, 31, 384), (9, 16, 256), (17, 37, 128)])
def test_one_matrix_and_up(N, M, K, form):
    for dtype in (F32, BF16, F16):
        x = mv.rows(N, K, dtype, N + K)
        check(x, *pair(M, K, form, M), out_dtype=F32)
        if dtype != F16:                                     # (a product of two such sums leaves fp16's range)
            check(x, *pair(M, K, form, M))


@pytest.mark.parametrize("form", ["mxfp4", (32, F32), (64, BF16), (128, F16)], ids=str)
@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 9])
def test_the_hidden_width(N, form):
    """K = 7,168: x of five rows, or of two in fp32, goes to shared memory in parts, for each round of tiles anew; more
    tiles than blocks take at once."""
    for dtype in (F32, BF16):
        x = mv.rows(N, 7168, dtype, N)
        got = check(x, *pair(48, 7168, form, 5), out_dtype=F32)
        assert torch.equal(got, moe.w4_matvec(x, *pair(48, 7168, form, 5)[0], up=pair(48, 7168, form, 5)[1], out_dtype=F32))
    gate, up = pair(5000, 7168, form, 8)
    x = mv.rows(N, 7168, BF16, N)
    check(x, gate, up)
    v = mv.values(*gate)
    mv.close(moe.w4_matvec(x.float(), *gate), x.double() @ v.T, mv.bound(v, x.float()))


def test_rows_do_not_depend_on_their_neighbours():
    """NaN and infinities of a row stay in it; a row's result is the same whatever the others are."""
    gate, up = pair(40, 512, "mxfp4", 3)
    x = mv.rows(8, 512, BF16, 4)
    want = moe.w4_matvec(x, *gate, up=up)
    z = x.clone()
    z[2], z[5, 7], z[6] = math.nan, math.inf, 0
    got = moe.w4_matvec(z, *gate, up=up)
    keep = [0, 1, 3, 4, 7]
    assert torch.equal(got[keep], want[keep]) and got[2].isnan().all() and (got[6] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided(dtype):
    """Rows and outputs with space between them, rows off 16 bytes, the transposed matrix of rows."""
    N, M, K = 6, 37, 416
    gate, up = pair(M, K, "mxfp4", 6)
    packed = mv.rows(N, K, dtype, 4)
    want = check(packed, gate, up)
    for pad, shift in ((8, 0), (3, 0), (8, 1)):
        store = torch.full((N, K + pad + shift), math.nan, device=DEV, dtype=dtype)
        x = store[:, shift:shift + K]
        x.copy_(packed)
        out = torch.full((N, M + 5), 77.0, device=DEV, dtype=dtype)
        moe.w4_matvec(x, *gate, up=up, out=out[:, 2:2 + M])
        assert torch.equal(out[:, 2:2 + M], want) and (out[:, :2] == 77).all() and (out[:, 2 + M:] == 77).all()
    assert torch.equal(moe.w4_matvec(packed.t().contiguous().t(), *gate, up=up), want)


def test_captured():
    """Replayed with new rows, beside an eager call."""
    gate, up = pair(300, 1024, (64, BF16), 2)
    x = mv.rows(5, 1024, BF16, 1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        moe.w4_matvec(x, *gate, up=up)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = moe.w4_matvec(x, *gate, up=up)
    for seed in (1, 7):
        x.copy_(mv.rows(5, 1024, BF16, seed))
        g.replay()
        want = check(x, gate, up)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ------------------------------------------------------------------ what is not read
@pytest.mark.parametrize("form", ["mxfp4", (64, BF16)], ids=str)
def test_dropped_slots_are_not_read(form):
    """NaN in the weights and rows of dropped slots, and in the matrices of experts that no slot names."""
    T, k, E, M, K = 5, 6, 7, 40, 256
    idx = mv.slots(T, k, E, 3)
    idx = torch.where(idx == 2, 3, idx)
    off = (idx < 0) | (idx >= E)
    assert off.any()
    gate, up = mv.weights((E, M, K), form, 1), mv.weights((E, M, K), form, 2)
    x, w = mv.rows(T * k, K, BF16, 4).view(T, k, K), torch.randn(T, k, generator=mv.gen(5), device=DEV)
    calls = (lambda: moe.w4_matvec(x, *gate, idx=idx), lambda: moe.w4_matvec(x, *gate, idx=idx, up=up), lambda: moe.w4_matvec(x, *gate, idx=idx, weights=w))
    want = [f() for f in calls]
    x[off], w[off] = math.nan, math.inf
    for m in (gate, up):
        m[1][2] = 255 if form == "mxfp4" else math.nan
    for f, y in zip(calls, want):
        got = f()
        assert got.isfinite().all() and torch.equal(got, y)


# ------------------------------------------------------------------ how large and how small
@pytest.mark.parametrize("form", ["mxfp4", (32, F32), (64, BF16)], ids=str)
@pytest.mark.parametrize("x_e,s_e,w_e", [(-60, 60, 0), (60, -60, 0), (0, 62, 48), (-30, -30, 60), (60, 62, -60), (62, -40, 62), (62, 30, None), (-62, 62, None), (-40, -40, None)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_numbers_below_2_to_the_63rd(dtype, x_e, s_e, w_e, form):
    """Rows, scales and weights up to 2^63 in magnitude: nothing on the way overflows that the sum does not.  (3 x 448 terms
    of 1.9 x 8 x 2^112 at most stay below 2^127.)"""
    T, k, E, M, K = 2, 3, 4, 24, 416 if form != (64, BF16) else 448
    codes, scales = mv.weights((E, M, K), form, 1, spread=2)
    scales = (scales.int() + s_e - 2).to(torch.uint8) if form == "mxfp4" else (scales.double() * 2.0 ** s_e).to(scales.dtype)
    x = torch.randn(T, K, generator=mv.gen(2), device=DEV).clamp(-1.9, 1.9).double().mul(2.0 ** x_e).to(dtype)
    v = mv.values(codes, scales)
    idx = torch.tensor([[0, 1, 3], [2, -1, 2]], dtype=torch.int32, device=DEV)
    if w_e is None:
        y, err = x[:1].double() @ v[0].T, mv.bound(v[0], x[:1])
        mv.close(moe.w4_matvec(x[:1], codes[0], scales[0], out_dtype=F32), y, err)
        return
    w = (torch.rand(T, k, generator=mv.gen(3), device=DEV).double() * 2.0 ** w_e).float()
    y, size = torch.zeros(T, M, dtype=torch.float64, device=DEV), torch.zeros(T, M, dtype=torch.float64, device=DEV)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if e >= 0:
                p = (x[t:t + 1].double() @ v[e].T)[0] * w[t, j].double()
                y[t] += p
                size[t] += mv.bound(v[e], x[t:t + 1])[0] * w[t, j].double() * (1 + k * K / 64 / 128) + 64 * U * p.abs()
    mv.close(moe.w4_matvec(x, codes, scales, idx=idx, weights=w, out_dtype=F32), y, size)
