"""Calls that the header allows and a program seldom makes: outputs left out,
unaligned and strided codes, scales off 16 bytes, outputs past 32 bits, special
values of 16 bits, the block in place and captured with its side stream."""
import ctypes as C

import numpy as np
import pytest
import torch

import synth
import test_gpu_block_norm as norms
import test_gpu_mx4 as base
import moe_expert_layer_top16_gb300 as moe
from gpu_util import gpu_plan
from moe_expert_layer_top16_gb300 import block

pytestmark = pytest.mark.gpu

DEV = base.DEV
F32, BF16, F16 = base.F32, base.BF16, base.F16


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T,D,t", [(40, 264, BF16), (333, 1001, F32), (170, 7168, F32), (41, 16383, BF16)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_norm_gradients_with_outputs_left_out(T, D, t, gate):
    """Each output alone, and all but each: within the roundings of what the whole call gives (another instance may sum
    a row in another order: both are within (D / 64 + 24) 2^-24 of the magnitudes, as test_gpu_block_norm derives)."""
    s = norms.make(T, D, t, t, F32, gate, seed=1)
    du, code = s["du"].to(t), block.DTYPES[t]
    work = torch.empty(moe.lib().moe_block_norm_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    names = ("dx", "dy", "dw_post", "dw_pre", "d_gate")

    def call(want):
        out = dict(dx=torch.empty(T, D, dtype=t, device=DEV), dy=torch.empty(T, D, dtype=t, device=DEV),
                   dw_post=torch.empty(D, device=DEV), dw_pre=torch.empty(D, device=DEV),
                   d_gate=torch.empty(D if gate == "channel" else T, device=DEV))
        p = {n: out[n].data_ptr() if n in want else None for n in names}
        a = block._BlockNormBackwardArgs(
            s["dh"].data_ptr(), D, du.data_ptr(), D, s["x"].data_ptr(), D, s["y"].data_ptr(), D, s["w_post"].data_ptr(),
            s["w_pre"].data_ptr(), s["gate"].data_ptr(), p["dx"], D, p["dy"], D, p["dw_post"], p["dw_pre"], p["d_gate"],
            work.data_ptr(), work.numel(), T, D, code, code, code, 0, block.GATES[gate], 0.75, 1e-6)
        assert moe.lib().moe_block_norm_backward(C.byref(a), stream()) == moe.MOE_OK
        return {n: out[n] for n in want}

    c = (D / 64 + 24) * 2.0 ** -24
    d = lambda v: v.double()  # noqa: E731
    rms = norms.rms
    hh, a, yh = d(s["x"]) / rms(d(s["x"])), d(du) * d(s["w_pre"]), d(s["y"]) / rms(d(s["y"]))
    mag = d(s["dh"]).abs() + (a.abs() + hh.abs() * (a * hh).abs().mean(-1, keepdim=True)) / rms(d(s["x"]))
    g = norms.gate64(s, gate).abs()
    pm = mag * g * d(s["w_post"]).abs()
    tm, more = mag * yh.abs(), 2 * c + (T + 24) * 2.0 ** -24
    size = dict(dx=mag * c, dy=(pm + yh.abs() * (pm * yh.abs()).mean(-1, keepdim=True)) / rms(d(s["y"])) * 2 * c,
                dw_post=(tm * g).sum(0) * more, dw_pre=(d(du) * hh).abs().sum(0) * more,
                d_gate=tm.sum(0) * d(s["w_post"]).abs() * more if gate == "channel" else (tm * d(s["w_post"]).abs()).sum(-1) * 3 * c)
    ref = call(names)
    for want in [(n,) for n in names] + [tuple(m for m in names if m != n) for n in names]:
        for n, v in call(want).items():
            step = norms.HALF[v.dtype] * 2 * (ref[n].double().abs() + size[n]) if v.dtype != F32 else 0.0
            assert ((v.double() - ref[n].double()).abs() <= 2 * size[n] + step + 2.0 ** -149).all(), (want, n)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 8), (1, 0), (0, 1), (3, 5)])
def test_codec_on_any_rows(dtype, off, pad):
    """Quantise from and decode to rows that lie anyhow, special values among them; what lies round the rows stays."""
    rows, K = 37, 160
    g = torch.Generator(device=DEV).manual_seed(off + pad)
    x = torch.randn(rows, K, generator=g, device=DEV)
    x[3, 40], x[5, 0], x[6, 159], x[7, :32] = float("inf"), float("nan"), -float("inf"), 0.0
    x = x.to(dtype)
    ld, L = K + pad, moe.lib()
    flat = torch.full((off + rows * ld + 32,), 9.0, device=DEV).to(dtype)
    view = flat.as_strided((rows, K), (ld, 1), off)
    view.copy_(x)
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, K // 32, dtype=torch.uint8, device=DEV)
    t = block.DTYPES[dtype]
    assert L.moe_mxfp4_quantize(view.data_ptr(), ld, t, rows, K, codes.data_ptr(), scales.data_ptr(), stream()) == moe.MOE_OK
    special = torch.zeros(rows, K // 32, dtype=torch.bool, device=DEV)
    special[3, 1] = special[5, 0] = special[6, 4] = True
    ec, es = moe.mxfp4_encode(torch.where(special.repeat_interleave(32, 1), 0.0, x.float()))
    assert torch.equal(codes, ec) and torch.equal(scales, torch.where(special, torch.full_like(es, 255), es))
    assert (scales[7, 0] == 0) and (codes[7, :16] == 0).all()
    out = torch.full_like(flat, 9.0)
    to = out.as_strided((rows, K), (ld, 1), off)
    assert L.moe_mxfp4_decode(codes.data_ptr(), scales.data_ptr(), rows, K, to.data_ptr(), ld, t, stream()) == moe.MOE_OK
    want = base.values(codes, torch.where(special, torch.zeros_like(scales), scales)).to(F32).to(dtype).to(DEV)
    nan = special.repeat_interleave(32, 1)
    assert to[nan].isnan().all() and torch.equal(to[~nan], want[~nan])
    to.fill_(9.0)
    assert (out == 9.0).all()


@pytest.mark.parametrize("M,N", [(300, 37), (384, 700)])
def test_product_of_scales_off_16_bytes(M, N):
    """Scales 4 bytes behind a multiple of 16, K a multiple of 512: gathered instead of copied, the same bits."""
    K = 1024
    a, sa, b, sb = base.operands(2, 1, M, N, K)
    want = moe.mx4_gemm(a[0], sa[0], b, sb)

    def moved(t):
        flat = torch.empty(t.numel() + 4, dtype=torch.uint8, device=DEV)
        v = flat[4:].view(t.shape)
        v.copy_(t)
        return v

    assert torch.equal(moe.mx4_gemm(a[0], moved(sa[0]), b, moved(sb)), want)
    assert torch.equal(moe.mx4_gemm(a[0], sa[0], b, moved(sb)), want)


def test_product_past_32_bits():
    """An output of more than 2^31 elements: its corners."""
    M, N, K = 66_000, 33_000, 128
    a, sa, b, sb = base.operands(4, 1, M, N, K)
    out = moe.mx4_gemm(a[0], sa[0], b, sb, out_dtype=BF16)
    rows, cols = [0, 1, N // 2, N - 200, N - 1], [0, 127, 128, M // 2, M - 257, M - 1]
    av, bv = base.values(a[0][cols], sa[0][cols]), base.values(b[rows], sb[rows])
    exact, mag = bv @ av.T, bv.abs() @ av.abs().T
    tol = mag * ((K + 8) * 2.0 ** -22)
    got = out[rows][:, cols].double().cpu()
    assert ((got - exact).abs() <= tol + (exact.abs() + tol) * 2.0 ** -8).all()


@pytest.mark.parametrize("out,x_dtype", [("f32", F32), ("bf16", BF16), ("f32", F16)])
@pytest.mark.parametrize("T", [1, 33, 1100])
def test_block_in_place_and_captured(out, x_dtype, T):
    """moe_forward_block with h in x's memory and next_u in u's, eager and captured, two blocks in a row; at 1,100
    tokens the layer forks its side stream.  The same bits as the norms and the layer apart."""
    wl = synth.workload("tiny" if out == "f32" else "tiny+bf16")
    plan, _ = gpu_plan(wl, max_tokens=1200)
    g = torch.Generator(device=DEV).manual_seed(T)
    D = wl.d_model
    x0 = (2 * torch.randn(T, D, generator=g, device=DEV)).to(x_dtype)
    w, p, gate, n = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(4))
    x, u, y = x0.clone(), torch.empty(T, D, dtype=BF16, device=DEV), torch.empty(T, D, dtype=plan.out_dtype, device=DEV)

    def args(**kw):
        a = block._BlockArgs()
        for k, v in dict(x=x, u=u, y=y, h=x, next_u=u, w_post=p, gate=gate, next_w_pre=n, **kw).items():
            setattr(a, k, v.data_ptr())
        a.x_dtype, a.gate_kind, a.res_scale, a.eps = block.DTYPES[x_dtype], block.GATE_CHANNEL, 0.7, 1e-6
        return a

    first, second = args(w_pre=w), args()
    second.u_ready = 1

    def two_blocks():
        for a in (first, second):
            assert moe.lib().moe_forward_block(plan._h, C.byref(a), T, stream()) == moe.MOE_OK

    kw = dict(w_post=p, gate=gate, gate_per="channel", res_scale=0.7, u_dtype=BF16)
    _, ru = moe.block_norm(x0, w_pre=w, u_dtype=BF16)
    rh, ru = moe.block_norm(x0, plan.forward(ru), w_pre=n, **kw)
    rh, ru = moe.block_norm(rh, plan.forward(ru), w_pre=n, **kw)
    two_blocks()
    assert torch.equal(x, rh) and torch.equal(u, ru)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        two_blocks()
    for _ in range(2):
        x.copy_(x0)
        u.fill_(float("nan"))
        graph.replay()
        assert torch.equal(x, rh) and torch.equal(u, ru)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, _ = plan.forward_block(x0, w_pre=w, w_post=p, gate=gate, gate_per="channel", res_scale=0.7, next_w_pre=n, need_next_u=True,
                              stream=side)
    side.synchronize()
    assert torch.equal(h, moe.block_norm(x0, plan.forward(moe.block_norm(x0, w_pre=w, u_dtype=BF16)[1]), w_pre=n, **kw)[0])
    assert plan.device_status() == moe.MOE_OK
    plan.close()


def test_decode_norm_repeats_itself():
    """The same bits every time, with other inputs between, eager and replayed."""
    s, o = (norms.make(64, 7168, BF16, F32, F32, "channel", seed=i) for i in (1, 2))
    call = lambda s: moe.block_norm(s["x"], s["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per="channel")  # noqa: E731
    ref = [t.clone() for t in call(s)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call(s)
    for _ in range(20):
        call(o)
        assert all(torch.equal(a, b) for a, b in zip(ref, call(s)))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(ref, kept))


def test_numpy_is_not_a_tensor():
    for f in (lambda: moe.block_norm(np.zeros((4, 64))), lambda: moe.mxfp4_quantize([1.0])):
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.code == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("T,D", [(5, 264), (3, 16384), (9, 1001)])
@pytest.mark.parametrize("size,eps", [(1e17, 1e-6), (1e17, 0.0), (1e-17, 0.0)])
@pytest.mark.parametrize("t", [F32, BF16])
def test_norms_of_large_and_small_values(T, D, size, eps, t):
    """The magnitudes that moe.h names, 10^-18 to 10^17: within the usual bounds of the formulas in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(D)
    v = lambda *s: ((0.1 + 0.89 * torch.rand(*s, generator=g, device=DEV)) *      # noqa: E731
                    torch.where(torch.rand(*s, generator=g, device=DEV) < 0.5, -1.0, 1.0))
    x, y, du, dh = (v(T, D) * size).to(t), (v(T, D) * size).to(t), v(T, D).to(t), v(T, D).to(t)
    w = v(D)
    assert float(torch.maximum(x.abs().max(), y.abs().max())) <= 1e17 and float(torch.minimum(x.abs().min(), y.abs().min())) >= 9e-19
    rms = lambda a: (a.square().mean(-1, keepdim=True) + eps).sqrt()      # noqa: E731
    c = (D / 64 + 24) * 2.0 ** -24
    xd, yd, wd = x.double(), y.double(), w.double()
    h, u = moe.block_norm(x, y, w_post=w, w_pre=w, res_scale=0.75, eps=eps)
    add = wd * yd / rms(yd)
    ref = 0.75 * xd + add
    tol = add.abs() * c + ref.abs() * 2.0 ** -23
    assert ((h.double() - ref).abs() <= tol + (ref.abs() + tol) * base.HALF[t]).all()
    # the norm alone, of values of that size
    _, u = moe.block_norm(x, w_pre=w, eps=eps)
    ref = wd * xd / rms(xd)
    assert ((u.double() - ref).abs() <= ref.abs() * (c + base.HALF[t] * (1 + c))).all()
    got = moe.block_norm_backward(dh, du, x, y, w_post=w, w_pre=w, res_scale=0.75, eps=eps)
    a, hh = du.double() * wd, xd / rms(xd)
    total = dh.double() + (a - hh * (a * hh).mean(-1, keepdim=True)) / rms(xd)
    mag = dh.double().abs() + (a.abs() + hh.abs() * (a * hh).abs().mean(-1, keepdim=True)) / rms(xd)
    ref = 0.75 * total
    assert ((got["dx"].double() - ref).abs() <= mag * c + (ref.abs() + mag * c) * base.HALF[t]).all()
    yh, p, pm = yd / rms(yd), total * wd, mag * wd.abs()
    ref = (p - yh * (p * yh).mean(-1, keepdim=True)) / rms(yd)
    m = (pm + yh.abs() * (pm * yh.abs()).mean(-1, keepdim=True)) / rms(yd)
    keep = ref.abs() < 1e38                               # what the gradient's type holds
    assert ((got["dy"].double() - ref).abs() <= m * 2 * c + (ref.abs() + m * 2 * c) * base.HALF[t] + norms.TINY[t])[keep].all()
    terms, tm = (total * yh).sum(0), (mag * yh.abs()).sum(0)
    assert ((got["dw_post"].double() - terms).abs() <= tm * (2 * c + (T + 24) * 2.0 ** -24)).all()
