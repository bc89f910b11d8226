"""Four-bit activations and four-bit products: the quantiser against the
oracle's weight encoder (the same rule), the decoder against the table of
values, the product against the exact product in 64 bits.

The product's terms are exact in fp32; each one is added to the accumulator
with an error of at most two units in the last place of the running sum, so
that the result is within (K + 8) 2^-22 of the sum of magnitudes (the bound of
the MXFP8 engine's test), plus half a step of the output's type."""
import numpy as np
import pytest
import torch

import oracle
import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def values(codes, scales):
    """Codes and scales as float64 [..., K]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long().cpu()
    v = torch.where(c >= 8, -LEVELS[c & 7], LEVELS[c & 7])
    return v * torch.exp2(scales.cpu().double() - 127).repeat_interleave(32, -1)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (7, 96), (5, 3584), (130, 352)])
def test_quantise_is_the_weight_encoder(rows, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, K, generator=g, device=DEV) * torch.exp(3 * torch.randn(rows, 1, generator=g, device=DEV))
    x[:, :32] *= (torch.rand(rows, 1, generator=g, device=DEV) < 0.5)          # zero blocks
    x = x.to(dtype)
    codes, scales = moe.mxfp4_quantize(x)
    ec, es = moe.mxfp4_encode(x.float())
    assert torch.equal(codes, ec) and torch.equal(scales, es)
    oc, os_ = oracle.mxfp4_encode(x.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), oc) and np.array_equal(scales.cpu().numpy(), os_)
    ref = values(codes, scales)
    for out in (F32, BF16):
        assert torch.equal(moe.mxfp4_decode(codes, scales, out).cpu(), ref.to(F32).to(out))


def test_every_16_bit_value():
    """Each finite bf16 and fp16 value beside a largest one that sets the scale, ties among them."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    for dtype in (BF16, F16):
        v = bits.view(dtype)
        v = v[torch.isfinite(v.float())]
        for top in (1.0, 1.5, 448.0, 2.0 ** -10):
            small = v[v.float().abs() <= top]
            n = small.numel() // 31 * 31
            x = torch.cat((torch.full((n // 31, 1), top, dtype=dtype), small[:n].view(-1, 31)), 1).to(DEV)
            codes, scales = moe.mxfp4_quantize(x)
            ec, es = moe.mxfp4_encode(x.float())
            assert torch.equal(codes, ec) and torch.equal(scales, es)


def test_fp32_values_next_to_midpoints():
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = torch.cat([torch.nextafter(mids, torch.tensor(9.0)), mids, torch.nextafter(mids, torch.tensor(0.0)), torch.full((11,), 6.0)])
    for s in (1.0, 2.0 ** 100, 2.0 ** -120):
        for sign in (1, -1):
            row = (sign * s * x).view(1, 32).to(DEV)
            codes, scales = moe.mxfp4_quantize(row)
            want = torch.cat((torch.arange(1, 8), torch.arange(0, 7), torch.arange(0, 7), torch.full((11,), 7)))
            c = torch.stack((codes & 15, codes >> 4), -1).flatten().cpu()
            assert torch.equal((c & 7).long(), want) and (((c >> 3) == (sign < 0)) | (want == 0)).all()
            ec, es = moe.mxfp4_encode(row)
            assert torch.equal(codes, ec) and torch.equal(scales, es)


def test_extreme_and_special_values():
    big = torch.finfo(F32).max
    x = torch.zeros(6, 64)
    x[0, 0], x[1, 0], x[2, 0] = big, 2.0 ** -149, 2.0 ** -126
    x[3, 5], x[4, 40], x[5, 7] = float("inf"), float("nan"), -float("inf")
    x[:, 1] = 2.0 ** -149
    codes, scales = moe.mxfp4_quantize(x.to(DEV))
    ec, es = moe.mxfp4_encode(x[:3].to(DEV))
    assert torch.equal(codes[:3], ec) and torch.equal(scales[:3], es)
    assert scales[3:].tolist() == [[255, 0], [0, 255], [255, 0]]
    assert (codes[3, :16] == 0).all() and (codes[4, 16:] == 0).all()
    v = moe.mxfp4_decode(codes, scales).cpu()
    assert v[3, :32].isnan().all() and v[4, 32:].isnan().all() and v[5, :32].isnan().all()
    assert not v[3, 32:].isnan().any() and not v[4, :32].isnan().any()
    # every code and scale decodes to its value
    all_codes = torch.arange(256, dtype=torch.uint8).view(16, 16).repeat(255, 1, 1).to(DEV)
    all_scales = torch.arange(255, dtype=torch.uint8).view(255, 1, 1).repeat(1, 16, 1).to(DEV)
    assert torch.equal(moe.mxfp4_decode(all_codes, all_scales).cpu(), values(all_codes, all_scales).float())
    assert torch.equal(moe.mxfp4_decode(all_codes, all_scales, F16).cpu(), values(all_codes, all_scales).to(F16))


def test_quantise_strided_rows():
    wide = torch.randn(9, 200, device=DEV)
    for x in (wide[:, :96], wide[:, 1:97], wide[:, 8:104], wide[:, ::2][:, :96]):
        a, b = moe.mxfp4_quantize(x), moe.mxfp4_quantize(x.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c, s = moe.mxfp4_quantize(wide.bfloat16()[:, 3:99])
    d, t = moe.mxfp4_quantize(wide.bfloat16()[:, 3:99].contiguous())
    assert torch.equal(c, d) and torch.equal(s, t)
    c, s = moe.mxfp4_quantize(torch.empty(0, 64, device=DEV))
    assert c.shape == (0, 32) and moe.mxfp4_decode(c, s).shape == (0, 64)


def operands(seed, G, M, N, K):
    g = torch.Generator(device=DEV).manual_seed(seed)
    b8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)  # noqa: E731
    return b8(0, 256, G, M, K // 2), b8(116, 130, G, M, K // 32), b8(0, 256, N, K // 2), b8(120, 134, N, K // 32)


def check(ops, bounds, out, dtype, K):
    ac, as_, bc, bs = ops
    for g in range(ac.shape[0]):
        lo, hi = bounds[g], bounds[g + 1]
        if lo == hi:
            continue
        a, b = values(ac[g], as_[g]).to(DEV), values(bc[lo:hi], bs[lo:hi]).to(DEV)
        exact, mag = b @ a.T, b.abs() @ a.abs().T
        tol = mag * ((K + 8) * 2.0 ** -22)
        tol = tol + (exact.abs() + tol) * HALF[dtype]
        got = out[lo:hi].double()
        assert torch.isfinite(got).all() and ((got - exact).abs() <= tol).all(), f"group {g}"


@pytest.mark.parametrize("M,N,K,dtype", [
    (128, 16, 256, F32), (128, 16, 128, F32), (128, 1, 512, F32), (1, 1, 128, BF16), (7, 3, 384, F16), (200, 17, 256, F32),
    (256, 33, 640, BF16), (384, 64, 3584, F32), (130, 65, 896, F32), (512, 129, 512, F16), (1000, 224, 1024, BF16),
    (129, 225, 384, F32), (8192, 300, 256, BF16), (640, 1000, 7168, F32), (33, 4000, 128, F32), (20000, 5, 256, BF16)])
def test_product(M, N, K, dtype):
    ops = operands(M + N, 1, M, N, K)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = moe.mx4_gemm(ops[0][0], ops[1][0], ops[2], ops[3], out_dtype=dtype, status=status)
    assert out.shape == (N, M) and out.dtype == dtype and status.item() == 0
    check(ops, [0, N], out, dtype, K)


@pytest.mark.parametrize("G,M,K,counts,dtype", [
    (2, 128, 256, [3, 0], F32), (3, 64, 384, [0, 0, 0], F32), (5, 100, 128, [1, 40, 0, 300, 17], BF16),
    (64, 256, 512, [i % 3 for i in range(64)], F32), (7, 130, 640, [500, 1, 2, 0, 0, 16, 15], F16),
    (1024, 8, 128, [1] * 1024, F32), (33, 300, 256, [33] * 33, BF16)])
@pytest.mark.parametrize("lead", [0, 5])
def test_grouped_product(G, M, K, counts, dtype, lead):
    N = lead + sum(counts) + 3
    ops = operands(G, G, M, N, K)
    bounds = (lead + np.concatenate([[0], np.cumsum(counts)])).tolist()
    offsets = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    keep = torch.full((N, M + 4), 7.0, device=DEV).to(dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = moe.mx4_gemm(*ops, offsets=offsets, out=keep[:, :M], status=status)
    assert status.item() == 0
    check(ops, bounds, out, dtype, K)
    # rows outside the groups, and what lies behind a row, stay
    assert (keep[:bounds[0]] == 7).all() and (keep[bounds[-1]:] == 7).all() and (keep[:, M:] == 7).all()


def test_one_hot_rows_pick_weight_columns():
    """A row with a single 1 at k returns column k of the weights, exactly: places of every code and scale."""
    M, K = 200, 640
    ops = operands(5, 1, M, K, K)
    x = torch.eye(K, device=DEV)
    codes, scales = moe.mxfp4_quantize(x)
    out = moe.mx4_gemm(ops[0][0], ops[1][0], codes, scales)
    assert torch.equal(out.cpu().double(), values(ops[0][0], ops[1][0]).T)


def test_not_a_number_stays_in_its_row():
    M, N, K = 256, 40, 512
    ops = operands(6, 1, M, N, K)
    ref = moe.mx4_gemm(ops[0][0], ops[1][0], ops[2], ops[3])
    ops[3][9, 4] = 255
    out = moe.mx4_gemm(ops[0][0], ops[1][0], ops[2], ops[3])
    keep = [i for i in range(N) if i != 9]
    assert torch.equal(out[keep], ref[keep]) and out[9].isnan().all()


def test_offsets_outside_the_rows_are_kept_inside():
    ops = operands(7, 2, 128, 20, 256)
    offsets = torch.tensor([-3, 12, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out = moe.mx4_gemm(*ops, offsets=offsets)
    check(ops, [0, 12, 20], out, F32, 256)


def test_empty_product():
    ops = operands(8, 1, 128, 4, 256)
    out = moe.mx4_gemm(ops[0][0], ops[1][0], ops[2][:0], ops[3][:0])
    assert out.shape == (0, 128)


@pytest.mark.parametrize("N,M,K", [(73, 256, 1024), (600, 512, 512), (9, 384, 128)])
def test_operands_written_just_before(N, M, K):
    """The product's launch overlaps the kernel before it: both operands written by that kernel, in memory that earlier
    calls have used, and its output read by the next, without a wait between them."""
    g = torch.Generator(device=DEV).manual_seed(N)
    xs = [torch.randn(N, K, generator=g, device=DEV) for _ in range(12)]
    ws = [torch.randn(M, K, generator=g, device=DEV) for _ in range(12)]
    out = [moe.mx4_gemm(*moe.mxfp4_quantize(w), *moe.mxfp4_quantize(x)) for x, w in zip(xs, ws)]
    back = [moe.mx4_gemm(*moe.mxfp4_quantize(x), *moe.mxfp4_quantize(w)) for x, w in zip(xs, ws)]
    again = [moe.mxfp4_quantize(o) for o in out] if M % 32 == 0 else []
    torch.cuda.synchronize()
    for i, (x, w) in enumerate(zip(xs, ws)):
        a, b = moe.mxfp4_quantize(w), moe.mxfp4_quantize(x)
        torch.cuda.synchronize()
        ref = moe.mx4_gemm(*a, *b)
        torch.cuda.synchronize()
        assert torch.equal(out[i], ref)
        # the other way round: the same products added in another grouping of rows, the same order of K
        assert torch.equal(back[i], ref.t())
        if again:
            q = moe.mxfp4_quantize(ref)
            assert torch.equal(again[i][0], q[0]) and torch.equal(again[i][1], q[1])
