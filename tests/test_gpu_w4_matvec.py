"""Products of a few rows with four-bit weights against the same sums in 64 bits.

Tolerance of a product, in units u = 2^-24 of sum |w x|: the products are exact
in fp32; 32 of them are added by eight MMAs at most, each off by 8 u (sixteen
terms aligned to the largest and cut): 64 u.  A group's sum meets two factors
and a sum over K / 32 groups, in eight warps: K / 256 + 2 additions, twice u each
for the truncated ones, then 8 warps times 3 parts: 128 u + K / 64 u covers them.
x is off by 2^-39 of the largest in its 32 (16-bit types; fp32: 2^-63), for 32
values of it.  SiLU passes on 1.1 of its argument's error, and its own exponential,
quotient and products are off by 8 u.  The output is off by half a step of its type."""
import math

import pytest
import torch

import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def weights(shape, form, seed, spread=3):
    """Random codes, and scales of uneven size: (codes, scales).  form: 'mxfp4' or (group, type)."""
    *lead, K = shape
    g = gen(seed)
    codes = torch.randint(0, 256, (*lead, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    if form == "mxfp4":
        return codes, torch.randint(127 - spread, 128 + spread, (*lead, K // 32), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    group, dtype = form
    return codes, (torch.randn(*lead, K // group, generator=g, device=DEV) * 0.1).to(dtype)


def values(codes, scales):
    """What they stand for, in 64 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    if scales.dtype == torch.uint8:
        v = torch.tensor(LEVELS + [-x for x in LEVELS], dtype=torch.float64, device=DEV)[c]
        s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127))
    else:
        v, s = c.double() - 8, scales.double()
    return v * s.repeat_interleave(v.shape[-1] // s.shape[-1], -1)


def bound(w, x, K=None):
    """Error of the products of w [M][K] with x [..., K] before rounding to the output's type."""
    K = K or w.shape[-1]
    top = x.double().abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(*x.shape[:-1], -1, 32).flatten(-2)
    lost = 2.0 ** (-63 if x.dtype == F32 else -39) * top
    return (x.double().abs() @ w.abs().T) * (128 + K / 64) * U + lost @ w.abs().T


def close(got, want, err):
    step = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else U
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    assert got.isfinite().all()
    assert ((got.double() - want).abs() <= err * (1 + step) + want.abs() * step + tiny).all()


def rows(N, K, dtype, seed):
    g = gen(seed)
    return (torch.randn(N, K, generator=g, device=DEV) * torch.exp(torch.randn(N, 1, generator=g, device=DEV))).to(dtype)


FORMS = ["mxfp4"] + [(g, t) for g in (32, 64, 128) for t in (F16, BF16, F32)]


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("N,M,K", [(1, 1, 128), (1, 16, 128), (1, 17, 384), (2, 100, 896), (3, 33, 1152), (4, 64, 256), (5, 48, 3584), (8, 40, 640), (9, 40, 512),
                                   (17, 20, 128), (1, 300, 7168), (4, 31, 7168)])
def test_one_matrix(N, M, K, form):
    for dtype in (F32, BF16, F16):
        x = rows(N, K, dtype, N + K)
        w = weights((M, K), form, M + K)
        v = values(*w)
        want, err = x.double() @ v.T, bound(v, x)
        close(moe.w4_matvec(x, *w), want, err)
        close(moe.w4_matvec(x, *w, out_dtype=F32), want, err)


@pytest.mark.parametrize("N,M,K", [(1, 5, 32), (2, 16, 96), (3, 17, 1056), (8, 9, 160), (1, 40, 992), (2, 40, 224), (6, 33, 7136)])
@pytest.mark.parametrize("form", ["mxfp4", (32, F16), (32, BF16), (32, F32)], ids=str)
def test_odd_numbers_of_groups(N, M, K, form):
    """Scales of a row that start on odd places, the last unit of K part filled."""
    for dtype in (F32, BF16):
        x, w = rows(N, K, dtype, K), weights((M, K), form, K)
        v = values(*w)
        close(moe.w4_matvec(x, *w, out_dtype=F32), x.double() @ v.T, bound(v, x))


@pytest.mark.parametrize("form", ["mxfp4", (64, BF16)], ids=str)
def test_one_row_and_none(form):
    w = weights((40, 256), form, 1)
    x = rows(3, 256, BF16, 2)
    y = moe.w4_matvec(x[1], *w)
    assert y.shape == (40,) and torch.equal(y, moe.w4_matvec(x[1:2], *w)[0])
    assert moe.w4_matvec(x[:0], *w).shape == (0, 40)
    w3 = weights((4, 40, 256), form, 1)
    none = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    assert moe.w4_matvec(x[:0], *w3, idx=none).shape == (0, 3, 40)
    assert moe.w4_matvec(x[:0], *w3, idx=none, weights=torch.zeros(0, 3, device=DEV)).shape == (0, 40)


def slots(T, k, E, seed):
    """Experts with some slots dropped (on both sides of the range), one token without any, one expert twice."""
    g = gen(seed)
    idx = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    r = torch.rand(T, k, generator=g, device=DEV)
    idx = torch.where(r < 0.15, -1, torch.where(r > 0.9, E, idx))
    if T > 1:
        idx[T - 1] = -5
    if k > 1:
        idx[0, 1] = idx[0, 0] = E - 1
    else:
        idx[0, 0] = E - 1
    return idx.contiguous()


CASES = [(1, 16, 20, 64, 3584), (3, 4, 7, 33, 256), (2, 1, 1, 5, 32), (5, 8, 3, 48, 416), (1, 32, 40, 17, 128), (9, 2, 5, 16, 128)]


@pytest.mark.parametrize("form", ["mxfp4", (32, F32), (64, BF16), (128, F16)], ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,k,E,M,K", CASES)
def test_experts_of_slots(T, k, E, M, K, dtype, form):
    if form != "mxfp4":
        K = (K + form[0] - 1) // form[0] * form[0]
    idx = slots(T, k, E, T + k)
    gate, up = weights((E, M, K), form, 3), weights((E, M, K), form, 4)
    vg, vu = values(*gate), values(*up)
    weight = torch.randn(T, k, generator=gen(6), device=DEV)
    for per_slot in (False, True):
        x = rows(T * k if per_slot else T, K, dtype, 5)
        x = x.view(T, k, K) if per_slot else x
        each = x if per_slot else x.unsqueeze(1).expand(T, k, K)
        want, err, silu, silu_err = (torch.zeros(T, k, M, dtype=torch.float64, device=DEV) for _ in range(4))
        for t in range(T):
            for j in range(k):
                e = int(idx[t, j])
                if 0 <= e < E:
                    r = each[t, j:j + 1]
                    a, b = (r.double() @ vg[e].T)[0], (r.double() @ vu[e].T)[0]
                    ea, eb = bound(vg[e], r)[0], bound(vu[e], r)[0]
                    want[t, j], err[t, j] = a, ea
                    s = a * torch.sigmoid(a)
                    silu[t, j], silu_err[t, j] = s * b, 1.1 * ea * b.abs() + (s.abs() + 1.1 * ea) * eb + 8 * U * (s * b).abs()
        got = moe.w4_matvec(x, *gate, idx=idx)
        close(got, want, err)
        assert (got[(idx < 0) | (idx >= E)] == 0).all()
        close(moe.w4_matvec(x, *gate, idx=idx, up=up, out_dtype=F32), silu, silu_err)
        # over a token's slots: the sum's magnitudes, and a chain k times as long
        y = (want * weight.double().unsqueeze(-1)).sum(1)
        size = (err * weight.double().abs().unsqueeze(-1)).sum(1) * (1 + k * K / 64 / 128) + 64 * U * (want * weight.double().unsqueeze(-1)).abs().sum(1)
        got = moe.w4_matvec(x, *gate, idx=idx, weights=weight)
        close(got, y, size)
        if T > 1:
            assert (got[T - 1] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_of_x_than_shared_memory_holds(dtype):
    """Units of K staged in several rounds: long rows, several of them, and a token's many slots."""
    for N, K in ((1, 65536), (4, 16384), (8, 40960)):
        x, w = rows(N, K, dtype, K), weights((33, K), "mxfp4", 1)
        v = values(*w)
        close(moe.w4_matvec(x, *w, out_dtype=F32), x.double() @ v.T, bound(v, x))
    T, k, E, M, K = 2, 32, 9, 24, 7168
    idx = torch.randint(0, E, (T, k), generator=gen(2), device=DEV, dtype=torch.int32)
    idx[1, ::2] = -1
    x, w, weight = rows(T * k, K, dtype, 3).view(T, k, K), weights((E, M, K), "mxfp4", 4), torch.randn(T, k, generator=gen(5), device=DEV)
    v = values(*w)
    want = torch.stack([sum(weight[t, j].double() * (v[int(idx[t, j])] @ x[t, j].double()) for j in range(k) if idx[t, j] >= 0) for t in range(T)])
    size = torch.stack([sum(weight[t, j].double().abs() * bound(v[int(idx[t, j])], x[t, j:j + 1], k * K)[0] for j in range(k) if idx[t, j] >= 0) for t in range(T)])
    close(moe.w4_matvec(x, *w, idx=idx, weights=weight, out_dtype=F32), want, size * 2)


def test_codes_one_by_one():
    """Every code at every place of a group, alone: exact."""
    K = 128
    eye = torch.eye(K, device=DEV)
    for form in ("mxfp4", (32, F32)):
        codes = torch.randint(0, 256, (64, K // 2), generator=gen(1), device=DEV, dtype=torch.uint8)
        codes[:16] = torch.arange(16, device=DEV, dtype=torch.uint8)[:, None] * 17
        scales = torch.full((64, K // 32), 128, dtype=torch.uint8, device=DEV) if form == "mxfp4" else torch.full((64, K // 32), 2.0, device=DEV)
        v = values(codes, scales)
        for dtype in (F32, BF16, F16):
            assert torch.equal(moe.w4_matvec(eye.to(dtype), codes, scales, out_dtype=F32).double(), v.T)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_values_of_very_different_size(dtype):
    """Largest values that meet zero weights: what lies below them is kept down to 2^-28 (fp32: 2^-39) exactly."""
    K, M = 256, 32
    codes = torch.full((M, K // 2), 0x72, dtype=torch.uint8, device=DEV)      # 1 and 6
    codes[:, ::16] = 0x70                                                      # the first of each 32 meets zero
    scales = torch.full((M, K // 32), 127, dtype=torch.uint8, device=DEV)
    v = values(codes, scales)
    g = gen(1)
    small = 2.0 ** (-39 if dtype == F32 else -13)
    sign = torch.randint(0, 2, (3, K), generator=g, device=DEV) * 2 - 1
    x = (sign * (1 + torch.rand(3, K, generator=g, device=DEV)) * small).to(dtype)
    inside = x.double().clone()
    x[:, ::32] = 1.0 if dtype == F32 else 2.0 ** 15
    inside[:, ::32] = 0
    close(moe.w4_matvec(x, codes, scales, out_dtype=F32), x.double() @ v.T, (inside.abs() @ v.abs().T) * (128 + K / 64) * U)
    # tiny and large rows: nothing underflows or overflows on the way
    for size in ((1e-38, 1e-30, 1e30) if dtype != F16 else (1e-7, 6e4)):
        x = (torch.randn(3, K, generator=gen(2), device=DEV) * size).clamp(-6.5e4 if dtype == F16 else -3e38, 6.5e4 if dtype == F16 else 3e38).to(dtype)
        close(moe.w4_matvec(x, codes, scales, out_dtype=F32), x.double() @ v.T, bound(v, x) + 1e-43)


def test_infinities_and_nan():
    K, M = 256, 40
    codes, scales = weights((M, K), "mxfp4", 1)
    v = values(codes, scales)
    for dtype in (F32, BF16, F16):
        x = rows(4, K, dtype, 2)
        x[0, 3], x[1, 100], x[2, 50], x[2, 51] = math.inf, math.nan, math.inf, -math.inf
        want = (x.double().unsqueeze(1) * v).sum(-1)
        got = moe.w4_matvec(x, codes, scales, out_dtype=F32).double()
        bad = ~want.isfinite()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[bad & ~want.isnan()], want[bad & ~want.isnan()])
        close(got[~bad].float(), want[~bad], bound(v, x.nan_to_num(0, 0, 0))[~bad])
    scales[5, 2] = 255                              # not a number
    x = rows(2, K, BF16, 3)
    got = moe.w4_matvec(x, codes, scales)
    assert got[:, 5].isnan().all() and got[:, :5].isfinite().all() and got[:, 6:].isfinite().all()
    scales[5, 2] = 0                                # 2^-127
    close(moe.w4_matvec(x, codes, scales), x.double() @ values(codes, scales).T, bound(values(codes, scales), x))


# ------------------------------------------------------------------ how they lie
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1), (16, 8)])
def test_strided_rows_and_outputs(dtype, pad, shift):
    N, M, K = 5, 37, 384
    store = torch.full((N, K + pad + shift), math.nan, device=DEV, dtype=dtype)
    x = store[:, shift:shift + K]
    x.copy_(rows(N, K, dtype, 4))
    w = weights((M, K), "mxfp4", 5)
    packed = moe.w4_matvec(x.contiguous(), *w)
    assert torch.equal(moe.w4_matvec(x, *w), packed)
    assert torch.equal(moe.w4_matvec(x.t().contiguous().t(), *w), packed)
    out = torch.full((N, M + 11), 77.0, device=DEV, dtype=dtype)
    assert moe.w4_matvec(x, *w, out=out[:, 3:3 + M]).data_ptr() == out[:, 3:].data_ptr()
    assert torch.equal(out[:, 3:3 + M], packed) and (out[:, :3] == 77).all() and (out[:, 3 + M:] == 77).all()
    idx = slots(N, 2, 4, 1)
    w = weights((4, M, K), "mxfp4", 6)
    big = torch.full((N * 2 + 2, M), 77.0, device=DEV, dtype=dtype)
    got = moe.w4_matvec(x, *w, idx=idx, out=big[1:-1].view(N, 2, M))
    assert torch.equal(got, moe.w4_matvec(x.contiguous(), *w, idx=idx)) and (big[0] == 77).all() and (big[-1] == 77).all()


@pytest.mark.parametrize("form,size", [("mxfp4", 1), ((32, F16), 2), ((32, F32), 4)], ids=str)
def test_scales_on_odd_addresses(form, size):
    """Scales whose pairs straddle words."""
    M, K = 20, 256
    codes, scales = weights((M, K), form, 7)
    store = torch.empty(scales.numel() + 1, dtype=scales.dtype, device=DEV)
    moved = store[1:].view_as(scales)
    moved.copy_(scales)
    x = rows(2, K, BF16, 8)
    assert moved.data_ptr() % (2 * size) and torch.equal(moe.w4_matvec(x, codes, moved), moe.w4_matvec(x, codes, scales))


def test_codes_past_31_bits():
    """The last of so many matrices that their bytes pass 2^31."""
    E, M, K = 1300, 1024, 3584
    codes = torch.zeros(E, M, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.full((E, M, K // 32), 127, dtype=torch.uint8, device=DEV)
    last = weights((M, K), "mxfp4", 1)
    codes[-1], scales[-1] = last
    x = rows(1, K, BF16, 2)
    idx = torch.tensor([[E - 1, 0]], dtype=torch.int32, device=DEV)
    got = moe.w4_matvec(x, codes, scales, idx=idx)
    v = values(*last)
    close(got[0, 0], (x.double() @ v.T)[0], bound(v, x)[0])
    assert (got[0, 1] == 0).all()


def test_agrees_with_the_product_of_decoded_weights():
    """mxfp4_quantize's codes and scales, as mxfp4_decode reads them."""
    codes, scales = moe.mxfp4_quantize(rows(200, 1024, F32, 1))
    x = rows(2, 1024, BF16, 2)
    v = moe.mxfp4_decode(codes, scales).double()
    close(moe.w4_matvec(x, codes, scales, out_dtype=F32), x.double() @ v.T, bound(v, x))
