"""Rows at which the router's operators can go wrong and that their other tests
do not have: equal keys on both sides of the last slot with a nearer key behind
them.

The order is compared with that of keys in 64 bits, exactly; gates within the
tolerance that test_gpu_router_ops.py derives."""
import math

import pytest
import torch

import test_gpu_router_ops as ops
import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
INF, NAN = math.inf, math.nan
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


# ------------------------------------------------------------------ equal keys round the last slot
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("row,E", [((20, 20, 20.125), 32), ((20, 20, 21), 3), ((-30, -30, -29), 3), ((-30, -30, -29), 40), ((20, 20, 20, 20, 30), 61),
                                   ((30, 30, 20, 20, 40), 61)])
def test_a_larger_key_behind_two_equal_ones(row, E, dtype):
    """k = 1: in 32 bits all of these keys are alike, the last one is the largest."""
    low = -5.0 if row[0] > 0 else -60.0
    x = torch.full((1, E), low, device=DEV)
    x[0, :len(row)] = torch.tensor(row, dtype=F32, device=DEV)
    x = x.to(dtype)
    idx, _ = ops.check_selection(x, 1, bias=torch.zeros(E, device=DEV))
    assert idx.item() == len(row) - 1


@pytest.mark.parametrize("more", [0, 30, 80])
@pytest.mark.parametrize("base", [20.0, -30.0])
@pytest.mark.parametrize("large", [0.0, 3.0, -1000.0])
@pytest.mark.parametrize("k", [1, 2, 4, 16, 32])
@pytest.mark.parametrize("apart", [False, True])
def test_equal_keys_across_the_last_slot(apart, k, large, base, more):
    """k - 1 winners well above; a pair equal in logit and bias for the last slot; behind it, by number, a truly larger key
    that 32 bits do not tell from the pair.  `more` further experts equal to the pair make candidates overflow 32 and 64.
    apart: as many of them as can be in different eights of neighbours, else side by side and anywhere."""
    E = 896
    n = k + 2 + more
    place = torch.arange(n, device=DEV)
    place = (place % 112 * 8 + place // 112).sort().values if apart else torch.randperm(E, generator=ops.gen(k), device=DEV)[:n].sort().values
    x = torch.full((2, E), base - 40, device=DEV)
    bias = torch.full((E,), large - 50.0, device=DEV)
    first, pair, best = place[:k - 1], place[k - 1:-1], place[-1:]
    x[:, first], bias[first] = 1.0, large + 2 + torch.arange(k - 1, device=DEV) * 0.5
    x[:, pair], bias[pair] = base, large
    x[:, best], bias[best] = base + 0.125, large
    x[1] = x[0].roll(7)
    for shift in (0, 7):
        idx, _ = ops.check_selection(x[shift // 7:shift // 7 + 1], k, bias=bias.roll(shift))
        if large == 0.0:
            assert (idx == (int(best) + shift) % E).any()


@pytest.mark.parametrize("steps", [False, True])
@pytest.mark.parametrize("k", [1, 2, 4, 16, 32])
@pytest.mark.parametrize("E", [32, 61, 128, 896])
def test_logits_in_steps(E, k, steps):
    """16-bit logits, most of them saturated on one side, and a bias of zeros or steps, as before and early in a training."""
    T = 20_000 if E < 896 else 4_000
    g = ops.gen(E + k)
    x = torch.randn(T, E, generator=g, device=DEV) * 6
    x[: T // 2] += 18
    x[T // 2:] -= 30
    bias = torch.zeros(E, device=DEV)
    if steps:
        bias = torch.randint(-2, 3, (E,), generator=g, device=DEV) * 2.0 ** -20
    for dtype in (BF16, F16):
        ops.check_selection((x * 4).round().div(4).to(dtype), k, bias=bias)


# ------------------------------------------------------------------ gradients that nothing may be made of
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [61, 64, 896])
@pytest.mark.parametrize("score,normalize", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_gate_gradients_of_closed_experts_are_not_read(score, normalize, E, dtype):
    """A slot that is dropped, or whose expert the logits close, has no gradient whatever stands in d_gates: a value there
    that is no number changes nothing, in its token's other slots neither."""
    T, k = 40, 6
    x = ops.data(T, E, dtype, 31)
    idx, _ = moe.select_experts(x, k, score=score)
    rows = torch.arange(T, device=DEV)
    for j, closed in ((1, -INF), (4, NAN)):
        x[rows[::2], idx[::2, j].long()] = closed            # behind the selection: its slot stays
    idx[::3, 0], idx[1::3, 2] = -1, E + 1
    l = ops.opened(x).gather(1, idx.long().clamp(0, E - 1))
    off = (idx < 0) | (idx >= E) | (l == -INF)
    dg = torch.randn(T, k, generator=ops.gen(32), device=DEV)
    want = moe.router_backward(x, idx, d_gates=torch.where(off, 0.0, dg), score=score, normalize=normalize, scale=2.5)
    assert want.isfinite().all() and off.any(1).sum() > T / 2
    for junk in (NAN, INF, -INF):
        got = moe.router_backward(x, idx, d_gates=torch.where(off, junk, dg), score=score, normalize=normalize, scale=2.5)
        assert torch.equal(got, want)
