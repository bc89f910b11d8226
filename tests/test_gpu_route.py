"""Tokens sorted by expert and back (moe_sort, moe_permute, moe_unpermute and
its gradients) against plain index arithmetic and sums in 64 bits.

Tolerances: a copy is exact.  A weighted sum of k terms in fp32 with FMAs is
off by at most k 2^-24 of the sum of the terms' magnitudes, and its store by
half a step of the output type; a dot product of D terms, summed by 32 lanes
and a butterfly, by at most (D/32 + 6) 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def plain_sort(idx, E):
    flat = idx.reshape(-1).tolist()
    kept = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < E)
    offsets = [sum(1 for e, _ in kept if e < x) for x in range(E + 1)] if len(kept) < 4000 else \
        np.searchsorted(np.array([e for e, _ in kept]), np.arange(E + 1)).tolist()
    sorted_slot = [i for _, i in kept] + [-1] * (len(flat) - len(kept))
    slot_pos = [-1] * len(flat)
    for p, (_, i) in enumerate(kept):
        slot_pos[i] = p
    return offsets, sorted_slot, slot_pos


def route(T, k, E, drop=0.0, seed=0, repeat=False):
    g = torch.Generator().manual_seed(seed)
    if repeat:
        idx = torch.randint(0, E, (T, k), generator=g)
    else:
        idx = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    idx = torch.where(torch.rand(T, k, generator=g) < drop, torch.full_like(idx, -1), idx)
    return idx.to(torch.int32).contiguous()


@pytest.mark.parametrize("T,k,E,drop,repeat", [
    (0, 4, 8, 0, False), (1, 1, 1, 0, False), (1, 16, 896, 0, False), (3, 5, 7, 0.3, True), (64, 16, 896, 0, False),
    (65, 32, 33, 0.1, False), (513, 16, 16, 0, True), (1000, 3, 1024, 0.9, True), (700, 12, 61, 0, True),
    (8192, 16, 896, 0.01, True), (5000, 8, 2, 0, True), (300, 4, 8, 1.1, False), (20000, 7, 100, 0.2, True)])
def test_sort(T, k, E, drop, repeat):
    idx = route(T, k, E, drop, repeat=repeat)
    offsets, sorted_slot, slot_pos = moe.sort_by_expert(idx.to(DEV), E)
    ref = plain_sort(idx, E)
    assert offsets.tolist() == ref[0]
    assert sorted_slot.tolist() == ref[1]
    assert slot_pos.reshape(-1).tolist() == ref[2]


def test_sort_ignores_entries_out_of_range():
    idx = torch.tensor([[0, 5], [2 ** 31 - 1, -2 ** 31], [4, 4]], dtype=torch.int32)
    offsets, sorted_slot, slot_pos = moe.sort_by_expert(idx.to(DEV), 5)
    assert offsets.tolist() == [0, 1, 1, 1, 1, 3]
    assert sorted_slot.tolist() == [0, 4, 5, -1, -1, -1]
    assert slot_pos.tolist() == [[0, -1], [-1, -1], [1, 2]]


@pytest.mark.parametrize("T,k,D,dtype,drop", [
    (1, 16, 3584, torch.bfloat16, 0), (1, 1, 1, torch.float32, 0), (5, 3, 7, torch.float16, 0.4), (9, 4, 1001, torch.bfloat16, 0.2),
    (64, 16, 1792, torch.uint8, 0), (33, 2, 112, torch.uint8, 0.1), (7, 5, 13, torch.uint8, 0.1), (300, 6, 520, torch.float32, 0.1),
    (17, 32, 66, torch.float16, 0.5)])
def test_permute_copies_rows_and_leaves_the_rest(T, k, D, dtype, drop):
    E = max(k, 11)
    idx = route(T, k, E, drop, seed=1)
    _, sorted_slot, slot_pos = moe.sort_by_expert(idx.to(DEV), E)
    wide = torch.randint(0, 200, (T, D + 3), device=DEV)
    x = wide.to(dtype)[:, :D]                                       # rows with a stride
    rows = torch.full((T * k + 2, D), 77, device=DEV).to(dtype)
    got = moe.permute(x, slot_pos, out=rows)
    assert got is rows
    order = sorted_slot.tolist()
    n = sum(1 for s in order if s >= 0)
    token = torch.tensor([s // k for s in order[:n]], device=DEV, dtype=torch.long)
    assert torch.equal(rows[:n], x[token])
    assert (rows[n:] == 77).all()
    # without an output of the caller's
    assert torch.equal(moe.permute(x, slot_pos)[:n], x[token])


def bad_places(slot_pos, n):
    """Some places outside the rows: they count as dropped."""
    p = slot_pos.clone()
    p.view(-1)[::7] = n
    p.view(-1)[1::11] = 2 ** 31 - 1
    p.view(-1)[2::13] = -5
    return p


@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,k,D,drop", [(1, 1, 8, 0), (1, 16, 3584, 0), (3, 32, 264, 0.3), (65, 6, 1001, 0.2), (40, 8, 96, 1.1),
                                        (257, 9, 33, 0.5)])
def test_unpermute_and_gradients(T, k, D, drop, dtype, out):
    E = max(k, 40)
    idx = route(T, k, E, drop, seed=2)
    _, _, slot_pos = moe.sort_by_expert(idx.to(DEV), E)
    n = T * k
    g = torch.Generator(device=DEV).manual_seed(3)
    rows = torch.randn(n, D, generator=g, device=DEV).to(dtype)
    w = torch.randn(T, k, generator=g, device=DEV)
    dy = torch.randn(T, D, generator=g, device=DEV).to(out)
    for pos in (slot_pos, bad_places(slot_pos, n)):
        held = (pos >= 0) & (pos < n)
        at = torch.where(held, pos, 0).long()
        picked = rows.double()[at] * held.unsqueeze(-1)                  # [T][k][D]
        used = torch.zeros(n, dtype=torch.bool, device=DEV)
        used[at[held]] = True
        # rows that are not read may hold anything
        dirty = torch.where(used.unsqueeze(-1), rows, torch.full_like(rows, float("nan")))
        for weights in (w, None):
            wd = (weights if weights is not None else torch.ones(T, k, device=DEV)).double()
            y = moe.unpermute(dirty, pos, weights, out_dtype=out)
            ref, mag = (wd.unsqueeze(-1) * picked).sum(1), (wd.abs().unsqueeze(-1) * picked.abs()).sum(1)
            tol = mag * (k * 2.0 ** -24) + (ref.abs() + mag * (k * 2.0 ** -24)) * HALF[out] + TINY[out]
            assert y.dtype == out and ((y.double() - ref).abs() <= tol).all()
            keep = torch.full_like(rows, 5.0)
            d_rows, d_w = moe.unpermute_backward(dy, dirty, pos, weights, out=keep)
            ref_rows = torch.full((n, D), 5.0, dtype=torch.float64, device=DEV)
            ref_rows[at[held]] = (wd.unsqueeze(-1) * dy.double().unsqueeze(1))[held]
            tol = ref_rows.abs() * (2.0 ** -24 + HALF[dtype] * (1 + 2.0 ** -24)) + TINY[dtype]
            assert d_rows is keep and ((d_rows.double() - ref_rows).abs() <= tol).all()
            dots = (picked * dy.double().unsqueeze(1))
            tol = dots.abs().sum(-1) * ((D / 32 + 6) * 2.0 ** -24) + 2.0 ** -149
            assert ((d_w.double() - dots.sum(-1)).abs() <= tol).all()
            assert (d_w[~held] == 0).all()
        # one gradient without the other
        only, none = moe.unpermute_backward(dy, dirty, pos, w, need_weights=False)
        assert none is None and torch.equal(only[used], moe.unpermute_backward(dy, dirty, pos, w)[0][used])
        none, only = moe.unpermute_backward(dy, dirty, pos, w, need_rows=False)
        assert none is None and torch.equal(only, moe.unpermute_backward(dy, dirty, pos, w)[1])


def test_gradients_are_those_of_the_formula_by_differences():
    """d_rows and d_w as directional derivatives of unpermute, in fp32 with an exactly linear map."""
    T, k, D, E = 19, 4, 40, 12
    idx = route(T, k, E, 0.2, seed=5)
    _, _, pos = moe.sort_by_expert(idx.to(DEV), E)
    g = torch.Generator(device=DEV).manual_seed(6)
    r = lambda *s: torch.randint(-8, 9, s, generator=g, device=DEV).float()  # noqa: E731  small integers: every sum is exact
    rows, w, dy, v, z = r(T * k, D), r(T, k), r(T, D), r(T * k, D), r(T, k)
    d_rows, d_w = moe.unpermute_backward(dy, rows, pos, w, out=torch.zeros_like(rows))
    base = moe.unpermute(rows, pos, w)
    assert float((d_rows * v).sum()) == float(((moe.unpermute(rows + v, pos, w) - base) * dy).sum())
    assert float((d_w * z).sum()) == float(((moe.unpermute(rows, pos, w + z) - base) * dy).sum())
    x, u = r(T, D), r(T * k, D)
    back = moe.permute_backward(u, pos)
    assert float((back * x).sum()) == float((moe.permute(x, pos, out=torch.zeros_like(u)) * u).sum())


def test_strided_rows_and_expanded_gradients():
    T, k, D, E = 21, 3, 48, 9
    idx = route(T, k, E, 0.0, seed=7)
    _, _, pos = moe.sort_by_expert(idx.to(DEV), E)
    wide = torch.randn(T * k, 2 * D, device=DEV)
    w = torch.rand(T, k, device=DEV)
    for rows in (wide[:, :D], wide[:, 1:D + 1], wide[:, ::2], wide.t()[:D].t()):
        assert torch.equal(moe.unpermute(rows, pos, w), moe.unpermute(rows.contiguous(), pos, w))
    out = torch.full((T, D + 5), 3.0, device=DEV)
    moe.unpermute(wide[:, :D], pos, w, out=out[:, :D])
    assert torch.equal(out[:, :D], moe.unpermute(wide[:, :D].contiguous(), pos, w)) and (out[:, D:] == 3).all()
    one = torch.ones((), device=DEV).expand(T, D)
    a, b = moe.unpermute_backward(one, wide[:, :D], pos, w)
    c, d = moe.unpermute_backward(one.contiguous(), wide[:, :D].contiguous(), pos, w)
    assert torch.equal(a, c) and torch.equal(b, d)


def test_places_past_32_bits():
    """Rows whose byte offsets pass 2^32 (a 5 GB matrix of which few rows are touched)."""
    D, n = 8192, 300_000
    rows = torch.empty(n, D, dtype=torch.bfloat16, device=DEV)
    pos = torch.tensor([[n - 1, 0], [n // 2, n - 2]], dtype=torch.int32, device=DEV)
    x = torch.randn(2, D, device=DEV).bfloat16()
    moe.permute(x, pos, out=rows)
    assert torch.equal(rows[n - 1], x[0]) and torch.equal(rows[0], x[0])
    assert torch.equal(rows[n // 2], x[1]) and torch.equal(rows[n - 2], x[1])
    assert torch.equal(moe.unpermute(rows, pos), (2 * x.float()).bfloat16())


def test_empty_batch():
    idx = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    offsets, sorted_slot, pos = moe.sort_by_expert(idx, 5)
    assert offsets.tolist() == [0] * 6 and sorted_slot.numel() == 0 and pos.shape == (0, 4)
    x = torch.empty(0, 16, device=DEV)
    assert moe.permute(x, pos).shape == (0, 16)
    assert moe.unpermute(x, pos).shape == (0, 16)
    d_rows, d_w = moe.unpermute_backward(x, x, pos)
    assert d_rows.shape == (0, 16) and d_w.shape == (0, 4)


@pytest.mark.parametrize("T,k,E", [(257, 16, 896), (1024, 16, 5), (2049, 16, 1024), (16384, 16, 896), (40001, 15, 64), (70000, 16, 1)])
def test_sort_at_its_launches_borders(T, k, E):
    """Few and many CTAs, short and long strips, against a stable sort."""
    g = torch.Generator(device=DEV).manual_seed(T)
    idx = torch.randint(-1 if T % 2 else 0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    offsets, sorted_slot, slot_pos = moe.sort_by_expert(idx, E)
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    n = int((flat >= 0).sum())
    assert torch.equal(offsets.long(), torch.searchsorted(key.sort().values, torch.arange(E + 1, device=DEV)))
    assert torch.equal(sorted_slot[:n].long(), order[:n]) and (sorted_slot[n:] == -1).all()
    place = torch.full_like(flat, -1)
    place[order[:n]] = torch.arange(n, device=DEV)
    assert torch.equal(slot_pos.reshape(-1).long(), place)
