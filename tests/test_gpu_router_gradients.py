"""The router's gradients against automatic differentiation of the definitions.

Gates and losses are written down in 64 bits, from torch's own sigmoid and
softmax, and differentiated by autograd: nothing here shares a derivation with
the kernels.  The gates' gradient and the losses' are compared apart, within the
tolerance that test_gpu_router_ops.py derives (160 u of the magnitudes that a
sum adds, u = 2^-24, and half a step of the output's type), and each case shows
that a gradient which is missing, or off by a hundredth, would not pass."""
import pytest
import torch

import test_gpu_router_ops as ops
import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
FORMS = [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)]


def gates(l, idx, score, normalize, scale):
    kept = (idx >= 0) & (idx < l.shape[1])
    picked = l.gather(1, torch.where(kept, idx, 0).long())
    if score == "sigmoid":
        w = torch.sigmoid(picked) * kept
        if normalize:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    elif normalize:
        some = kept.any(1, keepdim=True)
        w = torch.softmax(picked.masked_fill(~kept & some, float("-inf")), 1) * kept
    else:
        w = torch.softmax(l, 1).gather(1, torch.where(kept, idx, 0).long()) * kept
    return scale * w


def losses(l, idx, cuts, score):
    E, k = l.shape[1], idx.shape[1]
    p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l) / torch.sigmoid(l).sum(1, keepdim=True)
    kept = (idx >= 0) & (idx < E)
    out = []
    for a, b in zip(cuts[:-1], cuts[1:]):
        used = kept[a:b].any(1)
        n = int(used.sum())
        counts = torch.zeros(E, dtype=torch.float64, device=DEV)
        counts.index_add_(0, idx[a:b][kept[a:b]].long(), torch.ones(int(kept[a:b].sum()), dtype=torch.float64, device=DEV))
        out.append(E / (k * n) * (counts * p[a:b][used].sum(0) / n).sum() if n else (l * 0).sum())
    return torch.stack(out)


def differentiated(logits, f):
    l = logits.double().requires_grad_()
    return torch.autograd.grad(f(l), l)[0]


def near(got, want, size, dtype):
    """Within the tolerance, which a hundredth of the gradient is outside of in nearly every row that has one (not where
    two slots happen to have the same entry, which cancel)."""
    fin = torch.finfo(dtype)
    step = want.abs() * fin.eps / 2 + fin.smallest_normal * fin.eps if dtype != torch.float32 else want.abs() * U + 1e-37
    limit = 160 * U * size + step
    assert ((got.double() - want).abs() <= limit).all()
    rows = (want.abs() > 1e-9 * size).any(1)
    assert rows.any() and (want.abs() > 100 * limit).any(1)[rows].double().mean() > 0.9


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,cuts", [(40, 96, 4, (0, 11, 11, 38)), (700, 896, 16, (0, 100, 101, 640)), (333, 61, 6, (5, 40, 300)), (65, 513, 32, (0, 65))])
@pytest.mark.parametrize("score,normalize", FORMS)
def test_gradients(score, normalize, T, E, k, cuts, dtype):
    x = ops.data(T, E, dtype, T + 7)
    idx = ops.routed(x, k, T)
    dg = torch.randn(T, k, generator=ops.gen(T + 8), device=DEV)
    S = len(cuts) - 1
    dl = (0.5 + torch.rand(S, generator=ops.gen(T + 9), device=DEV)) * T
    seq = ops.offsets(*cuts)

    got = moe.router_backward(x, idx, d_gates=dg, score=score, normalize=normalize, scale=2.5)
    want = differentiated(x, lambda l: (gates(l, idx, score, normalize, 2.5) * dg.double()).sum())
    _, size = ops.gradient(x, idx, score, normalize, 2.5, None, dg, None)
    near(got, want, size, dtype)

    loss, counts, tokens = moe.balance_loss(x, idx, score=score, sequences=seq)
    value = losses(x.double(), idx, cuts, score)
    assert ((loss.double() - value).abs() <= 160 * U * value).all()
    got = moe.router_backward(x, idx, d_loss=dl, counts=counts, tokens=tokens, sequences=seq, score=score)
    want = differentiated(x, lambda l: (losses(l, idx, cuts, score) * dl.double()).sum())
    _, size = ops.gradient(x, idx, score, normalize, 1.0, seq, None, dl)
    near(got, want, size, dtype)


@pytest.mark.parametrize("score,normalize", FORMS)
def test_differences(score, normalize):
    """(f(x + h v) - f(x - h v)) / 2h in 64 bits, off by h^2 = 1e-10 of the third derivatives and 2^-53 / h of f, against the
    kernel's gradient along v, which has the gradient's signs so that nothing cancels."""
    T, E, k, h = 48, 96, 4, 1e-5
    cuts = (0, 11, 11, 38)
    x = ops.data(T, E, torch.float32, 51)
    idx = ops.routed(x, k, 52)
    dg, dl = torch.randn(T, k, generator=ops.gen(53), device=DEV), 1 + torch.rand(3, generator=ops.gen(54), device=DEV)
    _, counts, tokens = moe.balance_loss(x, idx, score=score, sequences=ops.offsets(*cuts))
    z = x.double()
    for f, d, size in (
            (lambda l: (gates(l, idx, score, normalize, 1.0) * dg.double()).sum(),
             moe.router_backward(x, idx, d_gates=dg, score=score, normalize=normalize),
             ops.gradient(x, idx, score, normalize, 1.0, None, dg, None)[1]),
            (lambda l: (losses(l, idx, cuts, score) * dl.double()).sum(),
             moe.router_backward(x, idx, d_loss=dl, counts=counts, tokens=tokens, sequences=ops.offsets(*cuts), score=score),
             ops.gradient(x, idx, score, normalize, 1.0, ops.offsets(*cuts), None, dl)[1])):
        v = (0.5 + torch.rand(T, E, generator=ops.gen(55), device=DEV, dtype=torch.float64)) * differentiated(x, f).sign()
        slope = float((f(z + h * v) - f(z - h * v)) / (2 * h))
        along = float((d.double() * v).sum())
        limit = float((size * v.abs()).sum()) * (161 * U + 1e-8) + abs(float(f(z))) * 2.0 ** -50 / h
        assert abs(slope - along) <= limit and abs(slope) > 20 * limit


# ------------------------------------------------------------------ losses that take more than one block
# (rows beyond those that a cluster for each sequence takes in one launch)
LARGE = [(2000, 513, 2, (0, 1, 700, 700, 1999)), (1500, 1023, 8, None), (152 * 4 + 1, 1024, 32, None), (152 * 11, 896, 16, (0, 152, 153, 1672)),
         (1300, 96, 5, tuple(sorted(list(range(0, 1301, 26)) + [26, 26, 650, 1300, 1300]))), (1200, 61, 6, tuple(range(1201))), (777, 500, 4, (3, 775))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,cuts", LARGE)
def test_losses_of_many_rows(T, E, k, cuts, score, dtype):
    x = ops.data(T, E, dtype, T)
    idx = ops.routed(x, k, T)
    seq = None if cuts is None else ops.offsets(*cuts)
    ops.check_loss(x, idx, score, seq)
    S = 1 if cuts is None else len(cuts) - 1
    ops.check_gradient(x, idx, score, True, 1.0, seq, None, torch.ones(S, device=DEV) * T)


@pytest.mark.parametrize("T,E,k,cuts", LARGE)
def test_nothing_beside_the_workspace_is_written(T, E, k, cuts):
    """Guards round a workspace of exactly the bytes asked for, and round the outputs."""
    x = ops.data(T, E, torch.float32, 3)
    idx = ops.routed(x, k, 4)
    cuts = (0, T) if cuts is None else cuts
    seq, S = ops.offsets(*cuts), len(cuts) - 1
    L = moe.lib()
    size = L.moe_balance_loss_workspace_bytes(T, E, S)
    assert size % 4 == 0

    def guarded(n, dtype):
        t = torch.full((n + 64,), 77, dtype=dtype, device=DEV)
        return t, t[32:32 + n]
    (loss_g, loss), (counts_g, counts), (tokens_g, tokens) = guarded(S, torch.float32), guarded(S * E, torch.int32), guarded(S, torch.int32)
    work_g, work = guarded(size // 4, torch.float32)
    a = moe.router._BalanceLossArgs(x.data_ptr(), E, idx.data_ptr(), seq.data_ptr(), loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(), work.data_ptr(), size,
                                    T, E, k, S, 0, 0)
    assert L.moe_balance_loss(a, torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
    for t in (loss_g, counts_g, tokens_g, work_g):
        assert (t[:32] == 77).all() and (t[-32:] == 77).all()
    assert (work != 77).any()                               # it is this path that writes parts
    want = moe.balance_loss(x, idx, sequences=seq)
    assert torch.equal(loss, want[0]) and torch.equal(counts.view(S, E), want[1]) and torch.equal(tokens, want[2])
