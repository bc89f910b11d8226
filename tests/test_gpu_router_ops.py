"""Selection, balance loss and their gradient against their formulas in 64 bits.

Tolerances, in units u = 2^-24 (half a step of fp32).  A share p = x / sum x:
the argument of an exponential is off by u |l - top|, which e^-d d <= 0.37 turns
into an absolute 0.4 u; the exponential by 2 steps (4 u), a sum of positive
values by one u an addition in its longest chain (32 in a lane, 5 over the
lanes), quotients and products by one u each: at most 50 u relative, 64 taken.
Gates have 32 values at most and no chain in a lane: 24 u.  Gradients are p (a -
inner): each factor 64 u of its terms' magnitudes and a sum of 37 additions, 160
u of the magnitudes taken.  A loss adds to its shares' error the tokens of a
warp, 16 warps, a quarter of 152 parts and the experts: 160 u.  Outputs in 16
bits are off by half a step more."""
import math

import pytest
import torch

import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
INF, NAN = math.inf, math.nan


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def opened(logits):
    l = logits.double()
    return torch.where(l.isnan(), -INF, l.clamp(max=torch.finfo(torch.float32).max))


def selection(logits, k, bias=None, mask=None):
    """Experts by (key descending, number ascending), -1 where none is open."""
    key = opened(logits)
    if bias is not None:
        key = torch.where(key > -INF, 1 / (1 + torch.exp(-key)) + opened(bias), key)
    if mask is not None:
        key = torch.where(mask[:, None], key, -INF)
    key, order = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(key[:, :k] > -INF, order[:, :k], -1)


def shares(l, score):
    """Shares of the score; every magnitude is kept in range by taking the largest out."""
    top = l.amax(1, keepdim=True)
    top = torch.where(top > -INF, top, 0.0)
    if score == "softmax":
        x = torch.exp(l - top)
    else:
        x = torch.exp(l.clamp(max=0) - top.clamp(max=0)) / (1 + torch.exp(-l.abs()))
    s = x.sum(1, keepdim=True)
    return torch.where(s > 0, x / s.clamp(min=1e-300), 0.0)


def gates_of(l, idx, score, normalize, scale):
    held = torch.where(idx >= 0, l.gather(1, idx.clamp(min=0)), -INF)
    if normalize:
        w = shares(held, score)
    else:
        w = 1 / (1 + torch.exp(-held)) if score == "sigmoid" else shares(l, score).gather(1, idx.clamp(min=0))
    return scale * torch.where(idx >= 0, w, 0.0)


def data(T, E, dtype, seed=0, spread=1.5):
    g = gen(seed)
    return (torch.randn(T, E, generator=g, device=DEV) * spread + torch.randn(E, generator=g, device=DEV) * 0.5).to(dtype)


def check_selection(logits, k, **kw):
    bias, mask = kw.get("bias"), kw.get("mask")
    score, normalize, scale = kw.get("score", "sigmoid"), kw.get("normalize", True), kw.get("scale", 1.0)
    idx, gates = moe.select_experts(logits, k, **kw)
    want = selection(logits, k, bias, mask)
    assert idx.dtype == torch.int32 and torch.equal(idx.long(), want)
    w = gates_of(opened(logits), want, score, normalize, scale)
    assert gates.dtype == torch.float32 and gates.isfinite().all()
    assert ((gates.double() - w).abs() <= (64 if not normalize else 24) * U * w + abs(scale) * U).all()
    return idx, gates


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", [(1, 896, 16), (300, 896, 16), (7, 1, 1), (65, 61, 6), (33, 32, 32), (64, 64, 17), (129, 1024, 32), (40, 1000, 1),
                                   (19, 1023, 31), (50, 256, 8), (50, 257, 8), (50, 512, 20), (50, 520, 16)])
def test_selection(T, E, k, dtype):
    x = data(T, E, dtype, T + E)
    bias = torch.randn(E, generator=gen(E), device=DEV) * 0.1
    mask = torch.rand(T, generator=gen(T), device=DEV) < 0.8
    check_selection(x, k, bias=bias)
    check_selection(x, k, bias=bias, mask=mask, normalize=False, scale=2.5)
    check_selection(x, k, score="softmax", mask=mask)
    check_selection(x, k, score="softmax", normalize=False, scale=0.5)
    check_selection(x, k)


@pytest.mark.parametrize("E,k", [(896, 16), (61, 6), (1024, 32)])
@pytest.mark.parametrize("kind", ["equal", "two values", "steps", "halves"])
def test_ties(E, k, kind):
    """Equal keys go to the lowest expert; so many of them that candidates do not fit their table."""
    e = torch.arange(E, device=DEV)
    row = {"equal": torch.zeros(E, device=DEV), "two values": (e % 3 == 1).float(), "steps": -(e // 5).float() / 8, "halves": (e >= E // 2).float()}[kind]
    x = torch.stack([row, row.flip(0), -row])
    check_selection(x, k)
    check_selection(x, k, score="softmax")
    check_selection(x, k, bias=torch.zeros(E, device=DEV))
    check_selection(x, k, bias=-row * 0.25)
    check_selection(x.bfloat16(), k, bias=row.flip(0) * 1e-9)


@pytest.mark.parametrize("spread", [0.0, 1e-9, 1e-7, 1e-5])
def test_keys_nearer_than_32_bits_tell(spread):
    """Keys sigmoid(l) + b made nearly equal by the bias: their order needs 64 bits."""
    E, k = 896, 16
    g = gen(3)
    x = torch.randn(64, E, generator=g, device=DEV)
    x[:, 100:160] = torch.linspace(3, 9, 60, device=DEV)
    bias = torch.full((E,), -5.0, device=DEV)
    bias[100:160] = ((1 - torch.sigmoid(x[0, 100:160].double())) + spread * torch.randn(60, generator=g, device=DEV).double()).float()
    check_selection(x, k, bias=bias)
    # saturated scores: 1 - sigmoid(l) is below half a step of fp32 from l = 18 on
    x[:, 200:260] = torch.linspace(17, 36, 60, device=DEV)
    check_selection(x, k, bias=torch.zeros(E, device=DEV))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,k", [(896, 16), (61, 6)])
def test_values_that_are_no_numbers(E, k, dtype):
    x = data(12, E, dtype, 5)
    low = torch.finfo(dtype).min
    x[0] = -INF
    x[1] = NAN
    x[2, 3:] = -INF                     # fewer open experts than slots
    x[3, ::2] = NAN
    x[4, 5], x[4, 9], x[4, 11] = INF, INF, -INF
    x[5] = low
    x[6, 2:] = low                      # masks of the type's lowest value
    x[7] = INF
    x[8] = -200 if dtype != torch.float16 else -2000
    x[8, 4] += 4
    bias = torch.randn(E, generator=gen(1), device=DEV)
    bias[1], bias[7], bias[8], bias[9] = -INF, NAN, INF, -1e30
    for kw in (dict(), dict(score="softmax"), dict(bias=bias), dict(bias=bias, normalize=False), dict(score="softmax", normalize=False)):
        idx, gates = check_selection(x, k, **kw)
        assert (idx[:2] == -1).all() and (gates[:2] == 0).all()
        if kw.get("normalize", True):
            held = (idx >= 0).any(1)
            assert ((gates.double().sum(1) - 1).abs()[held] <= 64 * U).all()


def test_no_tokens_and_masks_of_everything():
    idx, gates = moe.select_experts(torch.zeros(0, 8, device=DEV), 2)
    assert idx.shape == (0, 2) and gates.shape == (0, 2)
    idx, gates = moe.select_experts(torch.zeros(5, 8, device=DEV), 2, mask=torch.zeros(5, dtype=torch.bool, device=DEV))
    assert (idx == -1).all() and (gates == 0).all()


# ------------------------------------------------------------------ balance loss
def sequence_rows(seq, T):
    cuts = [0, T] if seq is None else [min(max(c, 0), T) for c in seq.tolist()]
    return list(zip(cuts[:-1], cuts[1:]))


def losses_of(l, idx, seq, score):
    """(losses, counts, tokens) with l in 64 bits."""
    E, k = l.shape[1], idx.shape[1]
    p = shares(l, score)
    kept = (idx >= 0) & (idx < E)
    out = []
    for a, b in sequence_rows(seq, l.shape[0]):
        used = kept[a:b].any(1) if b > a else torch.zeros(0, dtype=torch.bool, device=DEV)
        n = int(used.sum())
        c = torch.bincount(idx[a:b][kept[a:b]].long(), minlength=E) if b > a else torch.zeros(E, dtype=torch.long, device=DEV)
        loss = E / (k * n) * (c.double() * p[a:b][used].mean(0)).sum() if n else torch.zeros((), dtype=torch.float64, device=DEV)
        out.append((loss, c, n))
    return torch.stack([o[0] for o in out]), torch.stack([o[1] for o in out]), torch.tensor([o[2] for o in out], device=DEV)


def offsets(*cuts):
    return torch.tensor(cuts, dtype=torch.int32, device=DEV)


def check_loss(logits, idx, score, seq):
    loss, counts, tokens = moe.balance_loss(logits, idx, score=score, sequences=seq)
    want, c, n = losses_of(opened(logits), idx, seq, score)
    assert torch.equal(counts.long(), c) and torch.equal(tokens.long(), n)
    assert ((loss.double() - want).abs() <= 160 * U * want).all()
    return counts, tokens


LAYOUTS = [(64, 32, 4, None), (1, 8, 2, None), (700, 896, 16, (0, 100, 100, 101, 640)), (333, 61, 6, (5, 40, 300)), (2000, 131, 3, tuple(range(0, 2001, 40))),
           (152 * 3 + 1, 1024, 32, (0, 457)), (90, 1000, 8, (0, 0, 90, 90)), (5, 16, 4, (2, 2)), (300, 513, 2, (0, 1, 2, 3, 299)), (40, 3, 3, tuple(range(41)))]


def routed(logits, k, seed):
    """A selection with some slots dropped, some tokens without any, numbers behind the last expert and one named twice."""
    T, E = logits.shape
    idx = moe.select_experts(logits, k, score="softmax")[0]
    r = torch.rand(T, k, generator=gen(seed), device=DEV)
    idx = torch.where(r < 0.1, -1, torch.where(r > 0.97, E + 3, idx))
    idx[torch.rand(T, generator=gen(seed + 1), device=DEV) < 0.1] = -1
    if k > 1:
        idx[::7, 1] = idx[::7, 0]
    return idx.contiguous()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,cuts", LAYOUTS)
def test_balance_loss(T, E, k, cuts, score, dtype):
    x = data(T, E, dtype, T)
    check_loss(x, routed(x, k, T), score, None if cuts is None else offsets(*cuts))


def gradient(logits, idx, score, normalize, scale, seq, d_gates, d_loss):
    """(d_logits, bound of its error before it is rounded) from the formulas, in 64 bits."""
    l, E, k = opened(logits), logits.shape[1], idx.shape[1]
    idx = torch.where((idx >= 0) & (idx < E), idx, -1).long()
    sig = 1 / (1 + torch.exp(-l))
    rest = 1 / (1 + torch.exp(l)) if score == "sigmoid" else torch.ones_like(l)
    p = shares(l, score)
    d, size = torch.zeros_like(l), torch.zeros_like(l)
    if d_loss is not None:
        _, c, n = losses_of(l, idx, seq, score)
        a = torch.zeros_like(l)
        for s, (lo, hi) in enumerate(sequence_rows(seq, l.shape[0])):
            if hi > lo and n[s]:
                a[lo:hi] = d_loss[s].double() * E / k * c[s].double() / n[s].double() ** 2
        a = a * (idx >= 0).any(1, keepdim=True)
        d += p * rest * (a - (p * a).sum(1, keepdim=True))
        size += p * rest * (a.abs() + (p * a.abs()).sum(1, keepdim=True))
    if d_gates is not None:
        at = idx.clamp(min=0)
        open_ = (idx >= 0) & (l.gather(1, at) > -INF)
        held = torch.where(open_, l.gather(1, at), -INF)
        g = torch.where(open_, scale * d_gates.double(), 0.0)
        r = rest.gather(1, at)
        if normalize:
            w = shares(held, score)
            v, m = w * r * (g - (w * g).sum(1, keepdim=True)), w * r * (g.abs() + (w * g.abs()).sum(1, keepdim=True))
        elif score == "sigmoid":
            v = g * sig.gather(1, at) * r
            m = v.abs()
        else:
            w = torch.where(open_, p.gather(1, at), 0.0)
            v = m = w * g
            m = m.abs()
            d -= p * v.sum(1, keepdim=True)
            size += p * m.sum(1, keepdim=True)
        v, m = torch.where(open_, v, 0.0), torch.where(open_, m, 0.0)
        d.scatter_add_(1, at, v)
        size.scatter_add_(1, at, m)
    return d, size


def check_gradient(logits, idx, score, normalize, scale, seq, d_gates, d_loss):
    kw = {}
    if d_loss is not None:
        _, counts, tokens = moe.balance_loss(logits, idx, score=score, sequences=seq)
        kw = dict(d_loss=d_loss, counts=counts, tokens=tokens, sequences=seq)
    got = moe.router_backward(logits, idx, d_gates=d_gates, score=score, normalize=normalize, scale=scale, **kw)
    want, size = gradient(logits, idx, score, normalize, scale, seq, d_gates, d_loss)
    fin = torch.finfo(logits.dtype)
    assert got.dtype == logits.dtype and got.shape == logits.shape and got.isfinite().all()
    step = want.abs() * fin.eps / 2 + fin.smallest_normal * fin.eps if logits.dtype != torch.float32 else want.abs() * U
    assert ((got.double() - want).abs() <= 160 * U * size + step + 1e-37).all()
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score,normalize", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("T,E,k,cuts", LAYOUTS)
def test_gradients(T, E, k, cuts, score, normalize, dtype):
    x = data(T, E, dtype, T + 1)
    idx = routed(x, k, T)
    seq = None if cuts is None else offsets(*cuts)
    S = 1 if cuts is None else len(cuts) - 1
    dg = torch.randn(T, k, generator=gen(T + 2), device=DEV)
    dl = torch.randn(S, generator=gen(T + 3), device=DEV) * T
    both = check_gradient(x, idx, score, normalize, 2.5, seq, dg, dl)
    check_gradient(x, idx, score, normalize, 2.5, None, dg, None)
    check_gradient(x, idx, score, normalize, 2.5, seq, None, dl)
    assert (both[~((idx >= 0) & (idx < E)).any(1)] == 0).all()


@pytest.mark.parametrize("score,normalize", [("sigmoid", True), ("softmax", True), ("sigmoid", False), ("softmax", False)])
def test_gradients_of_closed_experts(score, normalize):
    """Closed and infinite logits: no NaN, nothing at closed experts, rows without any open expert are zero."""
    x = data(9, 61, torch.float32, 8)
    x[0] = -INF
    x[1, 4:] = -INF
    x[2, ::2] = NAN
    x[3, 5] = INF
    x[4] = torch.finfo(torch.float32).min
    x[5] = -300.0
    x[6, 10] = -INF
    idx = moe.select_experts(x, 6, score=score)[0]
    idx[6, 2] = 10                       # a slot of a closed expert
    dg, dl = torch.randn(9, 6, generator=gen(1), device=DEV), torch.ones(1, device=DEV)
    got = check_gradient(x, idx, score, normalize, 1.0, None, dg, dl)
    assert (got[opened(x) == -INF] == 0).all()


@pytest.mark.parametrize("score,normalize", [("sigmoid", True), ("softmax", True), ("sigmoid", False), ("softmax", False)])
def test_gradients_against_differences(score, normalize):
    """(f(x + h v) - f(x - h v)) / 2h, f the gates and the loss weighted at random.  The gates are off by 24 u and the
    losses by 160 u of their sizes, which 1 / 2h turns into 160 u (sum |weights|) / h; the third derivatives of f along
    v add at most h^2 times the same sum times |v|^3 < 30 (the selection does not change: idx is held)."""
    T, E, k, h = 40, 96, 4, 2.0 ** -7
    x = data(T, E, torch.float32, 21)
    idx, _ = moe.select_experts(x, k, score=score)
    v = torch.randn(T, E, generator=gen(22), device=DEV)
    dg, dl = torch.randn(T, k, generator=gen(23), device=DEV), torch.randn(3, generator=gen(24), device=DEV)
    seq = offsets(0, 11, 11, 38)

    def f(z):
        loss, _, _ = moe.balance_loss(z, idx, score=score, sequences=seq)
        # the gates of the experts held: ranked by themselves, each token's slots meet idx by number
        i, w = moe.select_experts(torch.where(torch.zeros_like(z).scatter_(1, idx.long(), 1) > 0, z, -INF) if normalize else z, k if normalize else 32, score=score,
                                  normalize=normalize)
        dense = torch.zeros(T, E + 1, device=DEV, dtype=torch.float64).scatter_(1, torch.where(i < 0, E, i).long(), w.double())
        return (dense.gather(1, idx.long()) * dg.double()).sum() + (loss.double() * dl.double()).sum()

    _, counts, tokens = moe.balance_loss(x, idx, score=score, sequences=seq)
    d = moe.router_backward(x, idx, d_gates=dg, d_loss=dl, counts=counts, tokens=tokens, sequences=seq, score=score, normalize=normalize)
    slope = (f(x + h * v) - f(x - h * v)) / (2 * h)
    size = float(dg.abs().sum() + dl.abs().sum())
    assert abs(float(slope - (d.double() * v.double()).sum())) <= size * (160 * U / h + 30 * h * h)


# ------------------------------------------------------------------ how they lie
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,pad,shift", [(896, 8, 0), (896, 8, 1), (896, 5, 0), (64, 64, 8), (61, 3, 2)])
def test_strided_and_shifted_rows(E, pad, shift, dtype):
    """Rows that go by 16 bytes with space between them, and rows off 16 bytes or of odd stride, element by element."""
    T, k = 37, 6
    store = torch.full((T, E + pad + shift), NAN, device=DEV, dtype=dtype)
    x = store[:, shift:shift + E]
    x.copy_(data(T, E, dtype, 3))
    bias = torch.randn(E, generator=gen(4), device=DEV) * 0.1
    idx, gates = check_selection(x, k, bias=bias)
    check_loss(x, idx, "sigmoid", offsets(0, 20, 37))
    check_gradient(x, idx, "sigmoid", True, 1.0, offsets(0, 20, 37), gates, torch.ones(2, device=DEV))
    check_selection(x.t().contiguous().t(), k, bias=bias)       # columns apart: copied


def test_gradient_in_place():
    """d_logits may be the logits themselves."""
    T, E, k = 50, 200, 5
    for dtype, code in ((torch.float32, 0), (torch.bfloat16, 1)):
        x = data(T, E, dtype, 9)
        idx, gates = moe.select_experts(x, k)
        _, counts, tokens = moe.balance_loss(x, idx)
        dl = torch.ones(1, device=DEV)
        want = moe.router_backward(x, idx, d_gates=gates, d_loss=dl, counts=counts, tokens=tokens)
        p = [t.data_ptr() for t in (idx, gates, dl, counts, tokens)]
        a = moe.router._RouterBackwardArgs(x.data_ptr(), E, p[0], p[1], p[2], p[3], p[4], None, x.data_ptr(), E, T, E, k, 1, code, 0, 1, 1.0)
        assert moe.lib().moe_router_backward(a, torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
        assert torch.equal(x, want)


def test_nothing_beside_the_outputs_is_written():
    """Rows in a wider matrix, and guards round every output."""
    T, E, k, S = 23, 96, 5, 2
    x = data(T, E, torch.float32, 2)
    L, s = moe.lib(), torch.cuda.current_stream().cuda_stream
    seq = offsets(0, 9, 20)

    def guarded(n, dtype):
        t = torch.full((n + 32,), 77, dtype=dtype, device=DEV)
        return t, t[16:16 + n]

    idx_g, idx = guarded(T * k, torch.int32)
    gates_g, gates = guarded(T * k, torch.float32)
    a = moe.router._SelectArgs(x.data_ptr(), E, None, None, idx.data_ptr(), gates.data_ptr(), T, E, k, 0, 0, 1, 1.0)
    assert L.moe_select(a, s) == moe.MOE_OK
    size = L.moe_balance_loss_workspace_bytes(T, E, S)
    loss_g, loss = guarded(S, torch.float32)
    counts_g, counts = guarded(S * E, torch.int32)
    tokens_g, tokens = guarded(S, torch.int32)
    work_g, work = guarded(size // 4, torch.float32)
    b = moe.router._BalanceLossArgs(x.data_ptr(), E, idx.data_ptr(), seq.data_ptr(), loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(), work.data_ptr(), size,
                                    T, E, k, S, 0, 0)
    assert L.moe_balance_loss(b, s) == moe.MOE_OK
    d = torch.full((T, E + 8), 77.0, device=DEV)
    dl = torch.ones(S, device=DEV)
    c = moe.router._RouterBackwardArgs(x.data_ptr(), E, idx.data_ptr(), gates.data_ptr(), dl.data_ptr(), counts.data_ptr(), tokens.data_ptr(), seq.data_ptr(),
                                       d.data_ptr(), E + 8, T, E, k, S, 0, 0, 1, 1.0)
    assert L.moe_router_backward(c, s) == moe.MOE_OK
    for t in (idx_g, gates_g, loss_g, counts_g, tokens_g, work_g):
        assert (t[:16] == 77).all() and (t[-16:] == 77).all()
    assert (d[:, E:] == 77).all()
    i2, g2 = moe.select_experts(x, k)
    assert torch.equal(idx.view(T, k), i2) and torch.equal(gates.view(T, k), g2)
    assert (d[20:, :E] != 0).any() and torch.equal(d[:, :E], moe.router_backward(x, i2, d_gates=g2, d_loss=dl, counts=counts.view(S, E), tokens=tokens, sequences=seq))


def test_results_do_not_change_from_call_to_call():
    x = data(3000, 896, torch.bfloat16, 12)
    seq = offsets(0, 700, 2999)
    dl = torch.ones(2, device=DEV)

    def run():
        idx, gates = moe.select_experts(x, 16)
        loss, counts, tokens = moe.balance_loss(x, idx, sequences=seq)
        return idx, gates, loss, counts, tokens, moe.router_backward(x, idx, d_gates=gates, d_loss=dl, counts=counts, tokens=tokens, sequences=seq)

    first = run()
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(first, run()))
