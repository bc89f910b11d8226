"""The router's operators and the experts' products as they are used together:
a training step and a decoded token, and the circumstances of real programs
(captured graphs, streams, host threads, a layer beside them).

Each step of a chain is compared with arithmetic in 64 bits on that step's own
inputs, within the tolerance that the step's own tests derive."""
import threading

import pytest
import torch

import test_gpu_router_ops as ops
import test_gpu_w4_matvec as mv
import moe_expert_layer_top16_gb300 as moe
from moe_expert_layer_top16_gb300 import router

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def batch(T, E, D, k, S, seed, dtype=F32):
    g = ops.gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    cuts = sorted(torch.randint(0, T + 1, (S - 1,), generator=g, device=DEV).tolist())
    return dict(logits=ops.data(T, E, dtype, seed), x=r(T, D), dy=r(T, D), bias=r(E) * 0.1, mask=torch.rand(T, generator=g, device=DEV) < 0.9,
                sequences=ops.offsets(0, *cuts, T), d_loss=r(S) * 10, k=k, E=E)


def train(s, **kw):
    """Selection, rows to their experts and back (the experts themselves left out), and all gradients."""
    idx, gates = moe.select_experts(s["logits"], s["k"], bias=s["bias"], mask=s["mask"], scale=2.5, **kw)
    first, order, pos = moe.sort_by_expert(idx, s["E"], **kw)
    rows = moe.permute(s["x"], pos, out=torch.zeros(idx.numel(), s["x"].shape[1], device=DEV), **kw)
    y = moe.unpermute(rows, pos, gates, **kw)
    loss, counts, tokens = moe.balance_loss(s["logits"], idx, sequences=s["sequences"], **kw)
    _, d_gates = moe.unpermute_backward(s["dy"], rows, pos, gates, need_rows=False, **kw)
    d = moe.router_backward(s["logits"], idx, d_gates=d_gates, d_loss=s["d_loss"], counts=counts, tokens=tokens,
                            sequences=s["sequences"], scale=2.5, **kw)
    return dict(idx=idx, gates=gates, first=first, y=y, loss=loss, counts=counts, tokens=tokens, d_gates=d_gates, d=d)


def experts(E, D, I, seed, form="mxfp4"):
    return dict(gate=mv.weights((E, I, D), form, seed), up=mv.weights((E, I, D), form, seed + 1), down=mv.weights((E, D, I), form, seed + 2))


def decode(s, w, **kw):
    idx, gates = moe.select_experts(s["logits"], s["k"], bias=s["bias"], **kw)
    h = moe.w4_matvec(s["x"], *w["gate"], up=w["up"], idx=idx, **kw)
    return dict(idx=idx, gates=gates, h=h, y=moe.w4_matvec(h, *w["down"], idx=idx, weights=gates, **kw))


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,D,k,S", [(1, 32, 64, 4, 1), (500, 896, 128, 16, 3), (333, 61, 40, 6, 7)])
def test_training_step(T, E, D, k, S, dtype):
    s = batch(T, E, D, k, S, T + E, dtype)
    r = train(s)
    want = ops.selection(s["logits"], k, s["bias"], s["mask"])
    assert torch.equal(r["idx"].long(), want)
    # the sort counts the slots that the loss counts
    assert torch.equal(r["first"].diff().long(), r["counts"].sum(0))
    assert int(r["tokens"].sum()) == int(s["mask"].sum())
    loss, _, _ = ops.losses_of(ops.opened(s["logits"]), r["idx"], s["sequences"], "sigmoid")
    assert ((r["loss"].double() - loss).abs() <= 160 * U * loss).all()
    d, size = ops.gradient(s["logits"], r["idx"], "sigmoid", True, 2.5, s["sequences"], r["d_gates"], s["d_loss"])
    fin = torch.finfo(dtype)
    step = d.abs() * fin.eps / 2 + fin.smallest_normal * fin.eps
    assert ((r["d"].double() - d).abs() <= 160 * U * size + step).all()


def test_training_step_against_differences():
    """The chain's gradient against the change of its results, slots held to their experts, in 64 bits: the difference's
    own error is of the order h^2 = 1e-10 of the third derivatives, some hundred times the first at most."""
    T, E, D, k, S = 40, 24, 16, 5, 3
    s = batch(T, E, D, k, S, 1)
    r = train(s)
    idx, kept = r["idx"].long().clamp(min=0), r["idx"] >= 0

    def f(z):
        gates = ops.gates_of(z, torch.where(kept, idx, -1), "sigmoid", True, 2.5)
        y = gates.sum(1, keepdim=True) * s["x"].double()          # rows come back unchanged
        loss, _, _ = ops.losses_of(z, r["idx"], s["sequences"], "sigmoid")
        return (y * s["dy"].double()).sum() + (loss * s["d_loss"].double()).sum()
    g = ops.gen(9)
    z = s["logits"].double()
    for _ in range(4):
        v = torch.randn(T, E, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-5
        slope = float((f(z + h * v) - f(z - h * v)) / (2 * h))
        _, size = ops.gradient(s["logits"], r["idx"], "sigmoid", True, 2.5, s["sequences"], r["d_gates"], s["d_loss"])
        # a gate's gradient is a sum of D products in fp32
        sums = (s["x"] * s["dy"]).abs().sum(1, keepdim=True).expand(-1, k)
        _, wide = ops.gradient(s["logits"], r["idx"], "sigmoid", True, 2.5, None, sums, None)
        near = float((size * v.abs()).sum()) * (160 * U + 1e-7) + float((wide * v.abs()).sum()) * 2 * D * U
        assert abs(float((r["d"].double() * v).sum()) - slope) <= near


@pytest.mark.parametrize("form", ["mxfp4", (64, BF16)], ids=str)
@pytest.mark.parametrize("T,E,D,I,k", [(1, 64, 256, 128, 8), (5, 9, 448, 96, 3)])
def test_decoded_tokens(T, E, D, I, k, form):
    if form != "mxfp4":
        D, I = ((v + form[0] - 1) // form[0] * form[0] for v in (D, I))
    s = batch(T, E, D, k, 1, T + k)
    s["x"] = s["x"].to(BF16)
    w = experts(E, D, I, 3, form)
    r = decode(s, w)
    assert torch.equal(r["idx"].long(), ops.selection(s["logits"], k, s["bias"]))
    assert r["h"].dtype == BF16 and r["h"].shape == (T, k, I) and r["y"].shape == (T, D)
    gate, up, down = (mv.values(*w[n]) for n in ("gate", "up", "down"))
    for t in range(T):
        size = torch.zeros(D, dtype=torch.float64, device=DEV)
        y = torch.zeros_like(size)
        for j, e in enumerate(r["idx"][t].tolist()):
            x = s["x"][t:t + 1]
            a, b = (x.double() @ gate[e].T)[0], (x.double() @ up[e].T)[0]
            ea, eb = mv.bound(gate[e], x)[0], mv.bound(up[e], x)[0]
            silu = a * torch.sigmoid(a)
            mv.close(r["h"][t, j], silu * b, 1.1 * ea * b.abs() + (silu.abs() + 1.1 * ea) * eb + 8 * U * (silu * b).abs())
            h, weight = r["h"][t, j:j + 1], float(r["gates"][t, j])
            part = (h.double() @ down[e].T)[0] * weight
            y += part
            size += mv.bound(down[e], h)[0] * abs(weight) * (1 + k * I / 64 / 128) + 64 * U * part.abs()
        mv.close(r["y"][t], y, size)


def test_captured_and_replayed():
    """Two graphs of a training step and a decoded token, each on its own workspaces, replayed one after the other and
    at once; eager calls between them; new inputs in the captured buffers."""
    a, s = batch(3000, 896, 64, 16, 4, 5), batch(2, 40, 256, 6, 1, 6)
    s["x"] = s["x"].to(BF16)
    w = experts(40, 256, 128, 4)
    step = lambda: {**train(a), **{"decode " + n: t for n, t in decode(s, w).items()}}  # noqa: E731
    eager = step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = step()
        graphs.append((g, r, torch.cuda.Stream()))
    for factor in (1.0, -0.5):
        a["logits"].mul_(factor)
        s["logits"].mul_(factor)
        s["x"].mul_(factor)
        eager = step()
        torch.cuda.synchronize()
        for g, _, stream in graphs * 3:
            with torch.cuda.stream(stream):
                g.replay()
        again = step()
        torch.cuda.synchronize()
        assert same(eager, again)
        for _, r, _ in graphs:
            assert same(eager, r)


def test_two_streams_at_once():
    a, b = batch(2000, 896, 64, 16, 5, 7), batch(1500, 131, 64, 6, 40, 8)
    ra, rb = train(a), train(b)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(one):
            qa = train(a)
        with torch.cuda.stream(two):
            qb = train(b)
    torch.cuda.synchronize()
    assert same(ra, qa) and same(rb, qb)


def test_stream_argument():
    """The calls run on the stream they are given, which has work before them; copies and workspaces are that stream's."""
    a, s = batch(2000, 131, 64, 6, 5, 9), batch(3, 40, 256, 6, 1, 10)
    s["x"] = s["x"].to(BF16)
    w = experts(40, 256, 128, 4)
    # strided: copied first
    a["bias"] = torch.stack([a["bias"], a["bias"]], 1)[:, 0]
    w["gate"] = (w["gate"][0].transpose(0, 1).contiguous().transpose(0, 1), w["gate"][1])
    want, token = train(a), decode(s, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                      # about ten milliseconds
        got, next_token = train(a, stream=side), decode(s, w, stream=side)
        junk = [torch.full((n,), -1, dtype=torch.int32, device=DEV) for n in (131, 40 * 128 * 128 // 4, 2000 * 6, 2000 * 131) * 4]
        torch.cuda.synchronize()
        assert same(want, got) and same(token, next_token)
        del junk


def test_first_calls_of_host_threads():
    """A thread's first CUDA call: the product encodes TMA descriptors, for which the thread has no context yet."""
    s = batch(3, 40, 256, 6, 1, 11)
    s["x"] = s["x"].to(BF16)
    w = experts(40, 256, 128, 4)
    idx, _ = moe.select_experts(s["logits"], 6)
    want = moe.w4_matvec(s["x"], *w["gate"], up=w["up"], idx=idx)
    out = torch.empty_like(want)
    calls = [(lambda: moe.w4_matvec(s["x"], *w["gate"], up=w["up"], idx=idx, out=out), want),
             (lambda: moe.select_experts(s["logits"], 6)[0], idx), (lambda: moe.balance_loss(s["logits"], idx)[0], moe.balance_loss(s["logits"], idx)[0])]
    torch.cuda.synchronize()
    for call, ref in calls:
        got = []
        t = threading.Thread(target=lambda: got.append(call()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref)


def test_threads_at_once():
    """Host threads that call the operators side by side, each on a stream of its own."""
    cases = [batch(400 + 100 * i, 131, 64, 6, 5, 20 + i) for i in range(4)]
    w = experts(131, 64, 32, 4)
    small = [dict(s, logits=s["logits"][:2], x=s["x"][:2].to(BF16)) for s in cases]
    want = [(train(s), decode(t, w)) for s, t in zip(cases, small)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                r, d = train(cases[i]), decode(small[i], w)
                torch.cuda.current_stream().synchronize()
                if not (same(want[i][0], r) and same(want[i][1], d)):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_status_stays_clear():
    s = batch(3, 40, 256, 6, 1, 12)
    w = experts(40, 256, 128, 4)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    idx, gates = moe.select_experts(s["logits"], 6)
    h = moe.w4_matvec(s["x"], *w["gate"], up=w["up"], idx=idx, status=status)
    y = moe.w4_matvec(h, *w["down"], idx=idx, weights=gates, status=status)
    assert int(status) == 0
    assert torch.equal(y, moe.w4_matvec(h, *w["down"], idx=idx, weights=gates))


def test_rows_behind_four_gigabytes():
    """Logits whose rows lie beyond 2^32 bytes, in a matrix of which the calls see a few columns."""
    T, E, k, wide = 70_000, 64, 4, 32_768
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    big = torch.empty(T, wide, dtype=BF16, device=DEV)
    x = big[:, 64:64 + E]
    x.copy_(ops.data(T, E, BF16, 3))
    packed = x.contiguous()
    idx, gates = moe.select_experts(x, k)
    want = moe.select_experts(packed, k)
    assert torch.equal(idx, want[0]) and torch.equal(gates, want[1])
    a, b = moe.balance_loss(x, idx), moe.balance_loss(packed, idx)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    one = torch.ones(1, device=DEV)
    d = [moe.router_backward(z, idx, d_gates=gates, d_loss=one, counts=r[1], tokens=r[2]) for z, r in ((x, a), (packed, b))]
    assert torch.equal(*d)


def test_losses_in_one_workspace():
    """Back to back in the same workspace and outputs, other slots each time: parts left from the call before would
    show in the counts."""
    T, E, k, S = 3001, 896, 16, 7
    s = batch(T, E, 8, k, S, 13)
    idx = [moe.select_experts(s["logits"] * (1 - 0.3 * i), k)[0] for i in range(8)]
    L, stream = moe.lib(), torch.cuda.current_stream().cuda_stream
    size = L.moe_balance_loss_workspace_bytes(T, E, S)
    work = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    out = [torch.empty(S, device=DEV), torch.empty(S, E, dtype=torch.int32, device=DEV), torch.empty(S, dtype=torch.int32, device=DEV)]
    kept = []
    torch.cuda.synchronize()
    for i in idx:
        a = router._BalanceLossArgs(s["logits"].data_ptr(), E, i.data_ptr(), s["sequences"].data_ptr(), *(t.data_ptr() for t in out),
                                    work.data_ptr(), size, T, E, k, S, router.DTYPES[F32], router.SCORE_SIGMOID_BIAS)
        assert L.moe_balance_loss(a, stream) == moe.MOE_OK
        kept.append([t.clone() for t in out])
    for i, got in zip(idx, kept):
        assert all(torch.equal(p, q) for p, q in zip(got, moe.balance_loss(s["logits"], i, sequences=s["sequences"])))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,S", [(500, 896, 3), (20_000, 896, 40), (20_000, 256, 5), (9000, 512, 1), (1000, 32, 12)])
def test_losses_of_rows_mostly_without_slots(T, E, S, dtype):
    """Runs of rows whose tokens are routed nowhere, which a warp passes in no time while their copies are on the way."""
    s = batch(T, E, 8, 4, S, T + E, dtype)
    s["logits"] = s["logits"] + torch.arange(T, device=DEV).to(dtype)[:, None] % 7         # rows of different size
    idx, _ = moe.select_experts(s["logits"], 4)
    routed = torch.rand(T, generator=ops.gen(T), device=DEV) < 0.03
    idx = torch.where(routed[:, None], idx, -1).contiguous()
    for _ in range(3):
        for score in ("sigmoid", "softmax"):
            ops.check_loss(s["logits"], idx, score, s["sequences"])
