"""The operators round the layer as they are used together: a block of expert
products in four bits between its norms, the layer inside its block, and the
circumstances of real programs (streams, captured graphs, another device).

Each step of a chain is compared with plain arithmetic in 64 bits on that
step's own inputs, within the tolerance that the step's own test derives."""
import numpy as np
import pytest
import torch

import synth
import moe_expert_layer_top16_gb300 as moe
from gpu_util import gpu_plan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16


def rms(v, eps=1e-6):
    return (v.square().mean(-1, keepdim=True) + eps).sqrt()


def make(T, k, E, D, I, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    idx = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    idx[::5, -1] = -1                                       # some slots are routed nowhere
    w = torch.rand(T, k, generator=g, device=DEV) + 0.1
    return dict(x=r(T, D, std=2.0).to(BF16), idx=idx, gates=w / w.sum(1, keepdim=True),
                up=moe.mxfp4_quantize(r(E, I, D, std=0.05)), down=moe.mxfp4_quantize(r(E, D, I, std=0.05)),
                w_pre=1 + r(D, std=0.1), w_post=1 + r(D, std=0.1), gate=0.5 + r(D, std=0.1))


def block(s, E):
    """Norm, rows to their experts, two four-bit products an expert, rows back, norm."""
    _, u = moe.block_norm(s["x"], w_pre=s["w_pre"])
    offsets, order, pos = moe.sort_by_expert(s["idx"], E)
    codes, scales = moe.mxfp4_quantize(u)
    n = pos.numel()
    rows = moe.permute(codes, pos, out=torch.zeros(n, codes.shape[1], dtype=torch.uint8, device=DEV))
    row_scales = moe.permute(scales, pos, out=torch.zeros(n, scales.shape[1], dtype=torch.uint8, device=DEV))
    mid = moe.mx4_gemm(*s["up"], rows, row_scales, offsets=offsets, out=torch.zeros(n, s["up"][0].shape[1], dtype=BF16, device=DEV))
    out = moe.mx4_gemm(*s["down"], *moe.mxfp4_quantize(mid), offsets=offsets,
                       out=torch.zeros(n, s["x"].shape[1], dtype=F32, device=DEV))
    y = moe.unpermute(out, pos, s["gates"])
    h, v = moe.block_norm(s["x"], y, w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per="channel", res_scale=0.9)
    return dict(u=u, offsets=offsets, order=order, pos=pos, codes=codes, scales=scales, rows=rows, row_scales=row_scales,
                mid=mid, out=out, y=y, h=h, v=v)


@pytest.mark.parametrize("T,k,E,D,I", [(1, 4, 8, 256, 128), (50, 3, 7, 384, 256), (300, 8, 40, 512, 384)])
def test_block_of_four_bit_experts(T, k, E, D, I):
    s = make(T, k, E, D, I)
    r = block(s, E)
    x = s["x"].double()
    ref = s["w_pre"].double() * x / rms(x)
    assert ((r["u"].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + (D / 64 + 16) * 2.0 ** -24)).all()
    order, bounds = r["order"].tolist(), r["offsets"].tolist()
    kept = [o for o in order if o >= 0]
    token = torch.tensor([o // k for o in kept], device=DEV, dtype=torch.long)
    assert bounds[-1] == len(kept) == int((s["idx"] >= 0).sum())
    assert torch.equal(r["rows"][:len(kept)], r["codes"][token]) and torch.equal(r["row_scales"][:len(kept)], r["scales"][token])
    # the products, a group at a time, on the values that the codes stand for
    for weights, a, out, half in ((s["up"], (r["rows"], r["row_scales"]), r["mid"], 2.0 ** -8),
                                  (s["down"], moe.mxfp4_quantize(r["mid"]), r["out"], 2.0 ** -24)):
        wv, av = moe.mxfp4_decode(*weights).double(), moe.mxfp4_decode(*a).double()
        K = av.shape[1]
        for e in range(E):
            lo, hi = bounds[e], bounds[e + 1]
            exact, mag = av[lo:hi] @ wv[e].T, av[lo:hi].abs() @ wv[e].abs().T
            tol = mag * ((K + 8) * 2.0 ** -22)
            assert ((out[lo:hi].double() - exact).abs() <= tol + (exact.abs() + tol) * half).all()
    # back to the tokens, and the norm behind the block
    y = torch.zeros(T, D, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(y)
    g = s["gates"].double().reshape(-1)[torch.tensor(kept, device=DEV, dtype=torch.long)].unsqueeze(-1)
    y.index_add_(0, token, g * r["out"][:len(kept)].double())
    mag.index_add_(0, token, g * r["out"][:len(kept)].double().abs())
    assert ((r["y"].double() - y).abs() <= mag * ((k + 2) * 2.0 ** -24)).all()
    yd = r["y"].double()
    add = s["gate"].double() * s["w_post"].double() * yd / rms(yd)
    ref = 0.9 * x + add
    tol = add.abs() * (D / 64 + 16) * 2.0 ** -24 + ref.abs() * 2.0 ** -23
    assert ((r["h"].double() - ref).abs() <= tol + (ref.abs() + tol) * 2.0 ** -8).all()


def test_training_step_gradients_meet():
    """The gradients of norm -> rows -> combine -> norm, chained by hand, against autograd of the same in 64 bits."""
    T, k, E, D = 37, 4, 9, 120
    s = make(T, k, E, 128, 128, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *z: torch.randn(*z, generator=g, device=DEV)  # noqa: E731
    x, w_pre, w_post, gate = r(T, D), 1 + 0.1 * r(D), 1 + 0.1 * r(D), 0.5 + 0.1 * r(T)
    dh, dv = r(T, D), r(T, D)
    _, _, pos = moe.sort_by_expert(s["idx"], E)
    zeros = torch.zeros(T * k, D, device=DEV)
    _, u = moe.block_norm(x, w_pre=w_pre)
    rows = moe.permute(u, pos, out=zeros.clone())
    y = moe.unpermute(rows, pos, s["gates"])
    h, v = moe.block_norm(x, y, w_post=w_post, w_pre=w_pre, gate=gate, gate_per="token", res_scale=0.8)
    out = moe.block_norm_backward(dh, dv, h, y, w_post=w_post, w_pre=w_pre, gate=gate, gate_per="token", res_scale=0.8)
    d_rows, d_gates = moe.unpermute_backward(out["dy"], rows, pos, s["gates"], out=zeros.clone())
    du = moe.permute_backward(d_rows, pos)
    inn = moe.block_norm_backward(None, du, x, w_pre=w_pre)
    dx, dw_pre = out["dx"] + inn["dx"], out["dw_pre"] + inn["dw_pre"]
    # the same in 64 bits
    leaf = {n: t.double().requires_grad_() for n, t in dict(x=x, w_pre=w_pre, w_post=w_post, gate=gate, gates=s["gates"]).items()}
    ud = leaf["w_pre"] * leaf["x"] / rms(leaf["x"])
    share = (leaf["gates"] * (s["idx"] >= 0)).sum(1, keepdim=True)
    yd = share * ud
    hd = 0.8 * leaf["x"] + leaf["gate"].unsqueeze(-1) * leaf["w_post"] * yd / rms(yd)
    vd = leaf["w_pre"] * hd / rms(hd)
    ((hd * dh.double()).sum() + (vd * dv.double()).sum()).backward()
    for n, got in (("x", dx), ("w_pre", dw_pre), ("w_post", out["dw_post"]), ("gate", out["d_gate"])):
        want = leaf[n].grad
        assert float((got.double() - want).norm()) <= 1e-5 * float(want.norm()), n
    # a gate's gradient is <dy, u>: through the norm behind it, which takes no scale, it nearly cancels
    want = leaf["gates"].grad * (s["idx"] >= 0)
    size = (out["dy"].double().abs() * u.double().abs()).sum(-1, keepdim=True)
    assert ((d_gates.double() - want).abs() <= 1e-5 * size).all() and (d_gates[s["idx"] < 0] == 0).all()


@pytest.mark.parametrize("out,x_dtype", [("f32", F32), ("bf16", BF16)])
def test_layer_inside_its_block(out, x_dtype):
    """forward_block is the norm, the layer and the norm, bit for bit, for two blocks in a row."""
    wl = synth.workload("tiny" if out == "f32" else "tiny+bf16")
    plan, _ = gpu_plan(wl)
    g = torch.Generator(device=DEV).manual_seed(1)
    D = wl.d_model
    for T in (1, 17, 64):
        x = (2 * torch.randn(T, D, generator=g, device=DEV)).to(x_dtype)
        w, p, gate, n = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(4))
        h, nxt = plan.forward_block(x, w_pre=w, w_post=p, gate=gate, gate_per="channel", res_scale=0.7, next_w_pre=n, need_next_u=True)
        _, u = moe.block_norm(x, w_pre=w, u_dtype=BF16)
        y = plan.forward(u)
        rh, ru = moe.block_norm(x, y, w_post=p, w_pre=n, gate=gate, gate_per="channel", res_scale=0.7, u_dtype=BF16)
        assert torch.equal(h, rh) and torch.equal(nxt, ru)
        h2, none = plan.forward_block(h, u=nxt, w_post=p)
        rh2, _ = moe.block_norm(rh, plan.forward(ru), w_post=p, need_u=False)
        assert none is None and torch.equal(h2, rh2)
    tok = torch.rand(T, generator=g, device=DEV)
    h3, _ = plan.forward_block(x, gate=tok, gate_per="token")
    assert torch.equal(h3, moe.block_norm(x, plan.forward(moe.block_norm(x, u_dtype=BF16)[1]), gate=tok, gate_per="token", need_u=False)[0])
    assert plan.device_status() == moe.MOE_OK
    for bad in (dict(gate=tok, gate_per="channel"), dict(u=x.float()), dict(next_w_pre=w), dict(w_pre=w[:-1]), dict(eps=-1.0)):
        with pytest.raises(moe.MoeError):
            plan.forward_block(x, **bad)
    with pytest.raises(moe.MoeError):
        plan.forward_block(torch.zeros(wl.tokens + 1, D, device=DEV))
    plan.close()


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


def test_captured_and_replayed():
    """A block captured into two graphs replays to the same bits as the eager calls, each graph on its own workspaces."""
    s = make(5000, 2, 40, 256, 128, seed=5)
    D = 256
    dh = torch.randn(5000, D, device=DEV).to(BF16)

    def step():
        r = block(s, 40)
        r.update(moe.block_norm_backward(dh, dh, r["h"], r["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                                         gate_per="channel", res_scale=0.9))
        r["d_rows"], r["d_w"] = moe.unpermute_backward(r["dy"], r["out"], r["pos"], s["gates"], out=torch.zeros_like(r["out"]))
        return {n: t for n, t in r.items() if t is not None}

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
        graphs.append((g, r))
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, r in graphs:
        assert same(eager, r)
    # new inputs in the captured buffers
    s["x"].mul_(-0.5)
    again = step()
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, r in graphs:
        assert same(again, r)


def test_two_streams_at_once():
    """Calls of the same operators on two streams do not disturb each other."""
    a, b = make(3000, 2, 40, 256, 128, seed=6), make(2500, 2, 40, 256, 128, seed=7)
    ra, rb = block(a, 40), block(b, 40)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(one):
            qa = block(a, 40)
        with torch.cuda.stream(two):
            qb = block(b, 40)
    torch.cuda.synchronize()
    assert same(ra, qa) and same(rb, qb)


def test_stream_argument():
    s = make(200, 4, 9, 256, 128, seed=8)
    ref = block(s, 9)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _, u = moe.block_norm(s["x"], w_pre=s["w_pre"], stream=side)
    offsets, order, pos = moe.sort_by_expert(s["idx"], 9, stream=side)
    codes, scales = moe.mxfp4_quantize(u, stream=side)
    rows = moe.permute(codes, pos, stream=side)
    out = moe.mx4_gemm(s["up"][0][0], s["up"][1][0], codes, scales, stream=side)
    y = moe.unpermute(ref["out"], pos, s["gates"], stream=side)
    side.synchronize()
    n = int(offsets[-1])
    assert torch.equal(u, ref["u"]) and torch.equal(order, ref["order"]) and torch.equal(codes, ref["codes"])
    assert torch.equal(rows[:n], ref["rows"][:n]) and torch.equal(y, ref["y"])
    assert torch.equal(out, moe.mx4_gemm(s["up"][0][0], s["up"][1][0], codes, scales))


def test_tensors_of_several_devices_are_refused():
    x = torch.zeros(4, 64, device=DEV)
    pos = torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: moe.permute(x, pos), lambda: moe.unpermute(x, pos), lambda: moe.block_norm(x, x.cpu()),
              lambda: moe.block_norm(x, w_pre=torch.ones(64)), lambda: moe.unpermute_backward(x, x.cpu(), pos.to(DEV)),
              lambda: moe.mx4_gemm(*moe.mxfp4_quantize(torch.zeros(4, 128, device=DEV)), pos.to(torch.uint8), pos.to(torch.uint8))):
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.code == moe.MOE_ERR_INVALID_ARG


def test_same_bits_again():
    s = make(777, 6, 33, 512, 256, seed=9)
    assert same(block(s, 33), block(s, 33))


def test_wide_batch_of_rows():
    """More rows than a grid's second dimension holds."""
    T, k, E, D = 70000, 2, 16, 40
    idx = torch.randint(0, E, (T, k), device=DEV, dtype=torch.int32)
    offsets, order, pos = moe.sort_by_expert(idx, E)
    x = torch.randn(T, D, device=DEV)
    rows = moe.permute(x, pos)
    assert torch.equal(moe.permute_backward(rows, pos), 2 * x)
    want = torch.sort(idx.reshape(-1), stable=True)
    assert torch.equal(order.long(), want.indices)
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(want.values.cpu().numpy(), np.arange(E + 1)))
    h, u = moe.block_norm(x, x)
    keep = [0, 65535, 65536, T - 1]
    assert torch.equal(h[keep], moe.block_norm(x[keep], x[keep])[0])


def test_memory_of_the_streams_argument():
    """Copies and workspaces of a call belong to the stream it runs on: the current stream may hand out and overwrite
    whatever was allocated and freed there while the other stream has not begun."""
    T, k, E, D = 3000, 4, 40, 256
    g = torch.Generator(device=DEV).manual_seed(3)
    idx = torch.randint(0, E, (k, T), generator=g, device=DEV, dtype=torch.int32).t()            # strided: copied first
    x = torch.randn(D, T, generator=g, device=DEV).t()
    du, y = torch.randn(T, D, generator=g, device=DEV), torch.randn(D, T, generator=g, device=DEV).t()
    w = torch.randn(D, generator=g, device=DEV)

    def calls(**kw):
        offsets, order, pos = moe.sort_by_expert(idx, E, **kw)
        b = moe.block_norm_backward(None, du, x, y, w_post=w, w_pre=w, **kw)
        return dict(offsets=offsets, order=order, pos=pos, rows=moe.permute(x, pos, **kw), q=moe.mxfp4_quantize(x, **kw)[0],
                    u=moe.block_norm(x, y, w_pre=w, **kw)[1], **{n: t for n, t in b.items() if t is not None})
    ref = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                      # about ten milliseconds
        got = calls(stream=side)
        junk = [torch.full((n,), -1, dtype=torch.int32, device=DEV) for n in (T * k, T * k, T * D, T * D, T * D, 2 * D * T, 64 * E) * 4]
        torch.cuda.synchronize()
        assert same(ref, got)
        del junk


def test_stream_of_another_device_kind_is_refused():
    x = torch.zeros(4, 64, device=DEV)
    for stream in (torch.cuda.current_stream().cuda_stream, torch.cuda.Event()):
        with pytest.raises(moe.MoeError) as e:
            moe.block_norm(x, stream=stream)
        assert e.value.code == moe.MOE_ERR_INVALID_ARG


def test_more_slots_than_32_bits_are_refused():
    idx = torch.zeros(1, 1, dtype=torch.int32, device=DEV).expand(2 ** 31, 1)
    with pytest.raises(moe.MoeError) as e:
        moe.sort_by_expert(idx, 4)
    assert e.value.code == moe.MOE_ERR_INVALID_ARG


def test_rows_behind_four_gigabytes():
    """Row offsets past 32 bits, in elements: a few tokens in the last rows of a tall matrix."""
    D, n = 8192, 2 ** 31 // 8192 + 40
    rows = torch.zeros(n, D, dtype=BF16, device=DEV)
    x = torch.randn(5, D, device=DEV).to(BF16)
    pos = torch.tensor([[n - 1, 0], [n - 2, -1], [n - 30, 3], [n - 31, n], [2, n - 9]], dtype=torch.int32, device=DEV)
    moe.permute(x, pos, out=rows)
    keep = pos.clamp(-1, n)
    for t in range(5):
        for p in keep[t].tolist():
            if 0 <= p < n:
                assert torch.equal(rows[p], x[t])
    w = torch.rand(5, 2, device=DEV)
    y = moe.unpermute(rows, pos, w, out_dtype=F32)
    ok = ((pos >= 0) & (pos < n)).float()
    want = x.double() * (w * ok).double().sum(1, keepdim=True)
    assert ((y.double() - want).abs() <= 3 * 2.0 ** -24 * x.double().abs() * (w * ok).double().sum(1, keepdim=True)).all()
    d_rows, d_w = moe.unpermute_backward(x, rows, pos, w, out=torch.zeros_like(rows))
    for t in range(5):
        for j, p in enumerate(pos[t].tolist()):
            if 0 <= p < n:
                assert torch.equal(d_rows[p], (x[t].float() * w[t, j]).to(BF16))
    del d_rows
    ref = (x.double() ** 2).sum(1, keepdim=True) * ok.double()
    assert ((d_w.double() - ref).abs() <= ref * (D / 32 + 8) * 2.0 ** -24).all()
    # the norms' first and last rows
    tall = rows.view(n, D)
    tall[-1], tall[0] = x[0], x[1]
    h, u = moe.block_norm(tall)
    assert torch.equal(u[[0, -1]], moe.block_norm(tall[[0, -1]])[1])
