"""The norms behind and before a block with gate and residual scale, and their
gradients, against the formulas in 64 bits.

Tolerances.  A row's sum of D squares in fp32 is off by at most
(D / threads + 12) 2^-24 relative, with at least 32 threads; half of it reaches
the reciprocal root, a few roundings follow: c = (D / 64 + 16) 2^-24 covers each
normalised value, relative to itself.  An output adds half a step of its type.
Gradients subtract two such terms, so they are compared with the magnitudes of
both; column sums add T 2^-24 of the sum of magnitudes."""
import pytest
import torch

import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}
EPS = 1e-6


def make(T, D, tx, ty, tw, gate, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    s = dict(x=(r(T, D, std=2.0)).to(tx), y=(r(T, D, std=0.3)).to(ty), w_post=(1 + r(D, std=0.1)).to(tw),
             w_pre=(1 + r(D, std=0.1)).to(tw), gate=None)
    if gate:
        s["gate"] = (0.5 + r(D if gate == "channel" else T, std=0.3)).to(tw)
    s["dh"], s["du"] = r(T, D, std=0.1).to(tx), r(T, D, std=0.2)
    return s


def gate64(s, gate):
    if gate is None:
        return torch.ones((), dtype=torch.float64, device=DEV)
    return s["gate"].double() if gate == "channel" else s["gate"].double().unsqueeze(-1)


def rms(v, eps=EPS):
    return (v.square().mean(-1, keepdim=True) + eps).sqrt()


CASES = [(1, 7168, BF16, F32, F32, "channel"), (1, 1, F32, F32, F32, "token"), (3, 8, BF16, BF16, BF16, "channel"),
         (5, 7, F16, F16, F16, "token"), (64, 256, F32, F32, F32, None), (130, 1001, BF16, F32, F32, "channel"),
         (33, 4096, F16, F32, F16, "token"), (7, 4104, F32, BF16, F32, "channel"), (9, 8200, BF16, BF16, F32, None),
         (2, 16384, F32, F32, F32, "channel"), (2, 16383, BF16, BF16, F32, "token"), (700, 64, BF16, BF16, F32, "token"),
         (4, 5000, BF16, BF16, BF16, "channel"), (3, 4099, F32, F32, F32, "channel")]


@pytest.mark.parametrize("T,D,tx,ty,tw,gate", CASES)
@pytest.mark.parametrize("tu", [None, BF16])
def test_forward(T, D, tx, ty, tw, gate, tu):
    s = make(T, D, tx, ty, tw, gate)
    tu_ = tu or tx
    h, u = moe.block_norm(s["x"], s["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per=gate,
                          res_scale=0.75, eps=EPS, u_dtype=tu)
    c = (D / 64 + 16) * 2.0 ** -24
    add = gate64(s, gate) * s["w_post"].double() * s["y"].double() / rms(s["y"].double())
    ref = 0.75 * s["x"].double() + add
    tol = add.abs() * c + ref.abs() * 2.0 ** -23
    assert h.dtype == tx and ((h.double() - ref).abs() <= tol + (ref.abs() + tol) * HALF[tx] + TINY[tx]).all()
    f = h.double()
    ref = s["w_pre"].double() * f / rms(f)
    assert u.dtype == tu_ and ((u.double() - ref).abs() <= ref.abs() * (c + HALF[tu_] * (1 + c)) + TINY[tu_]).all()
    # the parts alone give the same
    h2, none = moe.block_norm(s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], gate_per=gate, res_scale=0.75, eps=EPS,
                              need_u=False)
    assert none is None and torch.equal(h2, h)
    x2, u2 = moe.block_norm(h, w_pre=s["w_pre"], eps=EPS, u_dtype=tu)
    assert x2 is h and torch.equal(u2, u)
    # in place on the residual stream
    x3 = s["x"].clone()
    h3, u3 = moe.block_norm(x3, s["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per=gate,
                            res_scale=0.75, eps=EPS, u_dtype=tu, out_h=x3)
    assert h3 is x3 and torch.equal(x3, h) and torch.equal(u3, u)


@pytest.mark.parametrize("T,D,tx,ty,tw,gate", CASES)
@pytest.mark.parametrize("given", ["both", "dh", "du", "pre"])
def test_backward(T, D, tx, ty, tw, gate, given):
    s = make(T, D, tx, ty, tw, gate, seed=1)
    dh = s["dh"] if given in ("both", "dh", "pre") else None
    du = s["du"].to(tx) if given in ("both", "du", "pre") else None
    kw = dict(w_pre=s["w_pre"] if du is not None else None, res_scale=0.75, eps=EPS)
    if given != "pre":
        kw.update(w_post=s["w_post"], gate=s["gate"], gate_per=gate)
    y_in = None if given == "pre" else s["y"]
    got = moe.block_norm_backward(dh, du, s["x"], y_in, **kw)
    c = (D / 64 + 24) * 2.0 ** -24
    h, total, mag = s["x"].double(), torch.zeros(T, D, dtype=torch.float64, device=DEV), torch.zeros(T, D, dtype=torch.float64, device=DEV)
    if dh is not None:
        total, mag = total + dh.double(), mag + dh.double().abs()
    if du is not None:
        a, hh = du.double() * s["w_pre"].double(), h / rms(h)
        total = total + (a - hh * (a * hh).mean(-1, keepdim=True)) / rms(h)
        mag = mag + (a.abs() + hh.abs() * (a * hh).abs().mean(-1, keepdim=True)) / rms(h)
        col = (du.double() * hh).abs().sum(0)
        assert ((got["dw_pre"].double() - (du.double() * hh).sum(0)).abs() <= col * (c + (T + 24) * 2.0 ** -24)).all()
    else:
        assert got["dw_pre"] is None
    scale = 1.0 if given == "pre" else 0.75
    ref = scale * total
    assert got["dx"].dtype == tx
    assert ((got["dx"].double() - ref).abs() <= mag * c + (ref.abs() + mag * c) * HALF[tx] + TINY[tx]).all()
    if given == "pre":
        assert got["dy"] is None and got["dw_post"] is None and got["d_gate"] is None
        return
    y, g, w = s["y"].double(), gate64(s, gate), s["w_post"].double()
    yh, p, pm = y / rms(y), total * g * w, mag * (g * w).abs()
    ref = (p - yh * (p * yh).mean(-1, keepdim=True)) / rms(y)
    m = (pm + yh.abs() * (pm * yh.abs()).mean(-1, keepdim=True)) / rms(y)
    assert got["dy"].dtype == ty
    assert ((got["dy"].double() - ref).abs() <= m * 2 * c + (ref.abs() + m * 2 * c) * HALF[ty] + TINY[ty]).all()
    terms, tm = total * yh, mag * yh.abs()
    tol = (tm * g.abs()).sum(0) * (2 * c + (T + 24) * 2.0 ** -24)
    assert ((got["dw_post"].double() - (terms * g).sum(0)).abs() <= tol).all()
    if gate == "channel":
        tol = tm.sum(0) * w.abs() * (2 * c + (T + 24) * 2.0 ** -24)
        assert ((got["d_gate"].double() - (terms * w).sum(0)).abs() <= tol).all()
    elif gate == "token":
        tol = (tm * w.abs()).sum(-1) * 3 * c
        assert got["d_gate"].shape == (T,) and ((got["d_gate"].double() - (terms * w).sum(-1)).abs() <= tol).all()
    else:
        assert got["d_gate"] is None


def test_gradient_by_differences():
    """Directional derivatives in 64 bits of the formula that the forward test holds the kernel to."""
    T, D = 6, 40
    s = make(T, D, F32, F32, F32, "channel", seed=2)
    names = ("x", "y", "w_post", "w_pre", "gate")
    g = torch.Generator(device=DEV).manual_seed(9)
    leaf = {n: s[n].double().requires_grad_() for n in names}

    def f(v):
        h = 0.75 * v["x"] + v["gate"] * v["w_post"] * v["y"] / rms(v["y"])
        return (h * s["dh"].double()).sum() + (v["w_pre"] * h / rms(h) * s["du"].double()).sum()

    h, _ = moe.block_norm(s["x"], s["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], res_scale=0.75, eps=EPS)
    got = moe.block_norm_backward(s["dh"], s["du"], h, s["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                                  res_scale=0.75, eps=EPS)
    for n, d in (("x", "dx"), ("y", "dy"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("gate", "d_gate")):
        v = torch.randn(leaf[n].shape, generator=g, device=DEV, dtype=torch.float64)
        e = 1e-5
        up, down = dict(leaf), dict(leaf)
        up[n], down[n] = leaf[n] + e * v, leaf[n] - e * v
        slope = float((f(up) - f(down)).detach()) / (2 * e)
        mine = float((got[d].double() * v).sum())
        # fp32 values (h among them, rounded once) against a difference quotient: both far below 1e-4 of the terms
        assert abs(mine - slope) <= 1e-4 * float((got[d].double() * v).abs().sum()), n


def test_shapes_strides_and_defaults():
    B, S, D = 3, 5, 72
    wide = torch.randn(B, S, 2 * D, device=DEV)
    x, y = wide[..., :D], wide[..., D:]
    h, u = moe.block_norm(x, y)
    hc, uc = moe.block_norm(x.contiguous().view(-1, D), y.contiguous().view(-1, D))
    assert h.shape == x.shape and torch.equal(h.reshape(-1, D), hc) and torch.equal(u.reshape(-1, D), uc)
    out = torch.full((B * S, D + 8), 9.0, device=DEV)
    moe.block_norm(x.reshape(-1, D), y.reshape(-1, D), out_h=out[:, :D])
    assert torch.equal(out[:, :D], hc) and (out[:, D:] == 9).all()
    got = moe.block_norm_backward(torch.ones((), device=DEV).expand(B, S, D), None, h, y)
    assert got["dx"].shape == x.shape and got["dw_post"] is None
    ones = torch.ones(D, device=DEV)
    want = moe.block_norm_backward(torch.ones(B * S, D, device=DEV), None, hc, y.contiguous().view(-1, D), w_post=ones)
    assert torch.equal(got["dy"].reshape(-1, D), want["dy"]) and want["dw_post"].shape == (D,)


def test_empty_rows_and_zero_rows():
    D = 48
    w = torch.ones(D, device=DEV)
    e = torch.empty(0, D, device=DEV)
    h, u = moe.block_norm(e, e, w_post=w, w_pre=w)
    assert h.shape == (0, D) and u.shape == (0, D)
    got = moe.block_norm_backward(e, e, e, e, w_post=w, w_pre=w, gate=w)
    assert got["dx"].shape == (0, D)
    assert all((got[n] == 0).all() and got[n].shape == (D,) for n in ("dw_post", "dw_pre", "d_gate"))
    z = torch.zeros(3, D, device=DEV)
    h, u = moe.block_norm(z, z, w_post=w, w_pre=w)
    assert (h == 0).all() and (u == 0).all()
    got = moe.block_norm_backward(z + 1, z, z, z, w_post=w, w_pre=w)
    assert (got["dx"] == 1).all() and torch.isfinite(got["dy"]).all()


def test_not_a_number_stays_in_its_row():
    x = torch.randn(5, 64, device=DEV)
    y = torch.randn(5, 64, device=DEV)
    ref = moe.block_norm(x, y)
    y[2, 3] = float("nan")
    h, u = moe.block_norm(x, y)
    keep = [0, 1, 3, 4]
    assert torch.equal(h[keep], ref[0][keep]) and torch.equal(u[keep], ref[1][keep])
    assert h[2].isnan().all() and u[2].isnan().all()


def test_same_call_same_bits():
    s = make(999, 1000, BF16, BF16, F32, "channel", seed=4)
    call = lambda: moe.block_norm_backward(s["dh"], s["du"].bfloat16(), s["x"], s["y"], w_post=s["w_post"],  # noqa: E731
                                           w_pre=s["w_pre"], gate=s["gate"])
    a, b = call(), call()
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("D", [1, 2, 3, 5, 7, 9, 13, 255, 1003])
@pytest.mark.parametrize("T", [1, 2, 9, 1300])
def test_narrow_and_odd_rows(T, D):
    """Rows that share 16-byte words: neighbours and what lies behind the last row stay as they were."""
    for t in (F32, BF16):
        s = make(T, D, t, t, F32, None, seed=T + D)
        w, r = s["w_post"], s["w_pre"]
        flat = torch.full((T * D + 64,), 3.0, device=DEV).to(t)
        h_out, u_out = flat[:T * D].view(T, D), flat.clone()[:T * D].view(T, D)
        h, u = moe.block_norm(s["x"], s["y"], w_post=w, w_pre=r, res_scale=0.75, eps=EPS, out_h=h_out, out_u=u_out)
        assert (flat[T * D:] == 3).all()
        c = (D / 64 + 16) * 2.0 ** -24
        add = w.double() * s["y"].double() / rms(s["y"].double())
        ref = 0.75 * s["x"].double() + add
        tol = add.abs() * c + ref.abs() * 2.0 ** -23
        assert ((h.double() - ref).abs() <= tol + (ref.abs() + tol) * HALF[t] + TINY[t]).all()
        f = h.double()
        ref = r.double() * f / rms(f)
        assert ((u.double() - ref).abs() <= ref.abs() * (c + HALF[t] * (1 + c)) + TINY[t]).all()
        got = moe.block_norm_backward(s["dh"], None, h, s["y"], w_post=w, res_scale=0.75, eps=EPS)
        yh = s["y"].double() / rms(s["y"].double())
        terms = s["dh"].double() * yh
        tol = terms.abs().sum(0) * (2 * c + (T + 24) * 2.0 ** -24)
        assert ((got["dw_post"].double() - terms.sum(0)).abs() <= tol).all()


# rows that several blocks share, many rows a block, first and last windows that are partial
WIDE = [(300, 7168, F32, F32, F32, "channel"), (41, 8200, F32, F32, F32, "token"), (600, 4101, F32, F32, F32, "channel"),
        (333, 8193, BF16, BF16, F32, "channel"), (190, 12288, BF16, BF16, BF16, "token"), (170, 7167, BF16, F32, F32, "channel"),
        (100, 16383, F32, F32, F32, "channel"), (640, 16384, F32, F32, F32, None), (90, 16384, F16, F32, F32, "token"),
        (1300, 2048, BF16, F32, F32, "channel"), (1300, 2056, BF16, BF16, F32, "token"), (1300, 1028, F32, F32, F32, "channel"),
        (900, 1031, F16, F16, F32, "channel"), (700, 3583, BF16, F32, F32, "token"), (200, 7168, F16, F16, F16, "channel"),
        (500, 1000, F16, F32, F16, "token"), (2500, 512, F16, F16, F32, None), (200, 8192, F32, F32, F32, "channel"),
        (2500, 512, F32, F32, F32, "channel"), (2500, 1024, F32, F32, F32, "token"), (900, 5120, F32, F32, F32, "channel"),
        (2500, 511, BF16, BF16, F32, "channel"), (2500, 96, F16, F32, F32, None)]


@pytest.mark.parametrize("T,D,tx,ty,tw,gate", WIDE)
@pytest.mark.parametrize("given", ["both", "dh", "du", "pre"])
def test_backward_wide(T, D, tx, ty, tw, gate, given):
    test_backward(T, D, tx, ty, tw, gate, given)


@pytest.mark.parametrize("T,D,tx,ty,tw,gate", WIDE)
def test_forward_wide(T, D, tx, ty, tw, gate):
    test_forward(T, D, tx, ty, tw, gate, None)


@pytest.mark.parametrize("T,D,tx,ty,tw,gate", [WIDE[0], WIDE[2], WIDE[6]])
def test_backward_wide_again_and_in_a_graph(T, D, tx, ty, tw, gate):
    """Split rows: the same bits in every run, eager and captured, two replays at once on two streams."""
    s = make(T, D, tx, ty, tw, gate, seed=3)
    call = lambda: moe.block_norm_backward(s["dh"], s["du"].to(tx), s["x"], s["y"], w_post=s["w_post"], w_pre=s["w_pre"],  # noqa: E731
                                           gate=s["gate"], gate_per=gate, res_scale=0.75, eps=EPS)
    ref = call()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        for n, t in ref.items():
            assert torch.equal(t, out[n]), n


@pytest.mark.parametrize("T,D,t", [(64, 256, BF16), (1300, 1001, BF16), (300, 7168, F32), (200, 7168, F16), (41, 5001, F32)])
def test_backward_in_place(T, D, t):
    """dx over dh or du, dy over y: the same bits as with outputs of their own (and a misaligned base, element by element)."""
    import ctypes as C
    from moe_expert_layer_top16_gb300 import block
    code = block.DTYPES[t]
    s = make(T, D, t, t, F32, "channel", seed=7)
    du = s["du"].to(t)
    work = torch.empty(moe.lib().moe_block_norm_workspace_bytes(T, D) + 64, dtype=torch.uint8, device=DEV)

    def call(dh, du, y, dx, dy):
        grads = [torch.empty(D, device=DEV) for _ in range(3)]
        a = block._BlockNormBackwardArgs(
            dh.data_ptr(), D, du.data_ptr(), D, s["x"].data_ptr(), D, y.data_ptr(), D, s["w_post"].data_ptr(), s["w_pre"].data_ptr(),
            s["gate"].data_ptr(), dx.data_ptr(), D, dy.data_ptr(), D, *(g.data_ptr() for g in grads), work.data_ptr(), work.numel(),
            T, D, code, code, code, 0, moe.block.GATE_CHANNEL, 0.75, EPS)
        assert moe.lib().moe_block_norm_backward(C.byref(a), torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
        return [dx.clone(), dy.clone()] + grads

    for off in (0, 1):                                      # off: bases of one element more than a multiple of 16 bytes
        own = lambda v: torch.cat([v.reshape(-1)[:off], v.reshape(-1)])[off:].view(T, D)  # noqa: E731
        ref = call(own(s["dh"]), own(du), own(s["y"]), own(s["dh"]), own(s["y"]))
        dh, y = own(s["dh"]), own(s["y"])
        for got in (call(dh, own(du), y, dh, y),):
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
        u, y = own(du), own(s["y"])
        got = call(own(s["dh"]), u, y, u, y)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
