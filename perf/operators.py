"""The operators around a sparse MoE layer's experts, as workloads to time and compare.

Five kinds of pass, each the call that a program makes in training or serving:

  dispatch       the (token, slot) pairs sorted by expert, and the tokens' rows copied into that order;
                 with "back" also the gradient that returns to the tokens
  combine        the experts' rows back to their tokens, weighted by the gates; with "back" also the
                 gradients of the rows and of the gates
  norm           the RMS norm behind a block with its gate and residual scale, and the norm before the
                 next block, in one pass
  norm_backward  the gradients of that pass
  quantise       activations to MXFP4 and back to the values that the codes stand for
  product        activations quantised to MXFP4 and multiplied by MXFP4 weights, one matrix or one for
                 each expert's group of rows

Where `own` is false, run() computes them from elementary torch operations in 32 bits."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
RES_SCALE = 0.75

# E2M1's magnitudes and the midpoints between them; a value on a midpoint takes the smaller level.
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def listed():
    return [
        # one decoded token of the K3-shaped layer's latent path: 16 of 896 experts, rows of 3584
        dict(name="dispatch one token", kind="dispatch", tokens=1, k=16, experts=896, width=3584, type="bf16", drop=0.0, back=False),
        # a prefill batch of the same layer
        dict(name="dispatch prefill", kind="dispatch", tokens=8192, k=16, experts=896, width=3584, type="bf16", drop=0.0, back=False),
        # a training step of a small layer whose batch is padded (some slots routed nowhere), odd sizes
        dict(name="dispatch ragged, with gradient", kind="dispatch", tokens=1537, k=6, experts=61, width=1001, type="f16", drop=0.1, back=True),
        # a decode batch: the experts' fp32 outputs back to 64 tokens
        dict(name="combine decode", kind="combine", tokens=64, k=16, experts=896, width=3584, type="f32", drop=0.0, back=False),
        # a training step's combine and its gradients
        dict(name="combine train", kind="combine", tokens=4096, k=16, experts=896, width=3584, type="bf16", drop=0.02, back=True),
        # decode: behind the layer (which writes fp32) and before the next block
        dict(name="norm decode", kind="norm", tokens=64, width=7168, type="bf16", y_type="f32", gate="channel"),
        # prefill, the residual stream in bf16
        dict(name="norm prefill", kind="norm", tokens=8192, width=7168, type="bf16", y_type="bf16", gate="channel"),
        # a training step's backward pass
        dict(name="norm backward", kind="norm_backward", tokens=4096, width=7168, type="bf16", y_type="bf16", gate="channel"),
        # an fp32 residual stream of an odd width, one gate a token
        dict(name="norm backward odd", kind="norm_backward", tokens=777, width=3583, type="f32", y_type="f32", gate="token"),
        # a prefill batch's hidden states in four bits
        dict(name="quantise prefill", kind="quantise", tokens=8192, width=7168, type="bf16"),
        # decode on one of 14 expert-parallel slices: 64 experts' gate/up (2 x 512 rows), about one row each
        dict(name="product decode", kind="product", tokens=73, groups=64, rows=1024, width=3584, type="bf16", out="f32"),
        # prefill through the two shared experts' gate/up (2 x 2 x 2048 rows)
        dict(name="product prefill", kind="product", tokens=8192, groups=1, rows=8192, width=7168, type="bf16", out="bf16"),
    ]


def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("dispatch", "combine", "norm", "norm_backward", "quantise", "product"))
    t = rng.choice(("bf16", "bf16", "f16", "f32"))
    if kind in ("dispatch", "combine"):
        k = rng.choice((1, 2, 4, 6, 8, 16))
        width = _size(rng, 64, 7168)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        most = 8192 * 16 * 3584 // (4 * k * width)  # rows of any type, with their gradients
        return dict(kind=kind, tokens=_size(rng, 1, max(1, min(16384, most))), k=k, experts=max(k, _size(rng, 8, 896)), width=width, type=t,
                    drop=rng.choice((0.0, 0.0, 0.05, 0.5)), back=rng.random() < 0.5)
    if kind in ("norm", "norm_backward"):
        width = _size(rng, 64, 8192)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        most = 8192 * 7168 // (2 * width)
        return dict(kind=kind, tokens=_size(rng, 1, max(1, min(16384, most))), width=width, type=t, y_type=rng.choice((t, "f32")), gate=rng.choice(("none", "channel", "token")))
    if kind == "quantise":
        width = 32 * _size(rng, 2, 224)
        return dict(kind=kind, tokens=_size(rng, 1, max(1, min(16384, 8192 * 7168 // (2 * width)))), width=width, type=t)
    groups = rng.choice((1, 1, _size(rng, 2, 64)))
    rows, width = _size(rng, 128, 8192 if groups == 1 else 1024), 128 * _size(rng, 1, 56 if groups == 1 else 28)
    return dict(kind=kind, tokens=_size(rng, 1, 8192), groups=groups, rows=rows, width=width, type=t, out=rng.choice(("f32", "bf16")))


def work(c):
    e = {"bf16": 2, "f16": 2, "f32": 4}
    T, D, b = c["tokens"], c["width"], e[c["type"]]
    if c["kind"] in ("dispatch", "combine"):
        S = T * c["k"]
        rows = S * (1.0 - c["drop"]) * D * b
        if c["kind"] == "dispatch":  # the experts' numbers in, the tables out, the rows; the gradient reads as many rows and writes the tokens'
            return {"bytes": (12 * S + 4 * c["experts"] + 4 + T * D * b + rows) + ((rows + 4 * S + T * D * b) if c["back"] else 0), "flops": S * D if c["back"] else 0}
        # forward: rows, places and gates in, tokens out; back: the tokens' gradient and the rows in, the rows' and the gates' gradients out
        return {"bytes": rows + 8 * S + T * D * b + ((2 * rows + 12 * S + T * D * b) if c["back"] else 0), "flops": S * D * (6 if c["back"] else 2)}
    if c["kind"] == "norm":
        return {"bytes": T * D * (3 * b + e[c["y_type"]]) + 12 * D, "flops": 12 * T * D}
    if c["kind"] == "norm_backward":
        return {"bytes": T * D * (4 * b + 2 * e[c["y_type"]]) + 24 * D, "flops": 24 * T * D}
    if c["kind"] == "quantise":
        # the values in and out; the codes and scales, which the second call reads, both ways
        return {"bytes": T * D * (2 * b + 2 * 17 / 32), "flops": 4 * T * D}
    used = min(c["groups"], T)
    return {"bytes": T * D * b + used * c["rows"] * D * 17 / 32 + T * c["rows"] * e[c["out"]], "flops": 2 * T * c["rows"] * D}


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, type=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(type)


def _route(g, c):
    """The experts of each token's slots, by scores with an uneven popularity; a dropped slot has -1."""
    T, k, E = c["tokens"], c["k"], c["experts"]
    scores = torch.randn(T, E, generator=g, device=DEV) + 0.3 * torch.randn(E, generator=g, device=DEV)
    idx = scores.topk(k, dim=1).indices.to(torch.int32)
    if c["drop"]:
        idx = torch.where(torch.rand(T, k, generator=g, device=DEV) < c["drop"], torch.full_like(idx, -1), idx)
    gates = torch.rand(T, k, generator=g, device=DEV) + 0.05
    return idx, gates / gates.sum(1, keepdim=True)


def _sorted(idx, E):
    """Offsets [E + 1], the flat slot at each sorted place and the place of each slot (-1: none)."""
    flat = idx.reshape(-1)
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=DEV, dtype=key.dtype)).to(torch.int32)
    kept = key < E
    place = torch.arange(n, device=DEV, dtype=torch.int32)
    gone = torch.full_like(place, -1)
    slot_pos = torch.empty_like(place)
    slot_pos[order] = torch.where(kept, place, gone)
    return offsets, torch.where(kept, order.to(torch.int32), gone), slot_pos.view_as(idx)


def _encode(x):
    """MXFP4 of x [..., K] in 32 bits: level numbers with signs [..., K/32, 32] and exponents [..., K/32]."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)  # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    level = torch.bucketize(torch.ldexp(b.abs(), -e.unsqueeze(-1)), torch.tensor(MIDS, device=x.device))
    return level, torch.signbit(b), e


def _decode(level, negative, e):
    v = torch.tensor(LEVELS, device=level.device)[level]
    return torch.ldexp(torch.where(negative, -v, v), e.unsqueeze(-1)).flatten(-2)


def _codes(x):
    """The same as packed codes [..., K/2] and E8M0 scales [..., K/32]."""
    level, negative, e = _encode(x)
    code = (level + 8 * negative).to(torch.uint8).flatten(-2)
    code = torch.where((e == -127).repeat_interleave(32, -1), torch.zeros_like(code), code)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """What packed codes and scales stand for, in 32 bits."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, 32))
    return _decode((code & 7).long(), code >= 8, scales.to(torch.int32) - 127)


def prepare(case, seed):
    c, g = case, _generator(seed)
    t = TYPES[c["type"]]
    s = dict(case=case)
    if c["kind"] in ("dispatch", "combine"):
        T, k, D = c["tokens"], c["k"], c["width"]
        s["idx"], gates = _route(g, c)
        s["rows"] = torch.zeros(T * k, D, dtype=t, device=DEV)  # places behind the last routed slot stay zero
        if c["kind"] == "dispatch":
            s["x"] = _normal(g, T, D, type=t)
            if c["back"]:
                s["d_rows"] = _normal(g, T * k, D, type=t)
        else:
            _, s["sorted_slot"], s["slot_pos"] = _sorted(s["idx"], c["experts"])
            s["gates"] = gates
            s["y_rows"] = _normal(g, T * k, D, type=t)
            if c["back"]:
                s["dy"] = _normal(g, T, D, type=t)
    elif c["kind"] in ("norm", "norm_backward"):
        T, D, ty = c["tokens"], c["width"], TYPES[c["y_type"]]
        s["w_post"], s["w_pre"] = 1 + _normal(g, D, std=0.1), 1 + _normal(g, D, std=0.1)
        s["gate"] = {"none": None, "channel": 0.5 + _normal(g, D, std=0.2), "token": 0.5 + _normal(g, T, std=0.2)}[c["gate"]]
        s["y"] = _normal(g, T, D, std=0.3, type=ty)
        # a residual stream: larger than what a block adds, and with a few large channels
        s["x"] = _normal(g, T, D, std=2.0) * (1 + 10 * (torch.rand(D, generator=g, device=DEV) < 0.002))
        s["x"] = s["x"].to(t)
        if c["kind"] == "norm_backward":
            s["dh"], s["du"] = _normal(g, T, D, std=0.02, type=t), _normal(g, T, D, std=0.05, type=t)
    elif c["kind"] == "quantise":
        # activations: tokens of different sizes
        s["x"] = (_normal(g, c["tokens"], c["width"]) * torch.exp(_normal(g, c["tokens"], 1))).to(t)
    else:
        N, G, M, K = c["tokens"], c["groups"], c["rows"], c["width"]
        s["x"] = _normal(g, N, K, type=t)
        codes, scales = zip(*(_codes(_normal(g, M, K, std=0.02)) for _ in range(G)))
        s["w_codes"], s["w_scales"] = torch.stack(codes), torch.stack(scales)
        # rows of each group: uneven, some groups without any
        share = torch.rand(G, generator=g, device=DEV) + 0.25
        group = torch.multinomial(share, N, replacement=True, generator=g).sort().values
        s["group"] = group
        s["offsets"] = torch.searchsorted(group, torch.arange(G + 1, device=DEV)).to(torch.int32)
        s["most"] = int(s["offsets"].diff().max())
    return s


def _gather(rows, place):
    """rows[place] in 32 bits, zeros where place is -1."""
    return torch.where((place >= 0).unsqueeze(-1), rows[place.clamp(min=0).long()].float(), torch.zeros((), device=DEV))


def _plain_dispatch(s, c):
    offsets, sorted_slot, slot_pos = _sorted(s["idx"], c["experts"])
    token = torch.div(sorted_slot, c["k"], rounding_mode="floor")
    rows = _gather(s["x"], token).to(s["x"].dtype)
    out = dict(offsets=offsets, sorted_slot=sorted_slot, slot_pos=slot_pos, rows=rows)
    if c["back"]:
        out["dx"] = _gather(s["d_rows"], slot_pos).sum(1).to(s["x"].dtype)
    return out


def _plain_combine(s, c):
    t = s["y_rows"].dtype
    w = s["gates"]
    picked = _gather(s["y_rows"], s["slot_pos"])
    out = dict(y=(w.unsqueeze(-1) * picked).sum(1).to(t))
    if c["back"]:
        out["d_gates"] = (picked * s["dy"].float().unsqueeze(1)).sum(-1)
        slot = s["sorted_slot"]
        weight = w.reshape(-1)[slot.clamp(min=0).long()].unsqueeze(-1)
        out["d_rows"] = (weight * _gather(s["dy"], torch.div(slot, c["k"], rounding_mode="floor"))).to(t)
    return out


def _gate(s, c):
    return {"none": 1.0, "channel": s["gate"], "token": None if s["gate"] is None else s["gate"].unsqueeze(-1)}[c["gate"]]


def _plain_norm(s, c):
    x, y = s["x"].float(), s["y"].float()
    y_hat = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    h = (RES_SCALE * x + _gate(s, c) * s["w_post"] * y_hat).to(s["x"].dtype)
    f = h.float()  # the next block's norm reads what is stored
    u = (s["w_pre"] * f / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)).to(s["x"].dtype)
    return dict(h=h, u=u)


def _norm_gradients(h, y, dh, du, w_post, w_pre, gate, kind):
    """Gradients of h = RES_SCALE x + gate w_post y / rms(y) and u = w_pre h / rms(h), in the type of the arguments."""
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    h_hat = h * r
    g = du * w_pre
    total = dh + r * (g - h_hat * (g * h_hat).mean(-1, keepdim=True))
    q = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    y_hat = y * q
    p = total * gate * w_post
    out = dict(dx=RES_SCALE * total, dy=q * (p - y_hat * (p * y_hat).mean(-1, keepdim=True)),
               dw_pre=(du * h_hat).sum(0), dw_post=(total * gate * y_hat).sum(0))
    if kind == "channel":
        out["d_gate"] = (total * w_post * y_hat).sum(0)
    elif kind == "token":
        out["d_gate"] = (total * w_post * y_hat).sum(-1)
    return out


def _plain_norm_backward(s, c):
    out = _norm_gradients(s["x"].float(), s["y"].float(), s["dh"].float(), s["du"].float(), s["w_post"], s["w_pre"], _gate(s, c), c["gate"])
    out["dx"], out["dy"] = out["dx"].to(s["x"].dtype), out["dy"].to(s["y"].dtype)
    return out


def _by_group(x, s, c, w):
    """x [N][K] times each row's group's matrix of w [G][M][K]."""
    if c["groups"] == 1:
        return x @ w[0].T
    first = s["offsets"][:-1].long()
    at = first.unsqueeze(1) + torch.arange(s["most"], device=DEV)
    held = at < s["offsets"][1:].long().unsqueeze(1)
    padded = torch.where(held.unsqueeze(-1), x[at.clamp(max=c["tokens"] - 1)], torch.zeros((), device=DEV, dtype=x.dtype))
    out = torch.bmm(padded, w.transpose(1, 2))
    return out[s["group"], torch.arange(c["tokens"], device=DEV) - first[s["group"]]]


def _plain(s, c):
    if c["kind"] == "dispatch":
        return _plain_dispatch(s, c)
    if c["kind"] == "combine":
        return _plain_combine(s, c)
    if c["kind"] == "norm":
        return _plain_norm(s, c)
    if c["kind"] == "norm_backward":
        return _plain_norm_backward(s, c)
    if c["kind"] == "quantise":
        return _decode(*_encode(s["x"])).to(s["x"].dtype)
    return _by_group(_decode(*_encode(s["x"])), s, c, _values(s["w_codes"], s["w_scales"])).to(TYPES[c["out"]])


def _own(s, c):
    import moe_expert_layer_top16_gb300 as moe

    if c["kind"] == "dispatch":
        offsets, sorted_slot, slot_pos = moe.sort_by_expert(s["idx"], c["experts"])
        rows = moe.permute(s["x"], slot_pos, out=s["rows"])
        out = dict(offsets=offsets, sorted_slot=sorted_slot, slot_pos=slot_pos, rows=rows)
        if c["back"]:
            out["dx"] = moe.permute_backward(s["d_rows"], slot_pos)
        return out
    if c["kind"] == "combine":
        out = dict(y=moe.unpermute(s["y_rows"], s["slot_pos"], s["gates"]))
        if c["back"]:
            out["d_rows"], out["d_gates"] = moe.unpermute_backward(s["dy"], s["y_rows"], s["slot_pos"], s["gates"], out=s["rows"])
        return out
    if c["kind"] == "norm":
        h, u = moe.block_norm(s["x"], s["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per=c["gate"], res_scale=RES_SCALE, eps=EPS)
        return dict(h=h, u=u)
    if c["kind"] == "norm_backward":
        got = moe.block_norm_backward(s["dh"], s["du"], s["x"], s["y"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_per=c["gate"], res_scale=RES_SCALE, eps=EPS)
        return {k: v for k, v in got.items() if v is not None}
    codes, scales = moe.mxfp4_quantize(s["x"])
    if c["kind"] == "quantise":
        return moe.mxfp4_decode(codes, scales, s["x"].dtype)
    if c["groups"] == 1:
        return moe.mx4_gemm(s["w_codes"][0], s["w_scales"][0], codes, scales, out_dtype=TYPES[c["out"]])
    return moe.mx4_gemm(s["w_codes"], s["w_scales"], codes, scales, offsets=s["offsets"], out_dtype=TYPES[c["out"]])


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


def _exact_values(x):
    """x in MXFP4, from the definition: the scale is the power of two two below the block's largest one, and each magnitude takes the nearest level."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    power = (top.view(torch.int64) >> 52) - 1023  # the exponent field of a double: floor(log2) of any value here
    step = torch.exp2((power - 2).clamp(-127, 127).double())
    a, v = b.abs(), torch.zeros_like(b)
    for below, above in zip(LEVELS[:-1], LEVELS[1:]):
        v += (above - below) * (a > (above + below) / 2 * step)
    return torch.where(top > 0, torch.sign(b) * v * step, torch.zeros_like(b)).flatten(-2)


def exact(case, seed):
    """run()'s floating outputs in 64 bits, written apart from the plain form; None for whole numbers."""
    s, c = prepare(case, seed), case
    if c["kind"] in ("dispatch", "combine"):
        T, k, D = c["tokens"], c["k"], c["width"]
        # places by counting: slots of a lower expert, and earlier slots of the same one
        flat = s["idx"].reshape(-1).long()
        used = (flat >= 0).nonzero().squeeze(-1)
        used = used[torch.argsort(flat[used] * (T * k) + used)]  # slots by (expert, slot)
        if c["kind"] == "dispatch":
            rows = torch.zeros(T * k, D, dtype=s["x"].dtype, device=DEV)
            rows[: used.numel()] = s["x"][used // k]
            out = dict(offsets=None, sorted_slot=None, slot_pos=None, rows=rows)
            if c["back"]:
                out["dx"] = torch.zeros(T, D, dtype=torch.float64, device=DEV).index_add_(0, used // k, s["d_rows"][: used.numel()].double())
            return out
        gate = s["gates"].double().reshape(-1)[used]
        y = torch.zeros(T, D, dtype=torch.float64, device=DEV)
        y.index_add_(0, used // k, s["y_rows"][: used.numel()].double() * gate.unsqueeze(-1))
        out = dict(y=y)
        if c["back"]:
            dy = s["dy"].double()[used // k]
            out["d_gates"] = torch.zeros(T * k, dtype=torch.float64, device=DEV)
            out["d_gates"][used] = (dy * s["y_rows"][: used.numel()].double()).sum(-1)
            out["d_gates"] = out["d_gates"].view(T, k)
            out["d_rows"] = torch.zeros(T * k, D, dtype=torch.float64, device=DEV)
            out["d_rows"][: used.numel()] = dy * gate.unsqueeze(-1)
        return out
    if c["kind"] in ("norm", "norm_backward"):
        D = c["width"]
        x, y, w_post, w_pre = (s[n].double() for n in ("x", "y", "w_post", "w_pre"))
        gate = torch.ones((), dtype=torch.float64, device=DEV) if s["gate"] is None else s["gate"].double()
        gate = gate.unsqueeze(-1) if c["gate"] == "token" else gate
        if c["kind"] == "norm":
            h = RES_SCALE * x + gate * w_post * y * (y.square().sum(-1, keepdim=True) / D + EPS).rsqrt()
            f = h.to(s["x"].dtype).double()
            return dict(h=h, u=w_pre * f * (f.square().sum(-1, keepdim=True) / D + EPS).rsqrt())
        # from the Jacobian of v -> v / rms(v): (I - v v^T / (D (mean v^2 + eps))) / rms(v)
        dh, du = s["dh"].double(), s["du"].double()
        mh, my = x.square().sum(-1, keepdim=True) / D + EPS, y.square().sum(-1, keepdim=True) / D + EPS
        a = du * w_pre
        total = dh + (a - x * (a * x).sum(-1, keepdim=True) / (D * mh)) / mh.sqrt()
        b = total * gate * w_post
        out = dict(dx=RES_SCALE * total, dy=(b - y * (b * y).sum(-1, keepdim=True) / (D * my)) / my.sqrt(),
                   dw_pre=(du * x / mh.sqrt()).sum(0), dw_post=(total * gate * y / my.sqrt()).sum(0))
        if c["gate"] != "none":
            out["d_gate"] = (total * w_post * y / my.sqrt()).sum(0 if c["gate"] == "channel" else -1)
        return out
    if c["kind"] == "quantise":
        return _exact_values(s["x"])
    x = _exact_values(s["x"])
    table = torch.tensor([v for v in LEVELS] + [-v for v in LEVELS], dtype=torch.float64, device=DEV)
    out = torch.empty(c["tokens"], c["rows"], dtype=torch.float64, device=DEV)
    bounds = s["offsets"].tolist()
    for g in range(c["groups"]):
        lo, hi = bounds[g], bounds[g + 1]
        if lo < hi:
            pair = s["w_codes"][g].int()
            w = torch.empty(c["rows"], c["width"], dtype=torch.float64, device=DEV)
            w[:, 0::2], w[:, 1::2] = table[pair % 16], table[pair // 16]
            w *= torch.exp2(s["w_scales"][g].double() - 127).repeat_interleave(32, -1)
            out[lo:hi] = x[lo:hi] @ w.T
    return out
