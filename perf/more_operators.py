"""The router of a sparse MoE layer as operators of its own, and its experts' products for single tokens, as
workloads to time and compare.

Five kinds of pass, each the calls that a program makes in training or serving:

  select    the k experts of each token by their scores, and the gates
  balance   experts' counts and balance loss of each sequence, and the loss's gradient
  step      a training step's router: selection, balance loss, and the gradient of gates and loss in one pass
  product   a few rows times a matrix of four-bit weights with a scale for each group of them
  experts   a few tokens through their experts: gate, up and SiLU, then down and the weighted sum, with the
            experts' numbers as the selection gives them

Where `own` is false, run() computes them from elementary torch operations in 32 bits (the values that are ranked
in 64)."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SCALE = 2.5  # what the normalised gates are multiplied with

# E2M1's magnitudes and the midpoints between them; a value on a midpoint takes the smaller level.
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def listed():
    return [
        # one decoded token of the K3-shaped layer: 16 of 896 experts by sigmoid score and selection bias
        dict(name="select one token", kind="select", tokens=1, k=16, experts=896, type="f32", score="sigmoid", bias=True, normalize=True, pad=0.0, banned=0.0),
        # a prefill batch of the same layer
        dict(name="select prefill", kind="select", tokens=8192, k=16, experts=896, type="f32", score="sigmoid", bias=True, normalize=True, pad=0.0, banned=0.0),
        # a padded batch of a small layer with softmax gates over all experts, some experts closed for a token, odd sizes
        dict(name="select ragged", kind="select", tokens=1537, k=6, experts=61, type="f16", score="softmax", bias=False, normalize=False, pad=0.1, banned=0.1),
        # one short sequence through the small layer
        dict(name="balance one sequence", kind="balance", tokens=64, k=4, experts=32, type="f32", score="softmax", sequences=1, pad=0.0, banned=0.0),
        # a training batch of nine sequences of different lengths
        dict(name="balance batch", kind="balance", tokens=16384, k=16, experts=896, type="bf16", score="softmax", sequences=9, pad=0.05, banned=0.0),
        # a training step of the K3-shaped router, each sequence's load balanced for itself
        dict(name="step train", kind="step", tokens=8192, k=16, experts=896, type="f32", score="sigmoid", bias=True, normalize=True, sequences=4, pad=0.02, banned=0.0),
        # the same of a small layer, logits in half precision, padded, odd sizes
        dict(name="step ragged", kind="step", tokens=1001, k=6, experts=131, type="f16", score="softmax", bias=False, normalize=True, sequences=13, pad=0.2, banned=0.1),
        # one decoded token through the two shared experts' gate and up (2 x 2 x 2048 rows)
        dict(name="product one token", kind="product", tokens=1, rows=8192, width=7168, type="bf16", out="bf16", format="mxfp4", group=32, scales="e8m0"),
        # eight decoded tokens and a large matrix, weights as integers with a scale for 128
        dict(name="product eight tokens", kind="product", tokens=8, rows=65536, width=7168, type="f16", out="f16", format="int4", group=128, scales="f16"),
        # activations in 32 bits, rows and groups of odd numbers
        dict(name="product odd", kind="product", tokens=3, rows=1001, width=1056, type="f32", out="f32", format="int4", group=32, scales="f32"),
        # one decoded token through its 16 of 896 experts
        dict(name="experts one token", kind="experts", tokens=1, k=16, experts=896, inner=512, width=3584, type="bf16", drop=0.0),
        # a small decode batch on one of 14 expert-parallel slices: slots of other slices' experts are dropped
        dict(name="experts slice", kind="experts", tokens=16, k=16, experts=64, inner=512, width=3584, type="bf16", drop=0.75),
    ]


def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("select", "balance", "step", "product", "product", "experts"))
    t = rng.choice(("bf16", "f16", "f32"))
    if kind in ("select", "balance", "step"):
        k = rng.choice((1, 2, 4, 6, 8, 16, 32))
        experts = max(2 * k, _size(rng, 8, 1024))
        if rng.random() < 0.5:
            experts = (experts + 31) // 32 * 32
        c = dict(kind=kind, tokens=_size(rng, 1, min(16384, 4096 * 896 // experts)), k=k, experts=experts, type=t, score=rng.choice(("sigmoid", "softmax")),
                 pad=rng.choice((0.0, 0.0, 0.1, 0.5)), banned=rng.choice((0.0, 0.0, 0.1)))
        if kind != "balance":
            c.update(bias=c["score"] == "sigmoid" and rng.random() < 0.7, normalize=rng.random() < 0.7)
        if kind != "select":
            c.update(sequences=min(c["tokens"], _size(rng, 1, 64)))
        return c
    if kind == "product":
        form = rng.choice(("mxfp4", "int4"))
        group = 32 if form == "mxfp4" else rng.choice((32, 64, 128))
        width = group * _size(rng, 1, 8192 // group)
        rows = _size(rng, 1, min(65536, 16384 * 7168 // width))
        return dict(kind=kind, tokens=rng.choice((1, 1, 2, _size(rng, 3, 8), _size(rng, 8, 24))), rows=rows, width=width, type=t, out=rng.choice((t, "f32")),
                    format=form, group=group, scales="e8m0" if form == "mxfp4" else rng.choice(("bf16", "f16", "f32")))
    k = rng.choice((1, 2, 4, 8, 16))
    return dict(kind=kind, tokens=_size(rng, 1, 16), k=k, experts=_size(rng, k, 64), inner=32 * _size(rng, 1, 32), width=32 * _size(rng, 2, 112), type=t,
                drop=rng.choice((0.0, 0.0, 0.5)))


BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e8m0": 1}


def work(c):
    T = c["tokens"]
    if c["kind"] in ("select", "balance", "step"):
        E, k = c["experts"], c["k"]
        matrix = T * E * BYTES[c["type"]]
        if c["kind"] == "select":  # the logits in, numbers and gates out
            return {"bytes": matrix + 8 * T * k + T + (4 * E if c["bias"] else 0), "flops": 4 * T * E}
        if c["kind"] == "balance":  # the logits and the experts' numbers in; the gradient and the counts out
            return {"bytes": 2 * matrix + 4 * T * k + c["sequences"] * (4 * E + 12), "flops": 12 * T * E}
        return {"bytes": 2 * matrix + 12 * T * k + T + c["sequences"] * (4 * E + 12) + (4 * E if c["bias"] else 0), "flops": 16 * T * E}
    if c["kind"] == "product":
        M, K = c["rows"], c["width"]
        weights = M * K / 2 + M * (K // c["group"]) * BYTES[c["scales"]]
        return {"bytes": weights + T * K * BYTES[c["type"]] + T * M * BYTES[c["out"]], "flops": 2 * T * M * K}
    L, I, b = c["width"], c["inner"], BYTES[c["type"]]
    slots = T * c["k"] * (1.0 - c["drop"])
    touched = c["experts"] * (1.0 - (1.0 - 1.0 / c["experts"]) ** slots) if c["drop"] else c["experts"] * (1.0 - (1.0 - c["k"] / c["experts"]) ** T)
    return {"bytes": touched * 3 * I * L * 17 / 32 + 2 * T * L * b + 8 * T * c["k"] + 2 * slots * I * b, "flops": 6 * slots * I * L}


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, type=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(type)


def _mxfp4(w):
    """MXFP4 of w [..., K]: packed codes [..., K/2] and E8M0 scales [..., K/32]."""
    b = w.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax).exponent - 3).clamp(-127, 127), torch.full_like(amax, -127, dtype=torch.int32))
    level = torch.bucketize(torch.ldexp(b.abs(), -e.unsqueeze(-1)), torch.tensor(MIDS, device=w.device), out_int32=True)
    code = (level + 8 * torch.signbit(b)).to(torch.uint8).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _int4(w, group, type):
    """w [..., K] as integers 0 to 15 that stand for -8 to 7, two to a byte, times a scale of `type` for each group of them."""
    b = w.float().unflatten(-1, (-1, group))
    scale = (b.abs().amax(-1) / 7).to(type)
    code = (torch.round(b / scale.float().unsqueeze(-1)).clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), scale


def prepare(case, seed):
    c, g = case, _generator(seed)
    t, T = TYPES[c["type"]], c["tokens"]
    s = dict(case=case)
    if c["kind"] in ("select", "balance", "step"):
        E, k = c["experts"], c["k"]
        # scores with an uneven popularity of the experts; a closed expert has minus infinity
        logits = _normal(g, T, E, std=1.5) + _normal(g, E, std=0.5)
        if c["banned"]:
            logits = torch.where(torch.rand(T, E, generator=g, device=DEV) < c["banned"], torch.full_like(logits, -math.inf), logits)
        s["logits"] = logits.to(t)
        valid = T - int(T * c["pad"])  # the rows behind are padding
        s["mask"] = torch.arange(T, device=DEV) < valid if c["pad"] else None
        if c["kind"] != "balance":
            s["bias"] = _normal(g, E, std=0.05) if c["bias"] else None
            s["d_gates"] = _normal(g, T, k, std=0.02)
        if c["kind"] != "select":
            cuts = (torch.rand(c["sequences"] - 1, generator=g, device=DEV) * valid).long().sort().values
            s["sequences"] = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), cuts, torch.full((1,), valid, device=DEV)]).to(torch.int32)
            # a loss's weight; in half precision with the scale that keeps gradients of this size above its smallest numbers
            s["d_loss"] = 0.01 * (32 * T if c["type"] == "f16" else 1) * (0.5 + torch.rand(c["sequences"], generator=g, device=DEV))
        if c["kind"] == "balance":
            idx = (s["logits"].float() + _normal(g, T, E, std=0.01)).topk(k, dim=1).indices.to(torch.int32)
            s["idx"] = idx if s["mask"] is None else torch.where(s["mask"].unsqueeze(1), idx, torch.full_like(idx, -1))
    elif c["kind"] == "product":
        w = _normal(g, c["rows"], c["width"], std=0.02)
        s["codes"], s["scales"] = _mxfp4(w) if c["format"] == "mxfp4" else _int4(w, c["group"], TYPES[c["scales"]])
        s["x"] = _normal(g, T, c["width"], type=t)
    else:
        E, k, I, L = c["experts"], c["k"], c["inner"], c["width"]
        for name, shape in (("gate", (I, L)), ("up", (I, L)), ("down", (L, I))):
            step = max(1, (1 << 27) // (I * L))
            parts = [_mxfp4(_normal(g, min(step, E - e), *shape, std=0.05)) for e in range(0, E, step)]
            s[name] = tuple(torch.cat(p) for p in zip(*parts))
        s["x"] = _normal(g, T, L, type=t)
        idx = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
        s["idx"] = torch.where(torch.rand(T, k, generator=g, device=DEV) < c["drop"], torch.full_like(idx, -1), idx) if c["drop"] else idx
        gates = torch.rand(T, k, generator=g, device=DEV) + 0.05
        s["gates"] = SCALE * gates / gates.sum(1, keepdim=True)
    return s


# ------------------------------------------------------------------ the plain forms
def _open(l):
    """Logits in 32 bits: what is not a number is closed like minus infinity, plus infinity the largest number."""
    return torch.nan_to_num(l.float(), nan=-math.inf, posinf=torch.finfo(torch.float32).max, neginf=-math.inf)


def _sigmoid(l):
    return 1 / (1 + torch.exp(-l))


def _shares(l, score):
    """Each expert's share of a token's score [T][E]; zeros in rows without an open expert."""
    if score == "softmax":
        top = l.amax(-1, keepdim=True)
        p = torch.where(l > -math.inf, torch.exp(l - torch.where(top > -math.inf, top, torch.zeros_like(top))), torch.zeros_like(l))
    else:
        p = _sigmoid(l)
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, torch.zeros_like(p))


def _plain_select(s, c):
    l, k = _open(s["logits"]), c["k"]
    key = l.double()
    if c["bias"]:
        key = torch.where(key > -math.inf, _sigmoid(key) + s["bias"].double(), key)
    if s["mask"] is not None:
        key = torch.where(s["mask"].unsqueeze(1), key, torch.full_like(key, -math.inf))
    key, order = torch.sort(key, dim=-1, descending=True, stable=True)
    kept = key[:, :k] > -math.inf
    order = order[:, :k]
    picked = l.gather(1, order)
    if c["score"] == "sigmoid":
        w = _sigmoid(picked)
    elif c["normalize"]:
        w = torch.exp(picked - picked[:, :1])
    else:
        w = _shares(l, "softmax").gather(1, order)
    w = torch.where(kept, w, torch.zeros_like(w))
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return torch.where(kept, order, torch.full_like(order, -1)).to(torch.int32), SCALE * w


def _sequence_of(s, c):
    """The sequence of each row, behind the last: their number."""
    offsets = s["sequences"].long()
    row = torch.arange(c["tokens"], device=DEV)
    seq = torch.searchsorted(offsets, row, right=True) - 1
    return torch.where(row < offsets[-1], seq, torch.full_like(seq, c["sequences"]))


def _plain_balance(s, c, idx):
    S, E, k = c["sequences"], c["experts"], c["k"]
    seq = torch.where((idx >= 0).any(1), _sequence_of(s, c), torch.full((c["tokens"],), S, device=DEV))
    p = _shares(_open(s["logits"]), c["score"])
    sums = torch.zeros(S + 1, E, dtype=torch.float64, device=DEV).index_add_(0, seq, p.double())[:S]
    tokens = torch.zeros(S + 1, dtype=torch.int32, device=DEV).index_add_(0, seq, torch.ones_like(seq, dtype=torch.int32))[:S]
    slot = seq.unsqueeze(1) * (E + 1) + torch.where(idx >= 0, idx, torch.full_like(idx, E)).long()
    counts = torch.zeros((S + 1) * (E + 1), dtype=torch.int32, device=DEV).index_add_(0, slot.flatten(), torch.ones(slot.numel(), dtype=torch.int32, device=DEV))
    counts = counts.view(S + 1, E + 1)[:S, :E].contiguous()
    n = tokens.double().clamp(min=1)
    loss = (E / k * (counts.double() * sums).sum(1) / (n * n)).float()
    return loss, counts, tokens


def _plain_gradient(s, c, idx, counts, tokens, d_gates=None):
    T, S, E, k = c["tokens"], c["sequences"], c["experts"], c["k"]
    l = _open(s["logits"])
    rest = 1 - _sigmoid(l) if c["score"] == "sigmoid" else torch.ones_like(l)
    p = _shares(l, c["score"])
    seq = torch.where((idx >= 0).any(1), _sequence_of(s, c), torch.full((T,), S, device=DEV))
    n = tokens.float().clamp(min=1)
    a = (s["d_loss"] * (E / k) / (n * n)).unsqueeze(1) * counts.float()
    a = torch.cat([a, torch.zeros(1, E, device=DEV)])[seq]
    d = p * rest * (a - (p * a).sum(1, keepdim=True))
    if d_gates is not None:
        at = idx.clamp(min=0).long()
        picked = torch.where(idx >= 0, l.gather(1, at), torch.full_like(d_gates, -math.inf))
        g = torch.where(idx >= 0, SCALE * d_gates, torch.zeros_like(d_gates))
        if c["normalize"]:
            w = _shares(picked, c["score"])
            v = w * (g - (w * g).sum(1, keepdim=True))
        else:
            w = torch.where(idx >= 0, _sigmoid(picked) if c["score"] == "sigmoid" else p.gather(1, at), torch.zeros_like(g))
            v = w * g
            if c["score"] == "softmax":
                d = d - p * v.sum(1, keepdim=True)
        if c["score"] == "sigmoid":
            v = v * (1 - _sigmoid(picked))
        d = d.scatter_add(1, at, v)
    return d.to(s["logits"].dtype)


def _values(codes, scales, form):
    """What packed codes and their scales stand for, in 32 bits."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (scales.shape[-1], -1))
    if form == "int4":
        return ((code.float() - 8) * scales.float().unsqueeze(-1)).flatten(-2)
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)[code.int()]
    return torch.ldexp(level, (scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _plain_experts(s, c):
    idx = s["idx"].flatten()
    at, kept = idx.clamp(min=0).long(), (idx >= 0).unsqueeze(-1)
    x = s["x"].float().repeat_interleave(c["k"], 0).unsqueeze(-1)
    pick = lambda name: _values(s[name][0][at], s[name][1][at], "mxfp4")  # noqa: E731
    gate, up = torch.bmm(pick("gate"), x).squeeze(-1), torch.bmm(pick("up"), x).squeeze(-1)
    h = torch.where(kept, gate * _sigmoid(gate) * up, torch.zeros_like(gate)).to(s["x"].dtype)
    o = torch.bmm(pick("down"), h.float().unsqueeze(-1)).squeeze(-1)
    y = torch.where(kept, s["gates"].flatten().unsqueeze(-1) * o, torch.zeros_like(o)).view(c["tokens"], c["k"], -1).sum(1)
    return dict(h=h.view(c["tokens"], c["k"], -1), y=y.to(s["x"].dtype))


def _plain(s, c):
    if c["kind"] == "product":
        return (s["x"].float() @ _values(s["codes"], s["scales"], c["format"]).T).to(TYPES[c["out"]])
    if c["kind"] == "experts":
        return _plain_experts(s, c)
    if c["kind"] == "balance":
        loss, counts, tokens = _plain_balance(s, c, s["idx"])
        return dict(loss=loss, counts=counts, tokens=tokens, d_logits=_plain_gradient(s, c, s["idx"], counts, tokens))
    idx, gates = _plain_select(s, c)
    if c["kind"] == "select":
        return dict(idx=idx, gates=gates)
    loss, counts, tokens = _plain_balance(s, c, idx)
    return dict(idx=idx, gates=gates, loss=loss, counts=counts, tokens=tokens, d_logits=_plain_gradient(s, c, idx, counts, tokens, s["d_gates"]))


# ------------------------------------------------------------------ the framework's calls
def _own(s, c):
    import moe_expert_layer_top16_gb300 as moe

    if c["kind"] == "product":
        return moe.w4_matvec(s["x"], s["codes"], s["scales"], out_dtype=TYPES[c["out"]])
    if c["kind"] == "experts":
        h = moe.w4_matvec(s["x"], *s["gate"], up=s["up"], idx=s["idx"])
        return dict(h=h, y=moe.w4_matvec(h, *s["down"], idx=s["idx"], weights=s["gates"]))
    if c["kind"] == "balance":
        loss, counts, tokens = moe.balance_loss(s["logits"], s["idx"], score=c["score"], sequences=s["sequences"])
        d = moe.router_backward(s["logits"], s["idx"], d_loss=s["d_loss"], counts=counts, tokens=tokens, sequences=s["sequences"], score=c["score"])
        return dict(loss=loss, counts=counts, tokens=tokens, d_logits=d)
    idx, gates = moe.select_experts(s["logits"], c["k"], bias=s["bias"], score=c["score"], normalize=c["normalize"], scale=SCALE, mask=s["mask"])
    if c["kind"] == "select":
        return dict(idx=idx, gates=gates)
    loss, counts, tokens = moe.balance_loss(s["logits"], idx, score=c["score"], sequences=s["sequences"])
    d = moe.router_backward(s["logits"], idx, d_gates=s["d_gates"], d_loss=s["d_loss"], counts=counts, tokens=tokens, sequences=s["sequences"], score=c["score"],
                            normalize=c["normalize"], scale=SCALE)
    return dict(idx=idx, gates=gates, loss=loss, counts=counts, tokens=tokens, d_logits=d)


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_selection(s, c):
    """The selection by k rounds of the largest key, the lowest number among equals; -1 where none is left."""
    l = s["logits"].double()
    key = l if s["bias"] is None else torch.where(l > -math.inf, torch.sigmoid(l) + s["bias"].double(), l)
    key = key.clone()
    if s["mask"] is not None:
        key[~s["mask"]] = -math.inf
    number, picks = torch.arange(c["experts"], device=DEV), []
    for _ in range(c["k"]):
        top = key.amax(1, keepdim=True)
        e = torch.where(key == top, number, c["experts"]).amin(1)
        picks.append(torch.where(top.squeeze(1) > -math.inf, e, torch.full_like(e, -1)))
        key.scatter_(1, e.unsqueeze(1), -math.inf)
    return torch.stack(picks, 1)


def _exact_gates(l, idx, c):
    """Gates [T][k] as a function of the logits (float64, with gradient)."""
    chosen = l.gather(1, idx.clamp(min=0)).masked_fill(idx < 0, -math.inf)
    some = (idx >= 0).any(1, keepdim=True)
    if c["normalize"]:
        w = torch.softmax(chosen.masked_fill(~some, 0.0), 1) if c["score"] == "softmax" else torch.sigmoid(chosen) / torch.sigmoid(chosen).sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.sigmoid(chosen) if c["score"] == "sigmoid" else torch.softmax(l, 1).gather(1, idx.clamp(min=0))
    return SCALE * w.masked_fill(idx < 0, 0.0)


def _exact_losses(l, idx, s, c):
    """One loss for each sequence, as a function of the logits."""
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l) / torch.sigmoid(l).sum(1, keepdim=True)
    cuts, losses = s["sequences"].tolist(), []
    for a, b in zip(cuts[:-1], cuts[1:]):
        used = (idx[a:b] >= 0).any(1)
        n = int(used.sum())
        if not n:
            losses.append((l[:1] * 0).nan_to_num().sum())
            continue
        held = torch.bincount(idx[a:b][idx[a:b] >= 0], minlength=c["experts"]).double()
        losses.append(c["experts"] / (c["k"] * n) * (held * p[a:b][used].mean(0)).sum())
    return torch.stack(losses)


def _exact_matrix(codes, scales, form):
    """The matrix that codes [M][K/2] and scales stand for."""
    pair = codes.int()
    w = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=DEV)
    if form == "int4":
        w[..., 0::2], w[..., 1::2] = pair % 16 - 8, pair // 16 - 8
        each = scales.double()
    else:
        table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=DEV)
        w[..., 0::2], w[..., 1::2] = table[pair % 16], table[pair // 16]
        each = torch.exp2(scales.double() - 127)
    return w * each.repeat_interleave(w.shape[-1] // scales.shape[-1], -1)


def exact(case, seed):
    """run()'s floating outputs in 64 bits, written apart from the plain form; None for whole numbers."""
    s, c = prepare(case, seed), case
    if c["kind"] == "product":
        out = torch.empty(c["tokens"], c["rows"], dtype=torch.float64, device=DEV)
        for a in range(0, c["rows"], 8192):  # a part of the matrix at a time
            out[:, a:a + 8192] = s["x"].double() @ _exact_matrix(s["codes"][a:a + 8192], s["scales"][a:a + 8192], c["format"]).T
        return out
    if c["kind"] == "experts":
        T, k = c["tokens"], c["k"]
        h = torch.zeros(T, k, c["inner"], dtype=torch.float64, device=DEV)
        y = torch.zeros(T, c["width"], dtype=torch.float64, device=DEV)
        for t, row in enumerate(s["idx"].tolist()):
            x = s["x"][t].double()
            for j, e in enumerate(row):
                if e >= 0:
                    m = {n: _exact_matrix(s[n][0][e], s[n][1][e], "mxfp4") for n in ("gate", "up", "down")}
                    h[t, j] = torch.nn.functional.silu(m["gate"] @ x) * (m["up"] @ x)
                    # the second product reads what the first one stored
                    y[t] += s["gates"][t, j].double() * (m["down"] @ h[t, j].to(s["x"].dtype).double())
        return dict(h=h, y=y)
    l = s["logits"].double().requires_grad_()
    if c["kind"] == "select":
        return dict(idx=None, gates=_exact_gates(l, _exact_selection(s, c), c).detach())
    idx = s["idx"].long() if c["kind"] == "balance" else _exact_selection(s, c)
    loss = _exact_losses(l, idx, s, c)
    total = (loss * s["d_loss"].double()).sum()
    out = dict(loss=loss.detach(), counts=None, tokens=None)
    if c["kind"] == "step":
        gates = _exact_gates(l, idx, c)
        total = total + (gates * s["d_gates"].double()).sum()
        out = dict(idx=None, gates=gates.detach(), **out)
    out["d_logits"] = torch.autograd.grad(total, l)[0]
    return out
